"""Scores that fall outside fp32's range, and running maxima that rise far and often.

Queries and keys are small whole numbers, so that every score is exact in fp32 (before the scale) and the
errors are those of the scale, the exponentials and the roundings of the weights and the output.
"""
import math

import numpy as np
import pytest
import torch

import mla_inputs as I
from oracle import mla_oracle as O
from tests.gpu_common import BF16_MAX_ABS, BF16_REL_L2, FP32_REL, errors, to_np
from tests.test_gpu_multi_token import KW, TYPES, Chunk, Prompt, _cu

pytestmark = pytest.mark.gpu
SCALE = 1 / math.sqrt(192)
LOWEST = float(torch.finfo(torch.bfloat16).min)


def _whole(shape, seed):
    return torch.randint(-1, 2, shape, generator=I.generator(seed)).float()


def _close(got, ref, dtype, big, keys, what):
    """`big`: the largest |score| in log2 units; its rounding to fp32 and the maximum's, 2^-24 each, are
    errors of the weight's logarithm on the fp32 path (on the bf16 path a common factor of all).  A sum of
    n positive weights takes n roundings of at most 2^-24 of itself, all to one side where the addends are
    equal, as many are here: n 2^-24 of the sum, 2e-3 for 33000 keys (2e-5 was seen there)."""
    rel, mx = errors(got, ref)
    if dtype == torch.bfloat16:
        assert rel <= BF16_REL_L2 and mx <= BF16_MAX_ABS, f"{what}: {rel:.3e} {mx:.3e}"
    else:
        tol = FP32_REL + 2 * big * 2 ** -24 * math.log(2) + keys * 2 ** -24
        assert rel <= tol and mx <= tol, f"{what}: {rel:.3e} {mx:.3e} of {tol:.3e}"


def _lse_tol(big, keys):
    # the score's and the maximum's roundings, the scale's own (two), the result's, and the sum's
    return 1e-4 + 5 * big * 2 ** -24 + keys * 2 ** -24


def _check_prompt(c, o, l, big, first=0, heads=(0, 13)):
    for b, n in enumerate(c.tokens):
        at = int(_cu(c.tokens)[b])
        mask = np.triu(np.ones((n, n), bool), 1)
        for h in heads:
            g = h // (c.H // c.Hk)
            k = np.concatenate([O.f64(c.kv[at:at + n, g, :128]), O.f64(c.kr[at:at + n, :64])], 1)
            s = np.where(mask, -np.inf, O.f64(c.q[at:at + n, h]) @ k.T * SCALE)
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            ref = e @ O.f64(c.kv[at:at + n, g, 128:]) / e.sum(1, keepdims=True)
            lse = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
            _close(to_np(o[at:at + n, h])[first:], ref[first:], c.dtype, big, n, f"o b={b} h={h}")
            np.testing.assert_allclose(to_np(l[at:at + n, h])[first:], lse[first:], rtol=0, atol=_lse_tol(big, n))


def _check_chunk(c, o, l, big):
    for b, n in enumerate(c.tokens):
        rows = O.gather_rows(c.cache.pool, c.cache.page_table[b].numpy(), c.lens[b])
        for i in range(n):
            t, vis = int(_cu(c.tokens)[b]) + i, c.lens[b] - n + i + 1
            q = O.f64(c.q[t])
            ro, rl = O.latent_attention(q[:, :512], q[:, 512:], rows[:vis, :512], rows[:vis, 512:])
            for cols in (slice(0, 1), slice(1, 512)):  # (the first column is far larger than the rest)
                _close(to_np(o[t])[:, cols], ro[:, cols], c.dtype, big, vis, f"o_lat b={b} i={i} {cols}")
            np.testing.assert_allclose(to_np(l[t]), rl, rtol=0, atol=_lse_tol(big, vis))


# A score of 4 x the type's lowest number is -inf in fp32: its key has no weight.  The keys behind such a
# beginning score -2048 / sqrt(192) or so, 2^-213 of a reference of 0.
FAR, FAR_LOG2 = -2048.0, 2100 * SCALE / math.log(2)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("tokens,extra", [([300], 0), ([260, 500], 0), ([900], 3196)],
                         ids=["one", "two", "pairs"])
def test_prompt_scores_of_minus_infinity_first(dtype, tokens, extra):
    c = Prompt(91, tokens, 16, 2, dtype, extra=extra)
    c.q, c.kr = (_whole(x.shape, 92 + i).to(dtype) for i, x in enumerate((c.q, c.kr)))
    c.kv[..., :128] = _whole(c.kv[..., :128].shape, 94).to(dtype)
    c.q[..., 0], c.kv[..., 0] = 4.0, FAR / 4
    for b in range(len(tokens)):
        at = int(_cu(tokens)[b])
        c.kv[at:at + 256, :, 0] = LOWEST
    o, l, st = c.run()
    assert st == 0
    _check_prompt(c, o, l, FAR_LOG2, first=256)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_chunk_scores_of_minus_infinity_first(dtype, splits):
    c = Chunk(95, [3, 20], [600, 900], 16, dtype)
    c.q = _whole(c.q.shape, 96).to(dtype)
    c.q[..., 0] = 4.0
    for b, n in enumerate(c.lens):
        for j in range(n):
            row = c.cache.pool[int(c.cache.page_table[b, j // 64]), j % 64]
            row[:] = _whole(row.shape, 97 + 1000 * b + j).to(dtype)
            row[0] = LOWEST if j < 300 else FAR / 4
    o, l, st = c.run(splits)
    assert st == 0
    _check_chunk(c, o, l, FAR_LOG2)


# A maximum that rises by more than 2^8 again and again, in every row: the output so far is scaled down
# each time.  Key j scores about 96 floor(j / step) / sqrt(192), 10 in log2 units a step, to 1024 / sqrt(192).
def _rising(j, step):
    return min(96.0 * (j // step), 1024.0)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("tokens,extra", [([1500], 0), ([700, 900], 0), ([1500], 2596), ([1900], 2196)],
                         ids=["one", "two", "pairs", "pairs2"])
def test_prompt_rising_maxima(dtype, tokens, extra):
    c = Prompt(101, tokens, 16, 2, dtype, extra=extra)
    c.q, c.kr = (_whole(x.shape, 102 + i).to(dtype) for i, x in enumerate((c.q, c.kr)))
    c.kv[..., :128] = _whole(c.kv[..., :128].shape, 104).to(dtype)
    c.q[..., 0] = 4.0
    for b, n in enumerate(tokens):
        at = int(_cu(tokens)[b])
        for j in range(n):
            c.kv[at + j, :, 0] = _rising(j, 100) / 4
    o, l, st = c.run()
    assert st == 0
    _check_prompt(c, o, l, 1100 * SCALE / math.log(2))


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("tokens,lens,splits", [([5], [1500], 1), ([5], [1500], 0), ([20, 1, 9], [1200, 700, 900], 1),
                                                ([20, 1, 9], [1200, 700, 900], 3),
                                                ([9, 9], [33000, 1400], 4)],  # (teams: two tiles each)
                         ids=lambda v: "-".join(map(str, v)) if isinstance(v, list) else str(v))
def test_chunk_rising_maxima(dtype, tokens, lens, splits):
    c = Chunk(105, tokens, lens, 16, dtype)
    c.q = _whole(c.q.shape, 106).to(dtype)
    c.q[..., 0] = 4.0
    for b, n in enumerate(lens):
        step = max(100, n // 16 // 100 * 100)
        rows = _whole((n, 576), 107 + b)
        rows[:, 0] = torch.tensor([_rising(j, step) / 4 for j in range(n)])
        for p in range((n + 63) // 64):
            part = rows[64 * p:64 * p + 64].to(dtype)
            c.cache.pool[int(c.cache.page_table[b, p]), :len(part)] = part
    o, l, st = c.run(splits)
    assert st == 0
    _check_chunk(c, o, l, 1100 * SCALE / math.log(2))


def test_chunk_longest_sequence():
    """The most rows that a page table may name, 2^31 - 64, all on one page: the page's own softmax, with a
    sum (2^31 - 64) / 64 times its own.  A part adds up to 2^31 / 24 / 128 blocks' sums one behind the other,
    each with a rounding of 2^-24 of the sum at most, all to one side: 4.2% of it."""
    import mla_latent_kv_37_b200 as M
    from tests.gpu_common import dev
    pages = (1 << 25) - 1
    g = I.generator(111)
    q, row = torch.randn(1, 16, 576, generator=g).bfloat16(), torch.randn(64, 576, generator=g).bfloat16()
    o = torch.empty(1, 16, 512, dtype=torch.bfloat16, device="cuda")
    l = torch.empty(1, 16, device="cuda")
    d = M.dims(1, 16)
    M.mla_chunk_attn(d, dev(q), dev(row)[None], torch.zeros(1, pages, dtype=torch.int32, device="cuda"),
                     dev(_cu([1])), dev(torch.tensor([64 * pages], dtype=torch.int32)), o,
                     M.chunk_workspace(d, 1), lse=l)
    assert M.mla_get_status() == 0
    r = O.f64(row)
    _, lse = O.latent_attention(O.f64(q[0])[:, :512], O.f64(q[0])[:, 512:], r[:, :512], r[:, 512:])
    np.testing.assert_allclose(to_np(l[0].cpu()), lse + math.log(pages), rtol=0, atol=0.042 + 1e-3)
    assert torch.isfinite(o).all()
