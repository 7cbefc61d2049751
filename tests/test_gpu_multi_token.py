"""Several new tokens per sequence on the GPU: mla_append_rows, mla_prompt_attn and mla_chunk_attn
against plain 64-bit forms, at the lengths, masks, head counts and layouts where they can go wrong,
and a run of them together.

Tolerances.  A rounding to a type t is off by at most finfo(t).eps / 2 of the value.
  * Attention, bf16: the weights p and the output are rounded to bf16 once each, so an output is off
    by at most 2^-8 (sum_j p_j |v_j|) + 2^-8 |o|; over many elements the two add up as independent
    errors of uniform size, sqrt(2 / 3) 2^-8 = 3.2e-3 of the norm: the framework's 5e-3 (and 2e-2 of
    the largest value) hold.  fp32: the framework's 1e-5.
  * lse: fp32 products and sums of at most 576 terms of exact bf16 (or fp32) products, |s| < 20, so
    576 x 2^-24 x 20 = 7e-4 at the very worst and sqrt(576) x 2^-24 x 20 = 3e-5 as a random walk.
  * Rotation: |cos, sin error| <= 2e-7 and three fp32 roundings, 4e-7 (|x0| + |x1|), and half a step
    of the storage type.
"""
import math

import numpy as np
import pytest
import torch

import mla_inputs as I
from oracle import mla_oracle as O
from tests.gpu_common import assert_close, dev, round_to, to_np

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]
LSE_TOL = 1e-4
KW = dict(ids=lambda v: str(v).replace("torch.", ""))


def _cu(tokens):
    return torch.tensor(np.concatenate([[0], np.cumsum(tokens)]), dtype=torch.int32)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype)


# --------------------------------------------------------------------------------------------
# rows into the cache
# --------------------------------------------------------------------------------------------
class Append:
    def __init__(self, seed, tokens, lens, H, dtype, extra=0):
        g = I.generator(seed)
        self.tokens, self.lens, self.H, self.dtype = tokens, lens, H, dtype
        T = self.T = sum(tokens) + extra
        self.cache = I.paged_cache(seed + 1, [max(n, 1) for n in lens], [0] * len(lens), dtype=dtype)
        # views of wider tensors, as projections leave them
        self.ckr = _randn(g, T, 600, dtype=dtype)
        self.q = _randn(g, T, H, 192, dtype=dtype)

    def run(self, q_to="cat", with_q=True, with_k=True, table=None, lens=None):
        import mla_latent_kv_37_b200 as M
        d = M.dims(len(self.tokens), self.H, dtype=self.dtype)
        ckr, q, pool = dev(self.ckr), dev(self.q), dev(self.cache.pool)
        k_rope = torch.full((self.T, 64), 7.0, dtype=self.dtype, device="cuda") if with_k else None
        cat = torch.full((self.T, self.H, 576), 7.0, dtype=self.dtype, device="cuda")
        q_in = q[..., 128:]
        q_out = q_in if q_to == "place" else cat[..., 512:]
        M.mla_append_rows(d, ckr[:, :512], ckr[:, 512:576], dev(_cu(self.tokens)),
                          dev(torch.tensor(lens or self.lens, dtype=torch.int32)),
                          dev(self.cache.page_table if table is None else table), pool,
                          k_rope=k_rope, q_rope=q_in if with_q else None,
                          q_rope_out=q_out if with_q else None)
        st = M.mla_get_status()
        return pool.cpu(), None if k_rope is None else k_rope.cpu(), q.cpu(), cat.cpu(), st

    def expected(self, skip=()):
        pool = self.cache.pool.double().clone()
        turned = {}
        for b, n in enumerate(self.tokens):
            for i in range(n):
                t, pos = int(_cu(self.tokens)[b]) + i, self.lens[b] - n + i
                if (b, i) in skip:
                    continue
                k = O.rope(self.ckr[t, 512:576].double().numpy(), pos)
                turned[t] = (k, O.rope(self.q[t, :, 128:].double().numpy(), pos))
                page = int(self.cache.page_table[b, pos // 64])
                pool[page, pos % 64, :512] = self.ckr[t, :512].double()
                pool[page, pos % 64, 512:] = torch.from_numpy(k)
        return pool, turned

    def close(self, got, exp, src):
        half = torch.finfo(self.dtype).eps / 2
        src = np.abs(src.double().numpy()).reshape(*src.shape[:-1], -1, 2).sum(-1).repeat(2, -1)
        got, exp = got.double().numpy(), np.asarray(exp)
        assert np.all(np.abs(got - exp) <= 4e-7 * src * (1 + half) + half * np.abs(exp) * (1 + 1e-6))


def _check_append(c, pool, k_rope, q_rope, skip=()):
    ref, turned = c.expected(skip)
    written = torch.zeros(ref.shape[:2], dtype=torch.bool)
    for b, n in enumerate(c.tokens):
        for i in range(n):
            if (b, i) in skip:
                continue
            pos, t = c.lens[b] - n + i, int(_cu(c.tokens)[b]) + i
            page = int(c.cache.page_table[b, pos // 64])
            written[page, pos % 64] = True
            assert torch.equal(pool[page, pos % 64, :512], c.ckr[t, :512])
            c.close(pool[page, pos % 64, 512:], turned[t][0], c.ckr[t, 512:576])
    assert torch.equal(pool[~written], c.cache.pool[~written])
    for t in range(c.T):
        if t in turned:
            if k_rope is not None:
                c.close(k_rope[t], turned[t][0], c.ckr[t, 512:576])
            if q_rope is not None:
                c.close(q_rope[t], turned[t][1], c.q[t, :, 128:])
        elif k_rope is not None:
            assert torch.all(k_rope[t] == 7.0)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("tokens,lens", [([1], [1]), ([1], [131072]), ([7, 0, 1, 65], [7, 0, 64, 200]),
                                         ([130, 3], [130, 4097]), ([1] * 40, list(range(1, 41)))])
@pytest.mark.parametrize("H", [16, 112])
def test_append_rows(dtype, tokens, lens, H):
    c = Append(11, tokens, lens, H, dtype, extra=3)  # three rows behind the last sequence
    pool, k_rope, q, cat, st = c.run()
    assert st == 0
    _check_append(c, pool, k_rope, cat[..., 512:])
    assert torch.all(cat[..., :512] == 7.0) and torch.all(cat[sum(tokens):] == 7.0)
    assert torch.equal(q, c.q)


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_append_rows_in_place_and_without_outputs(dtype):
    c = Append(12, [9, 30], [100, 30], 48, dtype)
    pool, k_rope, q, cat, st = c.run(q_to="place", with_k=False)
    assert st == 0 and torch.all(cat == 7.0)
    _check_append(c, pool, None, q[..., 128:])
    assert torch.equal(q[..., :128], c.q[..., :128])
    pool, k_rope, q, cat, st = c.run(with_q=False)
    _check_append(c, pool, k_rope, None)
    assert st == 0 and torch.equal(q, c.q) and torch.all(cat == 7.0)


def test_append_rows_many_sequences():
    # more sequences than one step of the search covers, many of them empty
    tokens = [(b * 7) % 3 for b in range(1100)]
    c = Append(13, tokens, [t + b % 5 for b, t in enumerate(tokens)], 16, torch.bfloat16)
    pool, k_rope, q, cat, st = c.run()
    assert st == 0
    _check_append(c, pool, k_rope, cat[..., 512:])


@pytest.mark.parametrize("theta", [100.0, 500000.0])
def test_append_rows_other_theta(theta):
    import mla_latent_kv_37_b200 as M
    c = Append(15, [3], [70001], 16, torch.float32)
    d = M.dims(1, 16, dtype=torch.float32, rope_theta=theta)
    k_rope = torch.empty(3, 64, device="cuda")
    M.mla_append_rows(d, dev(c.ckr)[:, :512], dev(c.ckr)[:, 512:576], dev(_cu([3])),
                      dev(torch.tensor([70001], dtype=torch.int32)), dev(c.cache.page_table),
                      dev(c.cache.pool), k_rope=k_rope)
    assert M.mla_get_status() == 0
    for i in range(3):
        c.close(k_rope[i].cpu(), O.rope(c.ckr[i, 512:576].double().numpy(), 69998 + i, theta),
                c.ckr[i, 512:576])


def test_append_rows_skips_what_has_no_slot():
    c = Append(14, [3, 2, 2], [100, 70, 5], 16, torch.bfloat16)
    table = c.cache.page_table.clone()
    table[1, 1] = c.cache.num_pages  # sequence 1's rows 68, 69 have no page
    pool, k_rope, q, cat, st = c.run(table=table)
    assert st == 0x1
    skip = {(1, 0), (1, 1)}
    _check_append(c, pool, k_rope, None, skip)
    # a length below the token count puts the first tokens in front of the cache; one past the
    # table puts the last behind it
    cap = c.cache.page_table.shape[1] * 64
    pool, k_rope, q, cat, st = c.run(lens=[2, cap + 1, 5])
    assert st == 0x8
    assert torch.all(k_rope[0] == 7.0) and torch.all(k_rope[4] == 7.0)
    assert not torch.any(k_rope[1] == 7.0) and torch.all(cat[4] == 7.0)


# --------------------------------------------------------------------------------------------
# whole prompts
# --------------------------------------------------------------------------------------------
class Prompt:
    def __init__(self, seed, tokens, H, Hk, dtype, extra=0, std=1.0):
        g = I.generator(seed)
        self.tokens, self.H, self.Hk, self.dtype = tokens, H, Hk, dtype
        T = self.T = sum(tokens) + extra
        self.q = _randn(g, T, H, 192) * std
        self.kv = _randn(g, T, Hk, 256)
        self.kr = _randn(g, T, 72) * std
        self.q, self.kv, self.kr = self.q.to(dtype), self.kv.to(dtype), self.kr.to(dtype)

    def run(self, head_major=False, scale=0.0, lse=True, stream=None):
        import mla_latent_kv_37_b200 as M
        d = M.dims(len(self.tokens), self.H, dtype=self.dtype)
        q, kv, kr = dev(self.q), dev(self.kv), dev(self.kr)
        if head_major:  # [H, T, D] storage
            q, kv = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, kv))
        o = torch.full((self.T, self.H, 128), 7.0, dtype=self.dtype, device="cuda")
        l = torch.full((self.T, self.H), 7.0, device="cuda") if lse else None
        M.mla_prompt_attn(d, q, kv[..., :128], kr[:, :64], kv[..., 128:], dev(_cu(self.tokens)), o,
                          lse=l, softmax_scale=scale)
        return o.cpu(), None if l is None else l.cpu(), M.mla_get_status()

    def check(self, o, l, scale=None, heads=None, seqs=None):
        scale = scale or 1 / math.sqrt(192)
        for b in seqs if seqs is not None else range(len(self.tokens)):
            n, at = self.tokens[b], int(_cu(self.tokens)[b])
            if n == 0:
                continue
            mask = np.triu(np.ones((n, n), bool), 1)
            for h in heads or range(self.H):
                g = h // (self.H // self.Hk)
                k = np.concatenate([O.f64(self.kv[at:at + n, g, :128]), O.f64(self.kr[at:at + n, :64])], 1)
                s = np.where(mask, -np.inf, O.f64(self.q[at:at + n, h]) @ k.T * scale)
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                ref = e @ O.f64(self.kv[at:at + n, g, 128:]) / e.sum(1, keepdims=True)
                assert_close(to_np(o[at:at + n, h]), ref, self.dtype, f"o b={b} h={h}")
                if l is not None:
                    np.testing.assert_allclose(to_np(l[at:at + n, h]), (m + np.log(e.sum(1, keepdims=True)))[:, 0],
                                               rtol=0, atol=LSE_TOL)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("tokens", [[1], [63], [64], [65], [127], [128], [129], [255], [256], [257],
                                    [1, 1, 1], [5, 0, 200, 64, 0], [300, 1, 129], [700]],
                         ids=lambda v: "-".join(map(str, v)))
def test_prompt_lengths(dtype, tokens):
    c = Prompt(21, tokens, 16, 16, dtype)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l, heads=[0, 7, 15])


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("H,Hk", [(16, 1), (16, 4), (48, 3), (96, 96), (128, 16)])
def test_prompt_heads(dtype, H, Hk):
    c = Prompt(22, [150, 70], H, Hk, dtype)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l, heads=sorted({0, 1, H // Hk - 1, H // Hk % H, H // 2, H - 1}))


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_prompt_layouts_and_scale(dtype):
    c = Prompt(23, [90, 200], 16, 8, dtype)
    a, la, _ = c.run(scale=0.1)
    c.check(a, la, scale=0.1, heads=[3, 12])
    b, lb, _ = c.run(scale=0.1, head_major=True)
    assert torch.equal(a, b) and torch.equal(la, lb)
    d, none, st = c.run(scale=0.1, lse=False)
    assert none is None and st == 0 and torch.equal(a, d)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), torch.finfo(torch.bfloat16).min])
def test_prompt_other_rows_have_no_influence(dtype, junk):
    # what lies behind the last sequence is neither read into a result nor written; what another
    # sequence holds stays there
    for tokens in ([100, 30], [128, 1], [129, 250]):
        c = Prompt(24, tokens, 16, 16, dtype, extra=5)
        a, la, _ = c.run()
        for x in (c.q, c.kv, c.kr):
            x[sum(tokens):] = junk
            x[:tokens[0]] = junk
        b, lb, st = c.run()
        n = sum(tokens)
        assert st == 0
        assert torch.equal(a[tokens[0]:n], b[tokens[0]:n])
        assert torch.equal(la[tokens[0]:n], lb[tokens[0]:n])
        assert torch.all(b[n:] == 7.0) and torch.all(lb[n:] == 7.0)
        c.check(a, la, heads=[2], seqs=[1])


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_prompt_large_logits(dtype):
    # logits of a spread of 16: the running maximum grows and the output is rescaled
    c = Prompt(25, [400], 16, 16, dtype, std=4.0)
    o, l, st = c.run()
    assert st == 0
    if dtype == torch.float32:
        # products up to |s| ~ 80: 80 x 192 x 2^-24 of a logit at worst, sqrt(192) as a walk (7e-5);
        # the weights carry that relative error
        for h in (0, 9):
            k = np.concatenate([O.f64(c.kv[:, h, :128]), O.f64(c.kr[:, :64])], 1)
            ref = O.causal_attention(O.f64(c.q[:, h]), k, O.f64(c.kv[:, h, 128:]), 1 / math.sqrt(192))
            assert np.linalg.norm(to_np(o[:, h]) - ref) <= 7e-5 * np.linalg.norm(ref)
    else:
        c.check(o, None, heads=[0, 9])


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_prompt_nan_stays_with_what_it_enters(dtype):
    c = Prompt(28, [200, 300], 16, 8, dtype)
    a, la, _ = c.run()
    c.q[250, 3, 100] = float("nan")
    b, lb, st = c.run()
    assert st == 0 and torch.isnan(b[250, 3]).all() and torch.isnan(lb[250, 3])
    keep = torch.ones(c.T, 16, dtype=torch.bool)
    keep[250, 3] = False
    assert torch.equal(a[keep], b[keep]) and torch.equal(la[keep], lb[keep])
    c.q[250, 3, 100] = 0
    c.kv[400, 2, 7] = float("nan")  # a key of key head 2: rows from its own on, heads 4 and 5
    b, lb, st = c.run()
    hit = torch.zeros(c.T, 16, dtype=torch.bool)
    hit[400:, 4:6] = True
    assert torch.isnan(b[hit]).all() and torch.isnan(lb[hit]).all()
    hit[250, 3] = True
    assert torch.equal(a[~hit], b[~hit]) and torch.equal(la[~hit], lb[~hit])


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_prompt_many_sequences(dtype):
    tokens = [(7 * b) % 13 for b in range(700)] + [260]
    c = Prompt(29, tokens, 16, 4, dtype)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l, heads=[0, 13], seqs=[*range(0, 700, 37), 1, 2, 700])


def test_prompt_long_fp32():
    c = Prompt(30, [1500, 900], 16, 2, torch.float32)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l, heads=[0, 15])


def test_prompt_long():
    c = Prompt(26, [3000, 2100], 16, 2, torch.bfloat16)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l, heads=[0, 15])


@pytest.mark.parametrize("tokens,H,Hk", [([4096], 16, 16), ([2100, 2000], 16, 1), ([8000, 37, 4300], 16, 2), ([4737, 0, 7655], 32, 4)],
                         ids=lambda v: str(v))
def test_prompt_pairs(tokens, H, Hk):
    # long on average: two SMs share every product; sequences that end inside a tile, a short one and
    # an empty one among them
    c = Prompt(44, tokens, H, Hk, torch.bfloat16, extra=3)
    c.q[sum(tokens):] = c.kv[sum(tokens):] = c.kr[sum(tokens):] = float("nan")
    o, l, st = c.run()
    assert st == 0
    c.check(o, l, heads=[1, H - 1])
    assert torch.all(o[sum(tokens):] == 7.0) and torch.all(l[sum(tokens):] == 7.0)
    o2, none, st = c.run(lse=False)
    assert st == 0 and none is None and torch.equal(o, o2)


def test_prompt_pairs_large_logits_and_waits_that_run_out(monkeypatch):
    c = Prompt(45, [4200], 16, 16, torch.bfloat16, std=4.0)
    o, l, st = c.run()
    assert st == 0
    c.check(o, None, heads=[0, 9])
    monkeypatch.setenv("MLA_WAIT_NS", "1")
    assert c.run()[2] in (0, 0x4)  # (a wait that succeeds at one of its first tries does not run out)
    monkeypatch.delenv("MLA_WAIT_NS")
    o2, l2, st = c.run()
    assert st == 0 and torch.equal(o, o2) and torch.equal(l, l2)


def test_prompt_bad_offsets_stay_in_bounds():
    import mla_latent_kv_37_b200 as M
    c = Prompt(27, [40, 30, 20], 16, 16, torch.bfloat16)
    d = M.dims(3, 16)
    for cu in ([0, 40, 30, 90], [0, 40, 70, 1000], [-5, 40, 70, 90], [50, 0, 90, 90]):
        o = torch.empty(90, 16, 128, dtype=torch.bfloat16, device="cuda")
        kv = dev(c.kv)
        M.mla_prompt_attn(d, dev(c.q), kv[..., :128], dev(c.kr[:, :64]), kv[..., 128:],
                          dev(torch.tensor(cu, dtype=torch.int32)), o)
        assert M.mla_get_status() == 0x2


# --------------------------------------------------------------------------------------------
# a chunk over the paged cache
# --------------------------------------------------------------------------------------------
class Chunk:
    def __init__(self, seed, tokens, lens, H, dtype, extra=0, sentinel=I.SENTINEL, scale=1.0):
        self.tokens, self.lens, self.H, self.dtype = tokens, lens, H, dtype
        self.T = sum(tokens) + extra
        self.q = I.query_cat(seed, self.T, H, scale, dtype)
        self.cache = I.paged_cache(seed + 1, lens, lens, scale, dtype, sentinel=sentinel)

    def run(self, splits=0, out=None, table=None, lens=None, cu=None, scale=0.0):
        import mla_latent_kv_37_b200 as M
        d = M.dims(len(self.tokens), self.H, dtype=self.dtype)
        o = torch.full((self.T, self.H, 512), 7.0, dtype=out or self.dtype, device="cuda")
        l = torch.full((self.T, self.H), 7.0, device="cuda")
        ws = M.chunk_workspace(d, self.T, splits)
        ws.fill_(255)  # nothing in it needs to start at zero
        M.mla_chunk_attn(d, dev(self.q), dev(self.cache.pool),
                         dev(self.cache.page_table if table is None else table),
                         dev(_cu(self.tokens) if cu is None else cu),
                         dev(torch.tensor(lens or self.lens, dtype=torch.int32)), o, ws, lse=l,
                         num_splits=splits, softmax_scale=scale)
        return o.cpu(), l.cpu(), M.mla_get_status()

    def check(self, o, l, every=1, scale=None, dtype=None):
        for b, n in enumerate(self.tokens):
            rows = O.gather_rows(self.cache.pool, self.cache.page_table[b].numpy(), self.lens[b])
            at = int(_cu(self.tokens)[b])
            got, ref, got_l, ref_l = [], [], [], []
            for i in sorted({*range(0, n, every), n - 1} if n else ()):
                vis = self.lens[b] - n + i + 1
                if vis <= 0:
                    assert torch.all(o[at + i] == 0) and torch.all(torch.isneginf(l[at + i]))
                    continue
                q = O.f64(self.q[at + i])
                ro, rl = O.latent_attention(q[:, :512], q[:, 512:], rows[:vis, :512], rows[:vis, 512:], scale)
                got.append(to_np(o[at + i])); ref.append(ro)
                got_l.append(to_np(l[at + i])); ref_l.append(rl)
            if got:
                assert_close(np.stack(got), np.stack(ref), dtype or self.dtype, f"o_lat b={b}")
                np.testing.assert_allclose(np.stack(got_l), np.stack(ref_l), rtol=0, atol=LSE_TOL)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("tokens,lens", [([1], [1]), ([1], [64]), ([1], [129]), ([2], [65]), ([3], [3]),
                                         ([65], [65]), ([5], [400]), ([130], [200]),
                                         ([1, 4, 0, 33], [300, 64, 90, 129]),
                                         ([3, 2, 1], [2, 0, 0]), ([70], [20])],
                         ids=lambda v: "-".join(map(str, v)))
def test_chunk_lengths(dtype, tokens, lens):
    c = Chunk(31, tokens, lens, 16, dtype, extra=2)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l)
    assert torch.all(o[sum(tokens):] == 7.0) and torch.all(l[sum(tokens):] == 7.0)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("H", [16, 48, 64, 96, 112, 128])
def test_chunk_heads(dtype, H):
    c = Chunk(32, [7, 1, 2], [150, 40, 257], H, dtype)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64, 500, 0])
def test_chunk_splits(dtype, splits):
    c = Chunk(33, [5, 1, 20, 0, 3], [1500, 700, 20, 100, 1], 48, dtype)
    o, l, st = c.run(splits)
    assert st == 0
    c.check(o, l)
    o2, l2, _ = c.run(splits)
    assert torch.equal(o, o2) and torch.equal(l, l2)


def test_chunk_fp32_output_of_bf16():
    c = Chunk(34, [4, 1, 9], [900, 2000, 9], 128, torch.bfloat16)
    a, la, _ = c.run(out=torch.float32)
    c.check(a, la)
    b, lb, _ = c.run()
    assert torch.equal(a.to(torch.bfloat16), b) and torch.equal(la, lb)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("junk", [float("nan"), float("inf"), float(torch.finfo(torch.bfloat16).min)])
def test_chunk_unused_slots_have_no_influence(dtype, junk):
    # slots behind a sequence's last row, in its last page and in pages the table does not use yet
    for tokens, lens, H in (([3, 1, 40], [70, 129, 40], 32), ([1, 2], [1, 65], 128), ([5], [1000], 16)):
        a = Chunk(35, tokens, lens, H, dtype, sentinel=0.0).run()
        b = Chunk(35, tokens, lens, H, dtype, sentinel=junk).run()
        assert a[2] == 0 and b[2] == 0
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_chunk_nan_stays_with_its_sequence(dtype):
    # a NaN in a query row or in a cached row shows in what it enters (split or not) and nowhere else
    c = Chunk(41, [3, 2, 1], [700, 900, 64], 16, dtype)
    good, lg, _ = c.run()
    c.q[1, 3, 5] = float("nan")
    o, l, st = c.run()
    assert st == 0 and torch.isnan(o[1, 3]).all() and torch.isnan(l[1, 3])
    keep = torch.ones(c.T, 16, dtype=torch.bool)
    keep[1, 3] = False
    assert torch.equal(o[keep], good[keep]) and torch.equal(l[keep], lg[keep])
    c.q[1, 3, 5] = 0
    c.cache.pool[int(c.cache.page_table[1, 3]), 7, 9] = float("nan")
    for splits in (0, 1):
        o, l, st = c.run(splits)
        assert st == 0 and torch.isnan(o[3:5]).all() and torch.isnan(l[3:5]).all()
        assert not torch.isnan(o[:3]).any() and not torch.isnan(o[5]).any()


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_chunk_scale_and_large_logits(dtype):
    c = Chunk(36, [6], [500], 16, dtype, scale=2.0)
    o, l, st = c.run(scale=0.05)
    assert st == 0
    c.check(o, l, scale=0.05)


def test_chunk_equals_decode_for_single_tokens():
    import mla_latent_kv_37_b200 as M
    lens = [1, 64, 700, 4097, 0]
    c = Chunk(37, [1] * 5, lens, 128, torch.bfloat16)
    o, l, st = c.run(out=torch.float32)
    d = M.dims(5, 128)
    o2 = torch.empty(5, 128, 512, device="cuda")
    l2 = torch.empty(5, 128, device="cuda")
    M.mla_decode_attn(d, dev(c.q), dev(c.cache.pool), dev(c.cache.page_table),
                      dev(torch.tensor(lens, dtype=torch.int32)), o2, M.workspace(d), lse=l2)
    assert st == 0 and M.mla_get_status() == 0
    assert_close(to_np(o), to_np(o2), torch.bfloat16, "against mla_decode_attn")
    assert torch.equal(torch.isneginf(l), torch.isneginf(l2.cpu()))
    fin = torch.isfinite(l)
    np.testing.assert_allclose(to_np(l[fin]), to_np(l2.cpu()[fin]), rtol=0, atol=2e-4)


def test_chunk_long_context():
    c = Chunk(38, [3, 260], [30000, 5000], 128, torch.bfloat16)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l, every=37)


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("n,H,lens", [(4, 128, [2500, 2501, 9000, 7, 0, 20000, 3, 64]), (9, 16, [40000, 130, 128]),
                                      (5, 48, [16500, 1, 16500, 5, 6]), (2, 96, [33000])],
                         ids=lambda v: str(v) if isinstance(v, int) else "")
def test_chunk_equal_counts_over_long_caches(dtype, n, H, lens):
    # as many tiles in every sequence: teams of parts, ranges that end inside a sequence, tiles of one
    # sequence that see different numbers of blocks, sequences without rows
    c = Chunk(42, [n] * len(lens), lens, H, dtype, extra=1)
    for splits in (0, 8, 16):
        o, l, st = c.run(splits)
        assert st == 0
        c.check(o, l, every=3)
        assert torch.all(o[-1] == 7.0) and torch.all(l[-1] == 7.0)


def test_chunk_shared_pages():
    # two sequences that begin alike share the pages of their beginning
    c = Chunk(43, [3, 2], [500, 450], 64, torch.bfloat16)
    c.cache.page_table[1, :4] = c.cache.page_table[0, :4]
    o, l, st = c.run()
    assert st == 0
    c.check(o, l)


def test_chunk_many_sequences():
    n = 1300
    tokens = [b % 3 for b in range(n)]
    c = Chunk(39, tokens, [t + b % 70 for b, t in enumerate(tokens)], 16, torch.bfloat16)
    o, l, st = c.run()
    assert st == 0
    c.check(o, l)


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_chunk_bad_pages_lengths_and_offsets(dtype):
    c = Chunk(40, [2, 3], [200, 100], 16, dtype)
    good, lg, _ = c.run()
    table = c.cache.page_table.clone()
    table[0, 1] = c.cache.num_pages + 7
    o, l, st = c.run(table=table)
    assert st == 0x1 and torch.equal(o[2:], good[2:])
    table[0, 1] = -1
    assert c.run(table=table)[2] == 0x1
    assert c.run(lens=[c.cache.page_table.shape[1] * 64 + 1, 100])[2] & 0x2
    assert c.run(lens=[-3, 100])[2] == 0x2
    for cu in ([0, 4, 3], [0, 2, 99], [-1, 2, 5], [5, 0, 5]):
        assert c.run(cu=torch.tensor(cu, dtype=torch.int32))[2] == 0x2
    o, l, st = c.run()
    assert st == 0 and torch.equal(o, good) and torch.equal(l, lg)


# --------------------------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------------------------
def test_prompt_then_chunks_agree_with_the_whole():
    """A prompt's rows enter the cache, its attention runs in the form without absorption; the same
    prompt over the cache in chunks, absorbed, gives the same heads (associativity)."""
    import mla_latent_kv_37_b200 as M
    tokens, H, T = [130, 77], 16, 207
    g = I.generator(51)
    w = I.weights(52, H, 1024)
    c_kv, k_r, q = (_randn(g, *s, dtype=torch.bfloat16) for s in ((T, 512), (T, 64), (T, H, 192)))
    d, cu, lens = M.dims(2, H), dev(_cu(tokens)), dev(torch.tensor(tokens, dtype=torch.int32))
    cache = I.paged_cache(53, tokens, [0, 0])
    pool, table = dev(cache.pool), dev(cache.page_table)
    q, k_rope = dev(q), torch.empty(T, 64, dtype=torch.bfloat16, device="cuda")
    M.mla_append_rows(d, dev(c_kv), dev(k_r), cu, lens, table, pool, k_rope=k_rope,
                      q_rope=q[..., 128:], q_rope_out=q[..., 128:])
    w_uk, w_uv = O.f64(w.w_uk).reshape(H, 128, 512), O.f64(w.w_uv).reshape(H, 128, 512)
    k_nope = np.einsum("tc,hdc->thd", O.f64(c_kv), w_uk)
    v = np.einsum("tc,hdc->thd", O.f64(c_kv), w_uv)
    as_bf16 = lambda x: dev(torch.from_numpy(x).to(torch.bfloat16))
    o = torch.empty(T, H, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    M.mla_prompt_attn(d, q, as_bf16(k_nope), k_rope, as_bf16(v), cu, o, lse=lse)
    # chunks: the first 100 / 50 tokens, then the rest, each over the cache as it then stands
    q_lat = np.einsum("thd,hdc->thc", O.f64(q[..., :128]), w_uk)
    q_cat = torch.cat((as_bf16(q_lat), q[..., 128:]), -1).contiguous()
    got, got_l = np.empty((T, H, 128)), torch.empty(T, H)
    for lo, hi in (((0, 0), (100, 50)), ((100, 50), (130, 77))):
        idx = torch.cat([torch.arange(int(cu[b]) + lo[b], int(cu[b]) + hi[b]) for b in range(2)])
        n = [hi[b] - lo[b] for b in range(2)]
        ol = torch.empty(len(idx), H, 512, device="cuda")
        ll = torch.empty(len(idx), H, device="cuda")
        M.mla_chunk_attn(d, q_cat[dev(idx)].contiguous(), pool, table, dev(_cu(n)),
                         dev(torch.tensor(hi, dtype=torch.int32)), ol,
                         M.chunk_workspace(d, len(idx)), lse=ll)
        got[idx] = np.einsum("thc,hdc->thd", to_np(ol), w_uv)
        got_l[idx] = ll.cpu()
    assert M.mla_get_status() == 0
    # both sides round: keys, values, weights and outputs on one, queries and weights on the other
    rel = np.linalg.norm(to_np(o) - got) / np.linalg.norm(got)
    assert rel <= 1e-2, rel
    assert torch.all((lse.cpu() - got_l).abs() < 2e-2)


def test_proposed_tokens_through_a_whole_layer():
    """Verification of proposed tokens with the framework's own calls: every token is a batch row of
    mla_append_absorb and mla_out_proj, and mla_chunk_attn attends to the sequences' tokens at once;
    against the oracle's step, token by token."""
    import mla_latent_kv_37_b200 as M
    H, D, hist, n = 16, 1024, [130, 5, 64], [3, 1, 4]
    T = sum(n)
    w, h = I.weights(61, H, D), I.hidden(62, T, D)
    cache = I.paged_cache(63, [a + b for a, b in zip(hist, n)], hist)
    pool, table = dev(cache.pool), dev(cache.page_table)
    seq = torch.repeat_interleave(torch.arange(3), torch.tensor(n))
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(hist, n)]).int()
    dt, db = M.dims(T, H, D), M.dims(3, H, D)
    ws, q_cat = M.workspace(dt), torch.empty(T, H, 576, dtype=torch.bfloat16, device="cuda")
    o_lat = torch.empty(T, H, 512, device="cuda")
    out = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    M.mla_append_absorb(dt, dev(h), dev(w.w_dkv), dev(w.w_kr), dev(w.w_q), dev(w.w_uk), dev(pos),
                        table[dev(seq)].contiguous(), pool, q_cat, ws)
    M.mla_chunk_attn(db, q_cat, pool, table, dev(_cu(n)), dev(torch.tensor(hist).int() + dev(torch.tensor(n)).cpu().int()),
                     o_lat, M.chunk_workspace(db, T))
    M.mla_out_proj(dt, o_lat, dev(w.w_uv), ws, w_o=dev(w.w_o), out=out)
    assert M.mla_get_status() == 0
    t = 0
    for b in range(3):
        rows = O.gather_rows(cache.pool, cache.page_table[b].numpy(), hist[b])
        for i in range(n[b]):
            ref = O.decode_step(h[t], w, rows, hist[b] + i, H, round_row=round_to(torch.bfloat16))
            assert_close(to_np(out[t]), ref["out"], torch.bfloat16, f"b={b} i={i}")
            rows = np.concatenate([rows, O.f64(ref["row"])[None]])
            t += 1


def test_graphs_streams_and_shared_workspace():
    """Captured and replayed on another stream, two graphs sharing one workspace in turn, with
    inputs that change between replays."""
    import mla_latent_kv_37_b200 as M
    c = Chunk(71, [4, 1, 30], [600, 90, 30], 128, torch.bfloat16)
    e = Chunk(72, [2, 2, 2], [2000, 64, 7], 128, torch.bfloat16)
    d = M.dims(3, 128)
    ws = M.chunk_workspace(d, max(c.T, e.T))
    side = torch.cuda.Stream()
    graphs = []
    for x in (c, e):
        args = [dev(x.q), dev(x.cache.pool), dev(x.cache.page_table), dev(_cu(x.tokens)),
                dev(torch.tensor(x.lens, dtype=torch.int32)),
                torch.zeros(x.T, 128, 512, dtype=torch.bfloat16, device="cuda")]
        p = Prompt(73, x.tokens, 16, 16, torch.bfloat16)
        pargs = [dev(p.q), dev(p.kv), dev(p.kr[:, :64].contiguous()), dev(_cu(p.tokens)),
                 torch.zeros(p.T, 16, 128, dtype=torch.bfloat16, device="cuda")]

        def call(args=args, pargs=pargs):
            M.mla_chunk_attn(d, *args, ws)
            q, kv, kr, cu, o = pargs
            M.mla_prompt_attn(M.dims(3, 16), q, kv[..., :128], kr, kv[..., 128:], cu, o)

        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                call()
        graphs.append((g, x, p, args, pargs))
    for _ in range(2):
        for g, x, p, args, pargs in graphs:
            args[-1].zero_()
            pargs[-1].zero_()
            args[0].neg_()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                g.replay()
    torch.cuda.synchronize()
    assert M.mla_get_status() == 0
    for g, x, p, args, pargs in graphs:
        o, l, _ = x.run()
        assert torch.equal(args[-1].cpu(), o)  # the query's sign flipped twice
        assert torch.equal(pargs[-1].cpu(), p.run()[0])


def test_calls_on_two_streams_at_once():
    import mla_latent_kv_37_b200 as M
    c = Chunk(74, [40, 3], [3000, 2000], 128, torch.bfloat16)
    p = Prompt(75, [700, 90], 32, 32, torch.bfloat16)
    d, dp = M.dims(2, 128), M.dims(2, 32)
    streams = [torch.cuda.Stream() for _ in range(3)]
    args = [dev(c.q), dev(c.cache.pool), dev(c.cache.page_table), dev(_cu(c.tokens)),
            dev(torch.tensor(c.lens, dtype=torch.int32))]
    q, kv, kr, cu = dev(p.q), dev(p.kv), dev(p.kr[:, :64].contiguous()), dev(_cu(p.tokens))
    outs = [torch.zeros(c.T, 128, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    po = torch.zeros(p.T, 32, 128, dtype=torch.bfloat16, device="cuda")
    ws = [M.chunk_workspace(d, c.T) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            M.mla_chunk_attn(d, *args, outs[i], ws[i], stream=streams[i])  # without lse
        M.mla_prompt_attn(dp, q, kv[..., :128], kr, kv[..., 128:], cu, po, stream=streams[2])
    torch.cuda.synchronize()
    assert M.mla_get_status() == 0
    o, l, _ = c.run()
    assert torch.equal(outs[0].cpu(), o) and torch.equal(outs[1].cpu(), o)
    assert torch.equal(po.cpu(), p.run()[0])


def test_waits_that_run_out_are_reported(monkeypatch):
    # a limit of 1 ns ends every wait that does not succeed at one of its first tries: the kernels
    # unwind, say so in the status word, and the next calls are as ever
    c = Chunk(76, [5, 300, 1], [700, 900, 64], 48, torch.bfloat16)
    p = Prompt(77, [300, 70, 1000], 16, 16, torch.bfloat16)
    good, lse, st = c.run()
    prompt = p.run()
    assert st == 0 and prompt[2] == 0
    monkeypatch.setenv("MLA_WAIT_NS", "1")
    raised = 0
    for _ in range(3):
        raised |= c.run()[2]
        raised |= p.run()[2]
    assert raised in (0, 0x4)
    monkeypatch.delenv("MLA_WAIT_NS")
    o, l, st = c.run()
    assert st == 0 and torch.equal(o, good) and torch.equal(l, lse)
    again = p.run()
    assert again[2] == 0 and torch.equal(again[0], prompt[0]) and torch.equal(again[1], prompt[1])


def test_no_tokens_do_nothing():
    import mla_latent_kv_37_b200 as M
    d = M.dims(2, 16)
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    cu, lens = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    table, pool = torch.zeros(2, 1, dtype=torch.int32, device="cuda"), z(1, 64, 576)
    n0 = M.mla_launch_count()
    M.mla_append_rows(d, z(0, 512), z(0, 64), cu, lens, table, pool)
    M.mla_prompt_attn(d, z(0, 16, 192), z(0, 4, 128), z(0, 64), z(0, 4, 128), cu, z(0, 16, 128))
    M.mla_chunk_attn(d, z(0, 16, 576), pool, table, cu, lens, z(0, 16, 512), M.chunk_workspace(d, 0))
    assert M.mla_launch_count() == n0 and M.mla_get_status() == 0
