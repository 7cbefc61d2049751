"""Waits that run out in the bf16 kernels of the calls with several new tokens per sequence.

MLA_TEST_STALL makes one warp of each CTA, or of one CTA of each pair, wait on a barrier nothing arrives
on, with a limit of 20 ms: every other role then waits for it in vain at some place, the kernel says so
in the status word and returns, and the next call is bit-equal to the one before.

A kernel that unwinds waits for its copies and products in flight, on a limit of 200 ms of its own that
raises the same status.  So the time shows whether it found them: every stalled role gives up within
20 ms of the last one that it hung on, 100 ms in all, and one wait in vain for a copy takes 200 ms.
"""
import pytest
import torch

from tests.gpu_common import dev
from tests.test_gpu_multi_token import Chunk, Prompt, _cu

pytestmark = pytest.mark.gpu
LIMIT_MS = 150


class Calls:
    """A call with its tensors on the device, whose time is the kernels'."""

    def __init__(self, call, outputs):
        self.call, self.outputs = call, outputs

    def __call__(self):
        import mla_latent_kv_37_b200 as M
        for x in self.outputs:
            x.fill_(7.0)
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        self.call()
        b.record()
        torch.cuda.synchronize()
        return [x.cpu() for x in self.outputs], M.mla_get_status(), a.elapsed_time(b)

    def stalled(self, monkeypatch, stall):
        monkeypatch.setenv("MLA_TEST_STALL", str(stall))
        monkeypatch.setenv("MLA_WAIT_NS", "20000000")
        try:
            return self()[1:]
        finally:
            monkeypatch.delenv("MLA_TEST_STALL")
            monkeypatch.delenv("MLA_WAIT_NS")


def _chunk(c, splits=0):
    import mla_latent_kv_37_b200 as M
    d = M.dims(len(c.tokens), c.H)
    ws = M.chunk_workspace(d, c.T, splits)
    args = [dev(x) for x in (c.q, c.cache.pool, c.cache.page_table, _cu(c.tokens),
                             torch.tensor(c.lens, dtype=torch.int32))]
    o = torch.empty(c.T, c.H, 512, dtype=torch.bfloat16, device="cuda")
    l = torch.empty(c.T, c.H, device="cuda")
    return Calls(lambda: M.mla_chunk_attn(d, *args, o, ws, lse=l, num_splits=splits), [o, l])


def _prompt(p):
    import mla_latent_kv_37_b200 as M
    d = M.dims(len(p.tokens), p.H)
    q, kv, kr, cu = dev(p.q), dev(p.kv), dev(p.kr), dev(_cu(p.tokens))
    o = torch.empty(p.T, p.H, 128, dtype=torch.bfloat16, device="cuda")
    l = torch.empty(p.T, p.H, device="cuda")
    return Calls(lambda: M.mla_prompt_attn(d, q, kv[..., :128], kr[:, :64], kv[..., 128:], cu, o, lse=l),
                 [o, l])


def _check_stalls(calls, monkeypatch, stalls):
    good, st, _ = calls()
    assert st == 0
    for stall in stalls:
        st, ms = calls.stalled(monkeypatch, stall)
        assert st == 0x4, stall
        assert ms < LIMIT_MS, (stall, ms)
        again, st, _ = calls()
        assert st == 0, stall
        assert all(torch.equal(a, b) for a, b in zip(good, again)), stall


# warps 0 ... 3 softmax, 4 queries and keys, 5 S, 6 values, 7 O (both issuers the first CTA's alone)
CHUNK_STALLS = [1, 104, 202, 5, 105, 205, 7, 107, 207, 6, 108]


@pytest.mark.parametrize("tokens,lens,H,splits", [
    ([5, 30, 1], [700, 900, 64], 48, 0),       # short: a ragged block or two a part
    ([40, 3], [3000, 2000], 128, 0),           # the rings go round before a part ends
    ([9, 2, 3], [129, 300, 3], 16, 1)])        # several segments a part, ragged ends between them
def test_chunk_waits_that_run_out(monkeypatch, tokens, lens, H, splits):
    _check_stalls(_chunk(Chunk(81, tokens, lens, H, torch.bfloat16), splits), monkeypatch, CHUNK_STALLS)


# warps 0 ... 7 softmax (four a tile), 8 producer, 9 and 10 the tiles' issuers (the first CTA's)
PAIR_STALLS = [1, 104, 203, 5, 208, 9, 109, 209, 10, 11, 110]


@pytest.mark.parametrize("tokens", [[2011], [1920], [130], [17]])
def test_prompt_pair_waits_that_run_out(monkeypatch, tokens):
    # (rows behind the last sequence make it 4096 tokens, for which pairs are taken)
    p = Prompt(82, tokens, 16, 4, torch.bfloat16, extra=4096 - sum(tokens))
    _check_stalls(_prompt(p), monkeypatch, PAIR_STALLS)


# warps 0 ... 7 softmax (four a tile), 8 producer, 9 issuer
@pytest.mark.parametrize("tokens", [[1], [130], [300, 70, 1000]])
def test_prompt_waits_that_run_out(monkeypatch, tokens):
    _check_stalls(_prompt(Prompt(83, tokens, 16, 4, torch.bfloat16)), monkeypatch, [1, 4, 5, 8, 9, 10])
