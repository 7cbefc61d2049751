"""Offsets (cu_tokens) that decrease or pass n_tokens are reported wherever they stand: behind the first
32 sequences, which the kernels look at together, and in entries that no token's search meets.  The
sequences in front of the fault are as ever, and the next call reports nothing."""
import pytest
import torch

from tests.gpu_common import dev

pytestmark = pytest.mark.gpu


def _cases(B, T):
    """cu of B sequences of a token each, then the same with a fault; T is n_tokens."""
    good = list(range(B + 1))
    yield good, 0
    for at in (1, 31, 32, 33, B // 2, B):  # (entry B is the last)
        if at > B:
            continue
        cu = list(good)
        cu[at] = T + 1  # passes n_tokens; what follows decreases
        yield cu, at
        cu = list(good)
        cu[at] = max(at - 3, -1) if at > 1 else -1  # decreases
        yield cu, at


def _run(call, cu):
    import mla_latent_kv_37_b200 as M
    call(dev(torch.tensor(cu, dtype=torch.int32)))
    return M.mla_get_status()


def _check(call, B, T):
    for cu, at in _cases(B, T):
        assert _run(call, cu) == (0x2 if at else 0), (at, cu[max(0, at - 1):at + 2])
    assert _run(call, list(range(B + 1))) == 0


@pytest.mark.parametrize("B", [2, 33, 40, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_prompt_offsets(dtype, B):
    import mla_latent_kv_37_b200 as M
    T, d = B + 5, M.dims(B, 16, dtype=dtype)
    q, k, kr = (torch.zeros(*s, dtype=dtype, device="cuda") for s in ((T, 16, 192), (T, 2, 128), (T, 64)))
    o = torch.empty(T, 16, 128, dtype=dtype, device="cuda")
    _check(lambda cu: M.mla_prompt_attn(d, q, k, kr, k, cu, o), B, T)


def test_prompt_offsets_on_pairs():
    import mla_latent_kv_37_b200 as M
    B, T = 40, 40 * 4096  # (pairs are taken from 4096 tokens a sequence on; most lie behind the last one)
    d = M.dims(B, 16)
    q, k, kr = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
                for s in ((T, 16, 192), (T, 1, 128), (T, 64)))
    o = torch.empty(T, 16, 128, dtype=torch.bfloat16, device="cuda")
    _check(lambda cu: M.mla_prompt_attn(d, q, k, kr, k, cu, o), B, T)


@pytest.mark.parametrize("B", [2, 33, 40, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_append_offsets(dtype, B):
    import mla_latent_kv_37_b200 as M
    T, d = B + 5, M.dims(B, 16, dtype=dtype)
    c, k = (torch.ones(T, w, dtype=dtype, device="cuda") for w in (512, 64))
    pool = torch.zeros(B, 64, 576, dtype=dtype, device="cuda")
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.full((B,), 64, dtype=torch.int32, device="cuda")
    _check(lambda cu: M.mla_append_rows(d, c, k, cu, lens, table, pool), B, T)


def test_append_offsets_between_the_steps_of_the_search():
    # 64 sequences: a token's search looks at every second offset first, and none of them is wrong here
    import mla_latent_kv_37_b200 as M
    B, T = 64, 640
    d = M.dims(B, 16)
    c, k = (torch.ones(T, w, dtype=torch.bfloat16, device="cuda") for w in (512, 64))
    pool = torch.zeros(B, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.full((B,), 64, dtype=torch.int32, device="cuda")
    for at, wrong in ((5, 33), (63, 600), (64, 650)):
        cu = list(range(0, T + 1, 10))
        cu[at] = wrong
        assert _run(lambda x: M.mla_append_rows(d, c, k, x, lens, table, pool), cu) == 0x2, at


def test_chunk_offsets():
    import mla_latent_kv_37_b200 as M
    B, T = 300, 305  # (more than the plan looks at together)
    for dtype in (torch.bfloat16, torch.float32):
        d = M.dims(B, 16, dtype=dtype)
        q = torch.zeros(T, 16, 576, dtype=dtype, device="cuda")
        pool = torch.zeros(1, 64, 576, dtype=dtype, device="cuda")
        table = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
        lens = torch.full((B,), 64, dtype=torch.int32, device="cuda")
        o, ws = torch.empty(T, 16, 512, dtype=dtype, device="cuda"), M.chunk_workspace(d, T)
        _check(lambda cu: M.mla_chunk_attn(d, q, pool, table, cu, lens, o, ws), B, T)
