"""The calls with several new tokens per sequence beside the framework's other calls, in captured graphs with
inputs that change, and twice with the same inputs."""
import numpy as np
import pytest
import torch

import mla_inputs as I
from tests.gpu_common import dev, to_np
from tests.test_gpu_multi_token import KW, TYPES, Append, Chunk, Prompt, _check_append, _cu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES, **KW)
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
def test_append_rows_as_cache_append_writes_them(dtype, theta):
    """The same row by both calls, the projections of mla_cache_append being identities: each is within
    4e-7 (|x0| + |x1|) and half a step of the rotation, so they are within twice that of one another."""
    import mla_latent_kv_37_b200 as M
    pos = [0, 1, 63, 64, 1000, 4097, 30011, 65535, 100003, 131071]
    B = len(pos)
    h = torch.randn(B, 576, generator=I.generator(121)).to(dtype)
    eye = torch.eye(576, dtype=dtype)
    d = M.dims(B, 16, 576, dtype=dtype, rope_theta=theta)
    table = torch.arange(B, dtype=torch.int32)[:, None].expand(B, 2048).contiguous()
    pools = [torch.zeros(B, 64, 576, dtype=dtype, device="cuda") for _ in range(2)]
    at = torch.tensor(pos, dtype=torch.int32)
    M.mla_cache_append(d, dev(h), dev(eye[:512].contiguous()), dev(eye[512:].contiguous()), dev(at), dev(table),
                       pools[0], M.workspace(d))
    M.mla_append_rows(d, dev(h)[:, :512], dev(h)[:, 512:], dev(_cu([1] * B)), dev(at + 1), dev(table), pools[1])
    assert M.mla_get_status() == 0
    a, b = (p.cpu()[torch.arange(B), at.long() % 64] for p in pools)
    assert torch.equal(a[:, :512], h[:, :512]) and torch.equal(b[:, :512], h[:, :512])
    a, b = to_np(a[:, 512:]), to_np(b[:, 512:])
    half = torch.finfo(dtype).eps / 2
    src = np.abs(to_np(h[:, 512:])).reshape(B, 32, 2).sum(-1).repeat(2, -1)
    assert np.all(np.abs(a - b) <= 8e-7 * src * (1 + half) + 2 * half * np.abs(b) * (1 + 1e-6))


def test_append_rows_captured_and_replayed():
    import mla_latent_kv_37_b200 as M
    c = Append(122, [9, 30, 1], [100, 30, 200], 32, torch.bfloat16)
    d = M.dims(3, 32)
    args = [dev(c.ckr), dev(_cu(c.tokens)), dev(torch.tensor(c.lens, dtype=torch.int32)),
            dev(c.cache.page_table), dev(c.cache.pool), dev(c.q)]
    k_rope = torch.empty(c.T, 64, dtype=torch.bfloat16, device="cuda")
    q_out = torch.empty(c.T, 32, 64, dtype=torch.bfloat16, device="cuda")

    def call():
        ckr, cu, lens, table, pool, q = args
        M.mla_append_rows(d, ckr[:, :512], ckr[:, 512:576], cu, lens, table, pool, k_rope=k_rope,
                          q_rope=q[..., 128:], q_rope_out=q_out)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([100, 30, 200], [64, 40, 129]):  # shorter and longer sequences, the same pages
        c.lens = [min(n, c.cache.page_table.shape[1] * 64) for n in lens]
        args[2].copy_(torch.tensor(c.lens, dtype=torch.int32))
        args[4].copy_(c.cache.pool)
        k_rope.zero_()
        q_out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert M.mla_get_status() == 0
        _check_append(c, args[4].cpu(), k_rope.cpu(), q_out.cpu())


@pytest.mark.parametrize("dtype", TYPES, **KW)
def test_results_repeat_themselves(dtype):
    p = Prompt(123, [700, 33, 129, 1], 16, 4, dtype)
    a, b = p.run(), p.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c = Chunk(124, [33, 1, 9, 1], [3000, 700, 900, 64], 48, dtype)
    for splits in (0, 5):
        a, b = c.run(splits), c.run(splits)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
