"""Refusals of the calls with several new tokens per sequence: all of them on the host, before any
CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def M():
    from mla_latent_kv_37_b200 import build
    build.build()
    import mla_latent_kv_37_b200 as m
    return m


F, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


def _d(M, **kw):
    d = M.dims(4, 128, 7168)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _append(M, d, **kw):
    a = dict(n=8, cu=F, lens=F, c=F, cs=512, k=F, ks=64, table=F, max_pages=4, pool=F, num_pages=10,
             k_rope=F, q=F, qt=192 * 128, qh=192, qo=F, qot=576 * 128, qoh=576)
    a.update(kw)
    return M.lib().mla_append_rows(None if d is None else ctypes.byref(d), *a.values(), None)


def _prompt(M, d, **kw):
    a = dict(n=8, kv=128, cu=F, q=F, qt=192 * 128, qh=192, k=F, kt=256 * 128, kh=256, kr=F, krs=64,
             v=F, vt=256 * 128, vh=256, scale=0.0, o=F, lse=F)
    a.update(kw)
    return M.lib().mla_prompt_attn(None if d is None else ctypes.byref(d), *a.values(), None)


def _chunk(M, d, **kw):
    a = dict(n=8, cu=F, q=F, pool=F, num_pages=10, table=F, max_pages=4, lens=F, scale=0.0, splits=0,
             ws=F, bytes=1 << 40, o=F, o_dtype=0, lse=F)
    a.update(kw)
    return M.lib().mla_chunk_attn(None if d is None else ctypes.byref(d), *a.values(), None)


CALLS = {"append": _append, "prompt": _prompt, "chunk": _chunk}


@pytest.mark.parametrize("call", CALLS)
def test_dims_and_counts(M, call):
    f = CALLS[call]
    assert f(M, None) == -1
    for bad in (dict(d_c=256), dict(n_heads=24), dict(page_size=32), dict(batch=0), dict(dtype=7)):
        assert f(M, _d(M, **bad)) == -2
    assert f(M, _d(M), n=-1) == -5
    assert f(M, _d(M), n=1 << 25) == -5  # n_tokens x heads beyond int32
    assert f(M, _d(M), n=0, **({"num_pages": 1} if call != "prompt" else {})) == 0
    if not torch.cuda.is_available():  # the batch is not limited to 128 here
        assert f(M, _d(M, batch=1000)) in (-6, -7)


@pytest.mark.parametrize("call,names", [("append", "cu lens c k table pool"),
                                        ("prompt", "cu q k kr v o"), ("chunk", "cu q pool table lens o")])
def test_required_pointers(M, call, names):
    for n in names.split():
        assert CALLS[call](M, _d(M), **{n: None}) == -1, n


@pytest.mark.parametrize("call,names", [("append", "c k pool k_rope q qo"),
                                        ("prompt", "q k kr v o"), ("chunk", "q pool o")])
def test_alignment(M, call, names):
    for n in names.split():
        assert CALLS[call](M, _d(M), **{n: ODD}) == -3, n
    two = ctypes.c_void_p(0x10002)
    for n in {"append": ("cu", "lens", "table"), "prompt": ("cu", "lse"),
              "chunk": ("cu", "lens", "table", "lse")}[call]:
        assert CALLS[call](M, _d(M), **{n: two}) == -3, n


@pytest.mark.parametrize("call,names", [("append", "cs ks qt qh qot qoh"),
                                        ("prompt", "qt qh kt kh krs vt vh")])
def test_strides(M, call, names):
    row = 64 if call == "append" else 192  # the append turns the query's rotary part alone
    good = {"cs": 512, "ks": 64, "qt": row, "qh": row, "qot": 64, "qoh": 64, "kt": 128, "kh": 128,
            "krs": 64, "vt": 128, "vh": 128}
    for n in names.split():
        for bad in (0, -512, 8, good[n] - 8, 1004, 1 << 36):
            assert CALLS[call](M, _d(M), **{n: bad}) == -5, (n, bad)
        # four fp32 are 16 bytes, four bf16 are not
        if not torch.cuda.is_available():
            assert CALLS[call](M, _d(M, dtype=1), **{n: 1004}) in (-6, -7), n


def test_append_query_goes_both_ways_or_not_at_all(M):
    assert _append(M, _d(M), q=None) == -1
    assert _append(M, _d(M), qo=None) == -1


@pytest.mark.parametrize("call", ["append", "chunk"])
def test_pages(M, call):
    for bad in (dict(max_pages=0), dict(num_pages=0), dict(max_pages=1 << 25), dict(num_pages=1 << 25)):
        assert CALLS[call](M, _d(M), **bad) == -5


def test_prompt_heads_and_scale(M):
    for bad in (0, -1, 3, 256):
        assert _prompt(M, _d(M), kv=bad) == -5
    for bad in (-1.0, float("nan"), float("inf")):
        assert _prompt(M, _d(M), scale=bad) == -5
        assert _chunk(M, _d(M), scale=bad) == -5


def test_chunk_splits_types_and_workspace(M):
    d = _d(M)
    assert _chunk(M, d, splits=-1) == -5 and _chunk(M, d, splits=65537) == -5
    assert _chunk(M, d, o_dtype=2) == -5
    assert _chunk(M, _d(M, dtype=1), o_dtype=0) == -5  # no bf16 output of the fp32 path
    assert _chunk(M, d, ws=None) == -4
    assert _chunk(M, d, ws=ctypes.c_void_p(0x10010)) == -3
    assert M.mla_chunk_workspace_size(d, 8, 65537) == 0
    assert M.mla_chunk_workspace_size(_d(M, d_c=1), 8) == 0
    assert M.mla_chunk_workspace_size(d, -1) == 0
    sizes = [M.mla_chunk_workspace_size(d, n, s) for n, s in ((1, 1), (1, 8), (5000, 9), (5000, 200))]
    assert sizes == sorted(sizes) and len(set(sizes)) == 4 and all(s % 256 == 0 for s in sizes)
    if torch.cuda.is_available():
        assert _chunk(M, d, bytes=M.mla_chunk_workspace_size(d, 8) - 1) == -4


def test_binding_refuses(M):
    d = M.dims(2, 16)
    t = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt)
    cu, lens = t(3, dt=torch.int32), t(2, dt=torch.int32)
    with pytest.raises(ValueError):  # host tensors
        M.mla_prompt_attn(d, t(4, 16, 192), t(4, 16, 128), t(4, 64), t(4, 16, 128), cu, t(4, 16, 128))
    with pytest.raises(ValueError):  # a wrong shape
        M.mla_prompt_attn(d, t(4, 16, 128), t(4, 16, 128), t(4, 64), t(4, 16, 128), cu, t(4, 16, 128))
    with pytest.raises(ValueError):
        M.mla_append_rows(d, t(4, 512), t(4, 64, dt=torch.float32), cu, lens, t(2, 1, dt=torch.int32),
                          t(1, 64, 576))
    with pytest.raises(ValueError):
        M.mla_chunk_attn(d, t(4, 16, 512), t(1, 64, 576), t(2, 1, dt=torch.int32), cu, lens,
                         t(4, 16, 512), t(1, dt=torch.uint8))
