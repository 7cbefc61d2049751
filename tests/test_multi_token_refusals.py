"""More of what the calls with several new tokens per sequence take and refuse, on the host before any CUDA
call (no GPU needed)."""
import pytest

from tests.test_multi_token_host import CALLS, M, _d  # noqa: F401  (M is a fixture)


@pytest.mark.parametrize("call", CALLS)
def test_d_model_is_not_used(M, call):  # noqa: F811
    for d_model in (0, -64, 7169):
        assert CALLS[call](M, _d(M, d_model=d_model), n=0) == 0
    assert M.mla_chunk_workspace_size(_d(M, d_model=0), 8) == M.mla_chunk_workspace_size(_d(M), 8) > 0
    # the calls that use it refuse it as ever
    assert M.mla_workspace_size(_d(M, d_model=0)) == 0
