"""The tensor-core attention kernel's timeout path: with the test hook on, the
first wait of the matrix instructions' warp counts as run out while copies are in
flight.  Every role then ends by itself, the call reports SPEC_ERR_TIMEOUT, and
the next call on the same workspace, hook off, is right."""
import pytest
import torch

from tests._cache_model import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [[700], [130, 900, 40, 2000, 5, 333] * 5])
def test_attention_timeout_path(sv, dtype, cache, dim, lens):
    gamma = 16
    case = Case(lens=lens, ell=[gamma - i % 3 for i in range(len(lens))], gamma=gamma, heads=8, kv_heads=2, dim=dim,
                dtype=dtype, cache=cache, page=16, seed=40)
    caches, q = case.caches(), case.q.cuda()
    out = torch.zeros_like(q)
    _, ws = case.call(sv, q=q, caches=caches, out=out)
    assert sv.read_status(ws) == 0
    sv.selftest_expire_first_wait(True)
    try:
        _, ws = case.call(sv, q=q, caches=caches, out=out, workspace=ws)
        st = sv.read_status(ws)
    finally:
        sv.selftest_expire_first_wait(False)
    assert st == sv.ERR_TIMEOUT
    lse = torch.zeros(q.shape[:-1], device="cuda")
    case.call(sv, q=q, caches=caches, out=out.zero_(), out_lse=lse, workspace=ws)
    assert sv.read_status(ws) == 0
    case.check(out, lse)
