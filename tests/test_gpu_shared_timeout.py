"""Shared-prefix attention whose waits have run out: no row keeps what an earlier
call left there or in the workspace."""
import pytest
import torch

from tests._share_model import SharedCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,share", [([20 + i % 50 for i in range(500)], [(list(range(0, 500, 3)), 1)]),
                                        ([300, 400], [([0, 1], 4)]), ([700], []), ([40, 77], [([0, 1], 2)]),
                                        ([1300, 900, 40, 1500, 5, 333] * 5, [([0, 1, 3, 6, 7, 9], 50), ([5, 11], 20)])])
def test_no_row_is_of_an_earlier_call(sv, dtype, cache, dim, lens, share):
    case = SharedCase(share=share, lens=lens, ell=[8 - i % 3 if len(lens) < 500 else i % 2 for i in range(len(lens))], gamma=8, heads=8,
                      kv_heads=8 if len(lens) == 500 else 2, dim=dim, dtype=dtype, cache=cache, seed=4)
    caches = case.caches()
    plan, _, _ = case.make_plan(sv)
    out, lse = torch.empty_like(case.q, device="cuda"), torch.empty(case.q.shape[:-1], device="cuda")
    _, ws = case.call(sv, caches=caches, plan=plan, out=out, out_lse=lse)     # its parts stay in the workspace
    assert sv.read_status(ws) == 0
    for x in (out, lse):
        x.fill_(7.0)
    sv.selftest_expire_first_wait(True)
    try:
        case.call(sv, caches=caches, plan=plan, out=out, out_lse=lse, workspace=ws)
        assert sv.read_status(ws) == sv.ERR_TIMEOUT
    finally:
        sv.selftest_expire_first_wait(False)
    for b, e in enumerate(case.ell):
        assert torch.isnan(out[b, :e + 1]).all() and torch.isnan(lse[b, :e + 1]).all()
        assert (out[b, e + 1:] == 7.0).all() and (lse[b, e + 1:] == 7.0).all()
    case.call(sv, caches=caches, plan=plan, out=out, out_lse=lse, workspace=ws)
    assert sv.read_status(ws) == 0
    case.check(out, lse)
