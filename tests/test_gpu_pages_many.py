"""Needs of pages whose sum passes what the prefix over the requests holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


def test_reserve_more_than_any_pool_holds(sv):
    """4095 requests of 262400 pages need more than 2^30: each one that does not
    fit says so, those behind the sum's end too, and nothing of theirs changes."""
    B, slots, pages = 4096, 262400, 1000
    assert (B - 3) * slots > 2 ** 30
    table = torch.full((B, slots), -1, dtype=torch.int32, device="cuda")
    num, ref = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, pages))
    lens = torch.full((B,), slots - 1, dtype=torch.int32, device="cuda")
    lens[0] = 3
    lens[B - 1] = 0
    num[B - 2], lens[B - 2] = 5, 4      # has its pages
    status, ws = sv.reserve_pages(table, num, ref, lens, gamma=0, page_size=1)
    want = torch.full((B,), sv.ERR_POOL, dtype=torch.int32)
    want[0] = want[B - 2] = sv.OK
    assert torch.equal(status.cpu(), want)
    assert sv.read_status(ws) == sv.ERR_POOL
    assert num.cpu()[[0, B - 2]].tolist() == [4, 5] and int(num.sum()) == 9
    assert table[0, :5].tolist() == [0, 1, 2, 3, -1] and int((table != -1).sum()) == 4
    assert ref[:4].tolist() == [1] * 4 and int(ref.sum()) == 4
