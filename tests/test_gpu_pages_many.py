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


def test_a_place_whose_request_has_ended(sv):
    """At verify length 0 and accept length -1 it takes a page for each round and
    gives it back, with no error, while its neighbours go on."""
    B, slots, pages, page = 3, 4, 12, 4
    table = torch.full((B, slots), -1, dtype=torch.int32, device="cuda")
    num, ref, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, pages, B))
    ws = sv.alloc_cache_workspace(B)

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def step(ell, accept):
        st, _ = sv.reserve_pages(table, num, ref, lens, i32(*ell), gamma=2, page_size=page, workspace=ws)
        assert st.tolist() == [0] * B
        held = num.tolist()
        sv.commit_pages(table, num, ref, lens, i32(*accept), page_size=page, workspace=ws)
        assert sv.read_status(ws) == 0
        return held

    step((2, 2, 2), (2, 2, 1))
    sv.free_pages(table, num, ref, lens, i32(1), workspace=ws)
    for k in range(1, 3):
        assert step((2, 0, 2), (2, -1, 1))[1] == 1
        assert lens.tolist() == [3 + 3 * k, 0, 2 + 2 * k] and num[1] == 0 and (table[1] == -1).all()
        assert int(ref.sum()) == int(num.sum())
