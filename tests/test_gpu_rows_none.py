"""Slot maps of batches of no requests."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_softmax_gb300 as m
    m.build()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows", [0, 5, 70_000])
def test_map_of_no_requests(sv, rows):
    """No request: no rows, and all places behind the last one say so."""
    table, num = torch.zeros(0, 4, dtype=torch.int32, device="cuda"), i32([])
    ref = i32([0, 1, 2])
    first, request, position, slot = i32([77]), i32([77] * rows), i32([77] * rows), torch.full((rows,), 77, device="cuda")
    got = sv.map_rows(table, num, ref, num, num, rows=rows, page_size=16, out_first=first, out_request=request,
                      out_position=position, out_slot=slot)
    assert sv.read_status(got[-1]) == 0
    assert first.tolist() == [0] and got[4].numel() == 0 and ref.tolist() == [0, 1, 2]
    for x in (request, position, slot):
        assert (x == -1).all()


def test_map_of_no_requests_in_a_graph(sv):
    table, num, ref = torch.zeros(0, 4, dtype=torch.int32, device="cuda"), i32([]), i32([0, 1, 2])
    first, request, position, slot = i32([77]), i32([77] * 9), i32([77] * 9), torch.full((9,), 77, device="cuda")
    ws = sv.alloc_cache_workspace(0)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sv.map_rows(table, num, ref, num, num, rows=9, page_size=16, out_first=first, out_request=request,
                    out_position=position, out_slot=slot, out_status=num, workspace=ws)
    assert first.tolist() == [77]
    g.replay()
    assert first.tolist() == [0] and request.tolist() == position.tolist() == slot.tolist() == [-1] * 9
