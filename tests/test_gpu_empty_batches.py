"""GPU tests of the calls around the experts with no tokens: sums over none of them are 0."""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [1, 63, 1024])
def test_no_slots_of_any_expert(E):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    i32 = dict(dtype=torch.int32, device="cuda")
    wide = torch.full((E + 2,), 7, **i32)
    ids, rows, positions = torch.empty(0, 8, **i32), torch.empty(0, **i32), torch.empty(0, 8, **i32)
    counts = wide[1:E + 1]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mg.moe_decode_sort_slots(ids, counts, rows, positions, stream=side)
    side.synchronize()
    assert bool((counts == 0).all()) and int(wide[0]) == 7 == int(wide[E + 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg.moe_decode_sort_slots(ids, counts, rows, positions, valid=torch.empty(0, dtype=torch.bool, device="cuda"))
    for _ in range(3):
        counts.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert bool((counts == 0).all())
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_sort_slots(ids, torch.empty(1025, **i32), rows, positions)
