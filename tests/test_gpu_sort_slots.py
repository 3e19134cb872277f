"""GPU tests of moe_decode_sort_slots: whole numbers, compared exactly with a stable
sort on the CPU."""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def reference(ids, valid, E):
    T, k = ids.shape
    key = ids.cpu().long().flatten()
    on = (key >= 0) & (key < E)
    if valid is not None:
        on &= valid.cpu().bool().repeat_interleave(k)
    key = torch.where(on, key, torch.full_like(key, E))
    order = torch.argsort(key, stable=True)
    n = int(on.sum())
    rows = torch.where(torch.arange(T * k) < n, order // k, torch.full_like(order, -1))
    at = torch.empty_like(order)
    at[order] = torch.arange(T * k)
    return torch.bincount(key, minlength=E + 1)[:E], rows, torch.where(on, at, torch.full_like(at, -1)).view(T, k)


def run(ids, valid, E, **kw):
    T, k = ids.shape
    out = [torch.full(s, 99, dtype=torch.int32, device=ids.device) for s in ((E,), (T * k,), (T, k))]
    mg.moe_decode_sort_slots(ids, *out, valid=valid, **kw)
    torch.cuda.synchronize()
    return out


def check(ids, valid, E):
    for got, ref, name in zip(run(ids, valid, E), reference(ids, valid, E), ("counts", "x_rows", "positions")):
        assert torch.equal(got.cpu().long(), ref), name


@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 8, 128), (3, 5, 7), (32, 8, 128), (63, 1, 1024), (64, 1, 2), (65, 3, 1000), (512, 8, 64),
                                   (513, 8, 64), (4096, 1, 3), (4097, 1, 1), (1000, 8, 128), (4096, 8, 128), (4095, 8, 1024), (1024, 8, 128), (8193, 1, 77), (4097, 8, 128), (32768, 1, 1000), (32769, 1, 1024), (262144, 1, 100), (262145, 1, 100), (10533, 6, 100), (20000, 64, 1024),
                                   (70001, 7, 1023), (300000, 8, 256), (16777215, 1, 16)], ids=str)
def test_sorted(dev, shape):
    T, k, E = shape
    print(f"sort {shape}", flush=True)
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32)
    check(ids.to(dev), None, E)
    if T > 400000:
        return
    ids = torch.randint(-3, E + 3, (T, k), generator=g, dtype=torch.int32).to(dev)
    check(ids, None, E)
    valid = torch.rand(T, generator=g) < 0.6
    check(ids, valid.to(dev), E)
    check(ids, (valid.to(torch.uint8) * 3).to(dev), E)


@pytest.mark.parametrize("T", [100, 5000])
def test_one_expert_none_and_all(dev, T):
    for E, ids in ((5, torch.full((T, 3), 4)), (1, torch.zeros(T, 3)), (8, torch.full((T, 3), -1)), (8, torch.full((T, 3), 2 ** 31 - 1)),
                   (1024, torch.arange(3 * T).view(T, 3) % 1024), (4, torch.full((T, 3), -2 ** 31))):
        ids = ids.to(torch.int32).to(dev)
        check(ids, None, E)
        check(ids, torch.zeros(T, dtype=torch.bool, device=dev), E)


def test_graph_stream_workspace(dev):
    T, k, E = 5000, 8, 128
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).to(dev)
    need = mg.moe_decode_sort_slots_workspace(T, E, k)
    assert need > 0 == mg.moe_decode_sort_slots_workspace(1024, E, k)
    ws = torch.full((need,), 0xAB, dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = [torch.empty(s, dtype=torch.int32, device=dev) for s in ((E,), (T * k,), (T, k))]
    mg.moe_decode_sort_slots(ids, *out, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a.cpu().long(), b) for a, b in zip(out, reference(ids, None, E)))
    with pytest.raises(ValueError):
        mg.moe_decode_sort_slots(ids, *out, stream=side)
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_sort_slots(ids, *out, workspace=ws[:256])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mg.moe_decode_sort_slots(ids, *out, workspace=ws)
    for _ in range(3):
        ids.copy_(torch.randint(0, E, (T, k), generator=g, dtype=torch.int32))
        ref = run(ids, None, E)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_refusals(dev):
    i32 = dict(dtype=torch.int32, device=dev)
    ids, counts, rows, pos = torch.zeros(4, 2, **i32), torch.empty(8, **i32), torch.empty(8, **i32), torch.empty(4, 2, **i32)
    for args in ((ids.long(), counts, rows, pos), (ids, counts.float(), rows, pos), (ids, counts, rows[:7], pos), (ids, counts, rows, pos.view(2, 4))):
        with pytest.raises(ValueError):
            mg.moe_decode_sort_slots(*args)
    with pytest.raises(ValueError):
        mg.moe_decode_sort_slots(ids, counts, rows, pos, valid=torch.ones(3, dtype=torch.bool, device=dev))
    with pytest.raises(mg.MoeDecodeError):   # onto its input
        mg.moe_decode_sort_slots(ids, counts, rows, ids)
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_sort_slots(ids, torch.empty(1025, **i32), rows, pos)
    mg.moe_decode_sort_slots(ids[:0], counts, rows[:0], pos[:0])
