"""Workspace sizes never go down where a batch grows: one sized for the largest batch does for all smaller ones (CPU only)."""
import pytest

import moe_gate_up_amd as mg


def sizes(top):
    return sorted({*range(0, 300), *range(300, 20000, 61), *(n + d for n in (384, 1024, 4480, 8192, 8193, 1 << 16) for d in (-1, 0, 1)),
                   *(1 << i for i in range(8, 26)), top - 1} & set(range(top)))


@pytest.mark.parametrize("K,R,L", [(8192, 64, 1), (8192, 64, 8), (4096, 8, 1023), (8, 8, 1), (1 << 20, 256, 1), (1 << 20, 8, 100), (2056, 128, 300)])
def test_adapters(K, R, L):
    last, at = 0, 0
    for M in sizes(1 << 22):
        n = mg.moe_decode_adapters_workspace.__wrapped__(M, K, 4096, R, L)
        assert n >= last, (at, last, M, n)
        last, at = n, M


@pytest.mark.parametrize("E,k", [(1, 1), (128, 8), (1024, 64)])
def test_sorted_slots(E, k):
    last = 0
    for T in sizes(((1 << 24) - 1) // k):
        n = mg.moe_decode_sort_slots_workspace.__wrapped__(T, E, k)
        assert n >= last, T
        last = n


@pytest.mark.parametrize("H", [1, 2048, 32768])
def test_norm_gradient(H):
    last = 0
    for M in sizes(1 << 22):
        n = mg.moe_decode_rms_norm_backward_workspace.__wrapped__(M, H)
        assert n >= last, M
        last = n


@pytest.mark.gpu
def test_one_workspace_for_all_batches():
    """Adapters of 8192 columns, rank 64: the largest batch's workspace, used again for smaller ones, the results those of a workspace of
    each batch's own."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    K, N, R, L = 8192, 64, 64, 1
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)   # noqa: E731
    a, b, scaling = rnd(L, R, K) / 90, rnd(L, N, R), torch.ones(L, device="cuda")
    ws = torch.full((mg.moe_decode_adapters_workspace(4480, K, N, R, L),), 0xAB, dtype=torch.uint8, device="cuda")
    for M in (4480, 4479, 3000, 64, 63, 1):
        x, ids = rnd(M, K), torch.zeros(M, dtype=torch.int32, device="cuda")
        y, own = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        mg.moe_decode_adapters(x, ids, a, b, scaling, y, workspace=ws)
        mg.moe_decode_adapters(x, ids, a, b, scaling, own)
        torch.cuda.synchronize()
        assert torch.equal(y, own), M
