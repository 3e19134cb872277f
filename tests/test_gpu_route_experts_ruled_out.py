"""GPU tests of moe_decode_route_experts where a row's lowest experts in play are chosen, or decide: few of them among ruled-out
ones at any ids, biases that are all the same, logits far from 0.  Against float64, with the tolerances of
test_gpu_route_experts.py.
"""
import pytest
import torch

from tests.test_gpu_route_experts import INF, check, dev, make  # noqa: F401

pytestmark = pytest.mark.gpu


def few_in_play(seed, T, E, most, dtype, dev, equal=False):
    """Rows with 1 to `most` finite logits at random ids; `equal`: a row's are all one number."""
    g = torch.Generator().manual_seed(seed)
    l = make(seed, T, E, dtype, torch.device("cpu"))
    if equal:
        l = (2 * torch.randn(T, 1, generator=g)).to(dtype).expand(T, E).clone()
    order = torch.argsort(torch.rand(T, E, generator=g), dim=1)
    n = torch.randint(1, min(most, E) + 1, (T, 1), generator=g)
    return torch.where(order < n, l, torch.full_like(l, -INF)).to(dev)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(64, 3, 1, 1), (64, 6, 1, 1), (128, 8, 8, 4), (256, 8, 8, 3), (48, 7, 3, 2), (512, 8, 1, 1), (512, 8, 16, 5),
                                   (1000, 33, 1, 1)], ids=str)
def test_few_experts_in_play(dev, shape, dtype):  # noqa: F811
    E, k, groups, top = shape
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))).to(dev)
    for equal in (False, True):
        l = few_in_play(E + k, 300, E, k + 2, dtype, dev, equal)
        for b in (None, bias, torch.full((E,), 0.3, device=dev)):
            for sigmoid in (False, True):
                for top2 in ((False, True) if groups > 1 else (False,)):
                    print(f"few {shape} {dtype} equal={equal} bias={None if b is None else float(b[0])} sigmoid={sigmoid} top2={top2}", flush=True)
                    check(l, b, k, sigmoid, True, groups, top, top2)
                    check(l, b, k, sigmoid, False, groups, top, top2, 2.5)


@pytest.mark.parametrize("value", [0.001, 0.05, 0.3, 1.5, 4.0, 5.0, 8.0, -0.7, 1000.1])
def test_one_bias_for_all(dev, value):  # noqa: F811
    """Scores that vanish beside the bias in FP32, or in the unit of its range: they still decide."""
    for E, k, groups, top in ((64, 6, 1, 1), (128, 8, 8, 4), (512, 8, 1, 1)):
        bias = torch.full((E,), value, device=dev)
        low = make(E, 100, E, torch.float32, dev)
        peaked = low.clone()
        peaked[torch.arange(100), torch.arange(100) * 7 % E] = 28.0
        for sigmoid, l in ((True, low - 16), (True, low - 21), (False, peaked), (False, few_in_play(E, 100, E, k + 1, torch.float32, dev) - 20)):
            for top2 in ((False, True) if groups > 1 else (False,)):
                print(f"bias {value} E={E} sigmoid={sigmoid} top2={top2}", flush=True)
                check(l, bias, k, sigmoid, True, groups, top, top2)


@pytest.mark.parametrize("offset", [-3000.0, -70.0, 1000.0, 30000.0])
def test_logits_far_from_zero(dev, offset):  # noqa: F811
    """A softmax does not depend on what all logits have in common; groups by the sum of their two largest scores."""
    for E, k, groups, top in ((128, 8, 8, 4), (100, 6, 5, 3), (1024, 8, 32, 11), (64, 4, 1, 1)):
        l = make(E, 2000, E, torch.float32, dev) + offset
        for top2 in (False, True):
            print(f"offset {offset} E={E} groups={groups} top2={top2}", flush=True)
            check(l, None, k, False, True, groups, top, top2)


def test_infinite_biases(dev):  # noqa: F811
    """-inf puts an expert behind all others, as it does in 64 bits, +inf in front; a row may also be ruled out by its logits."""
    for E, k, groups, top in ((64, 6, 1, 1), (128, 8, 8, 4), (512, 8, 1, 1)):
        base = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))
        l = make(E, 60, E, torch.float32, dev)
        l[::2] = few_in_play(E, 30, E, k + 1, torch.float32, dev)
        for value in (-INF, INF):
            for on in (slice(5, 6), slice(0, E - 3), slice(0, E)):
                bias = base.clone()
                bias[on] = value
                for sigmoid in (False, True):
                    print(f"bias {value} of {on} E={E} sigmoid={sigmoid}", flush=True)
                    check(l, bias.to(dev), k, sigmoid, True, groups, top, groups > 1)
