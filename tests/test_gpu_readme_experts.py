"""The README's program of the router's training pass and the block-scaled experts, run as it stands there: padded
tokens, groups and ids out of range through moe_decode_balance, and its counts through
moe_decode_matmul_fp8_experts.  Every counted slot's row is its own expert's product, to the bound of
test_gpu_matmul_fp8; the other slots' rows are left alone."""
import os
import textwrap

import pytest
import torch

import moe_gate_up_amd as mg
from tests.test_gpu_matmul_fp8 import check, codes, scales, values

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def program():
    """The code block that calls the experts' product."""
    blocks, lines = [], []
    for line in open(README, encoding="utf-8"):
        if line.startswith("    ") or (lines and not line.strip()):
            lines.append(line)
        elif lines:
            blocks.append(textwrap.dedent("".join(lines)))
            lines = []
    return next(b for b in blocks if "moe_decode_matmul_fp8_experts" in b)


@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("mask", [None, "random", "padded", "empty"])
def test_readme_program(dev, G, mask):
    T, E, k, K, N = 150, 12, 4, 272, 200
    print(f"README program G={G} mask={mask}", flush=True)
    g = torch.Generator().manual_seed(G)
    logits = torch.randn(T, E, generator=g)
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    ids[5, 1], ids[77, 0] = -1, E + 3
    valid = {None: None, "random": torch.rand(T, generator=g) < 0.6, "padded": torch.arange(T) % (T // G) < 31,
             "empty": torch.zeros(T, dtype=torch.bool)}[mask]
    x = torch.randn(T, K, generator=g)
    w, sw, we, swe = codes(g, N, K), scales(g, 2, 3), codes(g, E, N, K), scales(g, E, 2, 3)
    scope = {"torch": torch, "mg": mg, "T": T, "E": E, "k": k, "G": G, "K": K, "N": N, "logits": logits.to(dev), "ids": ids.to(dev),
             "valid": None if valid is None else valid.to(dev), "grad_losses": torch.ones(2, device=dev), "x": x.to(dev),
             "w": w.to(dev), "sw": sw.to(dev), "w_experts": we.to(dev), "sw_experts": swe.to(dev)}
    exec(program(), scope)   # this repository's own text
    torch.cuda.synchronize()
    X, W = values(scope["q"].cpu(), scope["s"].cpu(), False), values(we, swe, True)
    on = torch.ones(T, dtype=torch.bool) if valid is None else valid
    got, seen = torch.full((T * k, N), float("nan"), dtype=torch.float64), scope["order"].cpu()
    got[seen] = scope["y_slots"].cpu().double()
    slots = [(t, j) for t in range(T) for j in range(k) if on[t] and 0 <= ids[t, j] < E]
    assert int(scope["counts"].sum()) == len(slots)
    left = torch.ones(T * k, dtype=torch.bool)
    if slots:
        at = torch.tensor([t * k + j for t, j in slots])
        left[at] = False
        ref = torch.stack([X[t] @ W[ids[t, j]].t() for t, j in slots])
        size = torch.stack([X[t].abs() @ W[ids[t, j]].abs().t() for t, j in slots])
        check(got[at].to(torch.bfloat16), ref, size, K, f"slots, G={G} mask={mask}")
    assert torch.all(got[left] == 0)   # as the program made them
    dense = values(w, sw, True)
    check(scope["y"], X @ dense.t(), X.abs() @ dense.abs().t(), K, "one matrix")
