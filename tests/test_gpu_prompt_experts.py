"""The router, its training pass and the block-scaled 8-bit operators run together
as a prompt's MoE layer: moe_decode_route, moe_decode_balance (its counts cut
the sorted rows by expert) and its gradient, moe_decode_quantize_fp8, the gate
and up products of the experts on the rows of x they were routed, SiLU(gate) *
up quantised, the down products, and the weighted sum of each token's k rows.

Every step is checked in float64 on the step before it as the GPU left it, to
the bounds derived in the operators' own tests; the result also against the
unquantised layer in float64.  There a value v with 2^e <= |v| < 2^(e+1) has
E4M3 steps of 2^(e-3) and an error spread evenly over one, 2^(e-3) / sqrt(12) in
the root mean square: for normally distributed v sqrt(E 4^e / E v^2) = 0.73, and
0.73 / 8 / sqrt(12) = 2.64 % of v's root mean square for each quantised operand.
A product's sums are then off by sqrt(2) * 2.64 = 3.73 % (gate g and up u, unit
variance); SiLU(g) u by sqrt(3.73^2 E silu'(g)^2 / E silu(g)^2 + 3.73^2) with
E silu'^2 = 0.380 and E silu^2 = 0.357, 5.36 %; and y, with the error of that
operand and of the down matrices, by sqrt(5.36^2 + 2 * 2.64^2) = 6.54 % of its
norm.  The bound is 1.15 times that, for the spread of one token's sum over 8
experts.
"""
import pytest
import torch

import moe_gate_up_amd as mg
import oracle
from tests.test_gpu_balance import check as check_balance, reference as balance_reference
from tests.test_gpu_matmul_fp8 import F8, check as check_product, values
from tests.test_gpu_quantize_fp8 import reference as quantize_reference, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


class Layer:
    """E experts of H x I in 8 bits with a scale for each 128 x 128 block; gate's rows first, then up's."""

    def __init__(self, seed, H, I, E, dev):
        g = torch.Generator().manual_seed(seed)
        self.H, self.I, self.E = H, I, E
        self.gate_up, self.down = torch.randn(E, 2 * I, H, generator=g) * H ** -0.5, torch.randn(E, H, I, generator=g) * I ** -0.5
        self.w1, self.s1 = (t.to(dev) for t in self.quantised(self.gate_up))
        self.w2, self.s2 = (t.to(dev) for t in self.quantised(self.down))

    @staticmethod
    def quantised(w):
        E, N, K = w.shape
        p = torch.zeros(E, -(-N // 128) * 128, -(-K // 128) * 128)
        p[:, :N, :K] = w
        p = p.view(E, -(-N // 128), 128, -(-K // 128), 128)
        s = p.abs().amax((2, 4)) / 448
        q = (p / s[:, :, None, :, None]).to(F8).view(torch.uint8).reshape(E, p.shape[1] * 128, p.shape[3] * 128)
        return q[:, :N, :K].contiguous(), s.contiguous()


class Run:
    """The buffers of one prompt of T tokens and the calls that fill them."""

    def __init__(self, L, T, k, dev):
        e = lambda *s, dtype=torch.float32: torch.empty(*s, dtype=dtype, device=dev)   # noqa: E731
        i32, u8, bf16 = torch.int32, torch.uint8, torch.bfloat16
        H, I, E, M = L.H, L.I, L.E, T * k
        self.L, self.T, self.k = L, T, k
        self.x, self.logits = e(T, H, dtype=bf16), e(T, E)
        self.ids, self.weights = e(T, k, dtype=i32), e(T, k)
        self.losses, self.counts, self.tokens = e(2), e(1, E, dtype=i32), e(2, dtype=i32)
        self.grad, self.dlogits = torch.tensor([1e-2, 1e-3], device=dev), e(T, E)
        self.workspace = e(max(1, mg.moe_decode_balance_workspace(T, E, k)), dtype=u8)
        self.xq, self.xs = e(T, H, dtype=u8), e(T, -(-H // 128))
        self.h = e(M, 2 * I, dtype=bf16)
        self.hq, self.hs = e(M, I, dtype=u8), e(M, -(-I // 128))
        self.out, self.y = e(M, H, dtype=bf16), e(T, H)

    def __call__(self):
        L = self.L
        mg.moe_decode_route(self.logits, self.ids, self.weights)
        mg.moe_decode_balance(self.logits, self.ids, self.losses, self.counts, self.tokens, workspace=self.workspace)
        mg.moe_decode_balance_backward(self.logits, self.counts, self.tokens, self.grad, self.dlogits, self.k)
        order = torch.argsort(self.ids.view(-1), stable=True)
        self.rows = (order // self.k).to(torch.int32)
        mg.moe_decode_quantize_fp8(self.x, self.xq, self.xs)
        mg.moe_decode_matmul_fp8_experts(self.xq, self.xs, self.counts[0], L.w1, L.s1, self.h, x_rows=self.rows)
        mg.moe_decode_quantize_fp8(self.h, self.hq, self.hs, swiglu=True)
        mg.moe_decode_matmul_fp8_experts(self.hq, self.hs, self.counts[0], L.w2, L.s2, self.out)
        self.y.zero_()
        self.y.index_add_(0, self.rows.long(), self.out.float() * self.weights.view(-1)[order][:, None])
        self.order = order


def fill(r, seed):
    g = torch.Generator().manual_seed(seed)
    r.x.copy_(torch.randn(r.T, r.L.H, generator=g).to(torch.bfloat16))
    r.logits.copy_(torch.randn(r.T, r.L.E, generator=g) + 0.5 * torch.randn(r.L.E, generator=g))


def products(q, s, w, sw, expert):
    """Rows of codes by their experts' matrices: the sums and the sums of magnitudes, float64."""
    X, W = values(q.cpu(), s.cpu(), False), values(w.cpu(), sw.cpu(), True)
    ref, size = torch.empty(len(expert), W.shape[1], dtype=torch.float64), torch.empty(len(expert), W.shape[1], dtype=torch.float64)
    for e in range(W.shape[0]):
        at = expert == e
        if at.any():
            ref[at], size[at] = X[at] @ W[e].t(), X[at].abs() @ W[e].abs().t()
    return ref, size


SHAPES = [(1, 2048, 768, 16, 8), (37, 512, 400, 12, 4), (300, 256, 144, 40, 6), (700, 768, 256, 6, 2)]   # T, H, I, E, k


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_prompt(dev, shape):
    T, H, I, E, k = shape
    L = Layer(T, H, I, E, dev)
    r = Run(L, T, k, dev)
    fill(r, T)
    print(f"prompt {shape}", flush=True)
    r()
    torch.cuda.synchronize()
    ids, w = oracle.route(r.logits.cpu().numpy(), k)
    assert (r.ids.cpu().numpy() == ids).all()
    gb, gz = (float(v) for v in r.grad.double())
    check_balance((r.losses, r.counts, r.tokens, r.dlogits), balance_reference(r.logits, r.ids, None, 1, gb, gz), torch.float32, f"prompt {shape}")
    same((r.xq.cpu(), r.xs.cpu()), quantize_reference(r.x.cpu().float()), shape)
    expert = r.ids.view(-1)[r.order].cpu().long()
    assert torch.equal(torch.bincount(expert, minlength=E), r.counts[0].cpu().long())
    token = r.rows.cpu().long()
    ref, size = products(r.xq[token.to(dev)], r.xs[token.to(dev)], L.w1, L.s1, expert)
    check_product(r.h, ref, size, H, f"gate and up {shape}")
    h = r.h.cpu().double()
    v = torch.sigmoid(h[:, :I]) * h[:, :I] * h[:, I:]
    sv = r.hs.cpu().double().repeat_interleave(128, 1)[:, :I]
    back = r.hq.cpu().view(F8).double() * sv
    err = v.abs() * (h[:, :I].abs() + 4) * 2.0 ** -23 + 1e-37
    tol = torch.maximum(v.abs() * 2.0 ** -4, sv * 2.0 ** -10) * (1 + 2.0 ** -20) + err * (1 + 2.0 ** -4)
    assert torch.all((back - v).abs() <= tol)
    ref, size = products(r.hq, r.hs, L.w2, L.s2, expert)
    check_product(r.out, ref, size, I, f"down {shape}")
    # the layer with nothing quantised
    x = r.x.cpu().double()
    weight = torch.from_numpy(w).double().view(-1)[r.order.cpu()]
    y = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        at = expert == e
        g = x[token[at]] @ L.gate_up[e].double().t()
        a = torch.sigmoid(g[:, :I]) * g[:, :I] * g[:, I:]
        y.index_add_(0, token[at], weight[at][:, None] * (a @ L.down[e].double().t()))
    rel = float((r.y.cpu().double() - y).norm() / y.norm())
    print(f"prompt {shape}: {100 * rel:.2f} % from the unquantised layer", flush=True)
    assert rel < 1.15 * 0.0654


def test_prompt_captured(dev):
    """The run in one graph, replayed on other prompts with eager runs between the replays."""
    L = Layer(5, 256, 128, 16, dev)
    T, k = 290, 4
    eager, graphed = Run(L, T, k, dev), Run(L, T, k, dev)
    for r in (eager, graphed):
        fill(r, 1)
        r()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed()
    for seed in range(2, 6):
        for r in (eager, graphed):
            fill(r, seed)
        eager()
        graph.replay()
        torch.cuda.synchronize()
        for n in ("ids", "weights", "losses", "counts", "tokens", "dlogits", "xq", "xs", "h", "hq", "hs", "out"):
            assert torch.equal(getattr(eager, n), getattr(graphed, n)), (seed, n)
