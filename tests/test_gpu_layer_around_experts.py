"""A mixture-of-experts block as a user runs it, through the public calls alone: norm with the residual -> router's
logits -> routing by scores -> sorted slots -> experts' products of 8-bit rows -> combine onto the residual stream, and
the gradients of routing, combine and norm back again; a prompt and a decode batch of one token, eager and from a
captured graph.  An adapter stands beside one more projection.

Each stage is compared with the same step in float64 of what the stage before it left (the values its codes stand for),
so that no stage's rounding is in another's tolerance: half a step of the stage's type (bf16 2^-8, E4M3 2^-4 of the value
or 2^-10 scales), and for a sum of n FP32 products n 2^-24 of the sum of their magnitudes.
"""
import pytest
import torch

import moe_gate_up_amd as mg

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def blocks(w):
    """E4M3 codes and scales of w [E, N, K] in blocks of 128 x 128, and the values they stand for."""
    E, N, K = w.shape
    v = w.view(E, N // 128, 128, K // 128, 128)
    s = v.abs().amax((2, 4)) / 448
    q = (v / s[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(E, N, K).contiguous(), s.contiguous(), (q.double() * s[:, :, None, :, None].double()).reshape(E, N, K)


class Block:
    def __init__(self, dev, H=256, I=128, E=16, k=4):
        g = torch.Generator(device=dev).manual_seed(1)
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)   # noqa: E731
        self.H, self.I, self.E, self.k, self.dev = H, I, E, k, dev
        self.norm = (1 + 0.1 * rnd(H)).to(BF)
        self.router = (rnd(H, E) * H ** -0.5).float()
        self.bias = 0.05 * rnd(E)
        self.w1, self.s1, self.v1 = blocks(rnd(E, 2 * I, H) * H ** -0.5)
        self.w2, self.s2, self.v2 = blocks(rnd(E, H, I) * I ** -0.5)

    def buffers(self, T):
        H, I, E, k = self.H, self.I, self.E, self.k
        e = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=self.dev)   # noqa: E731
        i32, u8 = torch.int32, torch.uint8
        return dict(y=e(T, H, t=BF), q=e(T, H, t=u8), sq=e(T, H // 128), sum=e(T, H, t=BF), rstd=e(T), logits=e(T, E), ids=e(T, k, t=i32),
                    w=e(T, k), counts=e(E, t=i32), rows=e(T * k, t=i32), at=e(T, k, t=i32), h=torch.zeros(T * k, 2 * I, dtype=BF, device=self.dev),
                    hq=e(T * k, I, t=u8), hs=e(T * k, I // 128), o=torch.zeros(T * k, H, dtype=BF, device=self.dev), out=e(T, H, t=BF))

    def forward(self, b, x, residual, valid):
        mg.moe_decode_rms_norm(x, self.norm, 1e-6, y=b["y"], q=b["q"], scales=b["sq"], residual=residual, sum_out=b["sum"], rstd=b["rstd"])
        torch.mm(b["y"].float(), self.router, out=b["logits"])
        mg.moe_decode_route_experts(b["logits"], b["ids"], b["w"], bias=self.bias, sigmoid=True, groups=4, top_groups=2, group_top2=True, scale=2.0)
        mg.moe_decode_sort_slots(b["ids"], b["counts"], b["rows"], b["at"], valid=valid)
        mg.moe_decode_matmul_fp8_experts(b["q"], b["sq"], b["counts"], self.w1, self.s1, b["h"], x_rows=b["rows"])
        mg.moe_decode_quantize_fp8(b["h"], b["hq"], b["hs"], swiglu=True)
        mg.moe_decode_matmul_fp8_experts(b["hq"], b["hs"], b["counts"], self.w2, self.s2, b["o"])
        mg.moe_decode_combine(b["o"], b["at"], b["w"], b["out"], add=b["sum"])
        return b["out"]

    def check(self, b, x, residual, valid):
        T, H, I, E, k = x.shape[0], self.H, self.I, self.E, self.k
        u, half = 2.0 ** -24, 2.0 ** -8

        def near(got, ref, size, n, step=half):
            """A sum of n products, the sum of whose magnitudes is `size`, rounded once."""
            err = n * u * size
            bad = (got.double() - ref).abs() - err - step * (ref.abs() + err) - 1e-30
            assert float(bad.max()) <= 0 if bad.numel() else True

        def stands_for(q, s):
            return q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)

        def quantised(q, s, v, rel):
            wide = s.double().repeat_interleave(128, 1)
            assert bool(((stands_for(q, s) - v).abs() <= 2.0 ** -4 * v.abs() * (1 + rel) + 2.0 ** -10 * wide + rel * v.abs()).all())

        r = (x.float() + residual.float()).to(BF)
        assert torch.equal(b["sum"], r)
        r = r.double()
        v = r / torch.sqrt(r.square().mean(1, keepdim=True) + 1e-6) * self.norm.double()
        near(b["y"], v, v.abs(), 52)      # the norm's own bound, 52 roundings
        quantised(b["q"], b["sq"], v, 60 * u)
        # the rows of each expert's product, in the order of its slots
        slot = 0
        on = torch.ones(T, dtype=torch.bool) if valid is None else valid.cpu()
        ids, counts, rows, at = (b[n].cpu() for n in ("ids", "counts", "rows", "at"))
        xv = stands_for(b["q"], b["sq"])
        for e in range(E):
            mine = [(t, j) for t in range(T) for j in range(k) if bool(on[t]) and int(ids[t, j]) == e]
            assert int(counts[e]) == len(mine)
            for t, j in mine:
                assert int(rows[slot]) == t and int(at[t, j]) == slot
                slot += 1
            if mine:
                sl = slice(slot - len(mine), slot)
                near(b["h"][sl], xv[[t for t, _ in mine]] @ self.v1[e].t(), xv[[t for t, _ in mine]].abs() @ self.v1[e].abs().t(), 2 * H)
                hv = stands_for(b["hq"][sl], b["hs"][sl])
                near(b["o"][sl], hv @ self.v2[e].t(), hv.abs() @ self.v2[e].abs().t(), 2 * I)
        h = b["h"][:slot].double()
        quantised(b["hq"][:slot], b["hs"][:slot], h[:, :I] * torch.sigmoid(h[:, :I]) * h[:, I:], 16 * u)
        # silu's own bound: (3.5 + |g| / 43) 2^-23 and the product, 16 u for |g| < 40
        out, size = r.clone(), r.abs()
        for t in range(T):
            for j in range(k):
                if bool(on[t]):
                    d = float(b["w"][t, j]) * b["o"][int(at[t, j])].double()
                    out[t] += d
                    size[t] += d.abs()
        near(b["out"], out, size, k + 1)


@pytest.mark.parametrize("T", [1, 50])
def test_a_block_forward(dev, T):
    m = Block(dev)
    g = torch.Generator(device=dev).manual_seed(T)
    x, residual = (torch.randn(T, m.H, generator=g, device=dev).to(BF) for _ in range(2))
    valid = None if T == 1 else torch.rand(T, generator=g, device=dev) < 0.8
    b = m.buffers(T)
    m.forward(b, x, residual, valid)
    torch.cuda.synchronize()
    m.check(b, x, residual, valid)
    if valid is not None:
        assert torch.equal(b["out"][~valid], b["sum"][~valid])   # a padded token keeps its residual


def test_a_block_from_a_graph(dev):
    m = Block(dev)
    T = 40
    g = torch.Generator(device=dev).manual_seed(3)
    x, residual = (torch.randn(T, m.H, generator=g, device=dev).to(BF) for _ in range(2))
    valid = torch.rand(T, generator=g, device=dev) < 0.8
    b, e = m.buffers(T), m.buffers(T)
    m.forward(b, x, residual, valid)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(b, x, residual, valid)
    for seed in (4, 5, 6):
        g.manual_seed(seed)
        x.copy_(torch.randn(T, m.H, generator=g, device=dev))
        valid.copy_(torch.rand(T, generator=g, device=dev) < 0.6)
        want = m.forward(e, x, residual, valid).clone()
        graph.replay()
        torch.cuda.synchronize()
        for name in ("out", "ids", "w", "at", "counts", "logits"):
            assert torch.equal(b[name], e[name]), name
        assert torch.equal(b["out"], want)


def test_the_gradients_of_a_block(dev):
    """Combine, routing and norm backwards, chained as in training, against autograd of the same steps in float64 (the
    experts' products taken as a matrix for each expert, in float64 too)."""
    m = Block(dev)
    T, H, E, k = 30, m.H, m.E, m.k
    g = torch.Generator(device=dev).manual_seed(9)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)   # noqa: E731
    x, mix = rnd(T, H), rnd(E, H, H) * H ** -0.5
    weight = 1 + 0.1 * rnd(H)
    b = m.buffers(T)
    f = dict(y=torch.empty(T, H, device=dev), rstd=b["rstd"])
    mg.moe_decode_rms_norm(x, weight, 1e-6, y=f["y"], rstd=f["rstd"])
    logits = f["y"] @ m.router
    mg.moe_decode_route_experts(logits, b["ids"], b["w"], bias=m.bias, sigmoid=True, groups=4, top_groups=2, group_top2=True, scale=2.0)
    mg.moe_decode_sort_slots(b["ids"], b["counts"], b["rows"], b["at"])
    rows = f["y"][b["rows"].long()]
    expert = torch.repeat_interleave(torch.arange(E, device=dev), b["counts"].long())
    o = torch.bmm(mix[expert], rows[:, :, None])[:, :, 0].contiguous()
    out = torch.empty(T, H, device=dev)
    mg.moe_decode_combine(o, b["at"], b["w"], out, add=x)
    dout = rnd(T, H)
    do, dw = torch.empty_like(o), torch.empty(T, k, device=dev)
    mg.moe_decode_combine_backward(dout, o, b["at"], b["w"], do, dw)
    drows = torch.bmm(mix[expert].transpose(1, 2).contiguous(), do[:, :, None])[:, :, 0].contiguous()
    dlogits = torch.empty_like(logits)
    mg.moe_decode_route_experts_backward(logits, b["ids"], dw, dlogits, sigmoid=True, scale=2.0)
    dy = dlogits @ m.router.t().contiguous()
    mg.moe_decode_combine(drows, b["at"], None, dy, add=dy)    # a token's slots' gradients onto the router's
    dx, dweight = dout.clone(), torch.empty(H, device=dev)
    mg.moe_decode_rms_norm_backward(dy, x, weight, f["rstd"], dx, dweight, dsum=dx)

    X, W = x.cpu().double().requires_grad_(), weight.cpu().double().requires_grad_()
    ids, M, R = b["ids"].cpu().long(), mix.cpu().double(), m.router.cpu().double()
    Y = X / torch.sqrt(X.square().mean(1, keepdim=True) + 1e-6) * W
    S = torch.sigmoid(Y @ R).gather(1, ids)
    P = 2.0 * S / S.sum(1, keepdim=True)
    out64 = X + sum(P[:, j, None] * torch.einsum("tij,tj->ti", M[ids[:, j]], Y) for j in range(k))
    out64.backward(dout.cpu().double())
    for got, want in ((out, out64.detach()), (dx, X.grad), (dweight, W.grad)):
        # FP32 sums of a few hundred terms, through four stages: 1e-5 of the largest
        assert float((got.cpu().double() - want).abs().max()) <= 1e-5 * float(want.abs().max())


def test_adapters_beside_a_projection(dev):
    """A decode batch through a shared 8-bit projection with each request's adapter added in place."""
    T, K, N, R, L = 9, 256, 384, 16, 5
    g = torch.Generator(device=dev).manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)   # noqa: E731
    x, residual = rnd(T, K).to(BF), rnd(T, K).to(BF)
    wq, ws, wv = blocks(rnd(1, N, K) * K ** -0.5)
    a, b, s = (rnd(L, R, K) * K ** -0.5).to(BF), rnd(L, N, R).to(BF), torch.rand(L, generator=g, device=dev)
    ids = torch.tensor([0, 1, 2, 3, 4, -1, 0, 1, 7], dtype=torch.int32, device=dev)
    y, q, sq = torch.empty_like(x), torch.empty(T, K, dtype=torch.uint8, device=dev), torch.empty(T, K // 128, device=dev)
    mg.moe_decode_rms_norm(x, torch.ones(K, dtype=BF, device=dev), 1e-6, y=y, q=q, scales=sq, residual=residual)
    out = torch.empty(T, N, dtype=BF, device=dev)
    mg.moe_decode_matmul_fp8(q, sq, wq[0], ws[0], out)
    shared = out.clone()
    mg.moe_decode_adapters(y, ids, a, b, s, out, base=out)
    for t in range(T):
        l = int(ids[t])
        if not 0 <= l < L:
            assert torch.equal(out[t], shared[t])
            continue
        v = a[l].double() @ y[t].double()
        d = float(s[l]) * (b[l].double() @ v)
        # v a sum of K products and as two bf16 numbers 2^-8 2^-8 of itself, then R products
        ev = K * 2.0 ** -24 * (a[l].double().abs() @ y[t].double().abs()) + (2.0 ** -16 + (2 * R + 8) * 2.0 ** -24) * v.abs()
        err = float(s[l]) * (b[l].double().abs() @ ev) + 2.0 ** -23 * (shared[t].double().abs() + d.abs())
        ref = shared[t].double() + d
        assert bool(((out[t].double() - ref).abs() <= err + 2.0 ** -8 * (ref.abs() + err)).all())
