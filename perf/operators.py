"""Cases of the router's balance loss and of the block-scaled 8-bit products, with their plain forms.

Three operators that stand beside the top-k router and the expert-centric path:

balance   per-expert counts and the two router losses of T tokens in G groups (sequences), and their
          gradient with respect to the logits.  For group g with n_g valid tokens, counts c_ge, router
          probabilities p_te = softmax(l_t)_e:
              balance = 1/G sum_g E / (k n_g) / n_g * sum_e c_ge sum_t p_te
              z       = 1/N sum_t logsumexp(l_t)^2                       N = sum_g n_g
quantize  rows to E4M3 codes with one FP32 scale for each 128 elements, scale = amax / 448 rounded to FP32
          and code = E4M3(value / scale), the quotient an FP32 number; optionally of silu(gate) * up.
matmul    y = x w^T of E4M3 codes, one scale for each row's 128 elements of x and one for each 128 x 128
          block of w; for one matrix, or for the matrices of E experts on rows sorted by expert.

H = 2048, I = 768, E = 128, k = 8 and H = 4096, I = 1536 are the layer shapes this repository measures.
"""
import math

import torch

own = False   # False: the plain forms; True: this package's calls

DEV = "cuda"
BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # the router statistics of one small decode batch: latency
        dict(name="balance_64", op="balance", G=1, S=64, E=128, k=8, dtype="f32", masked=False, step=False),
        # one training micro-batch of 4096 tokens, loss and gradient
        dict(name="balance_step_4k", op="balance", G=1, S=4096, E=128, k=8, dtype="f32", masked=False, step=True),
        # 64 padded sequences of 4096 tokens, the loss taken per sequence
        dict(name="balance_step_256k", op="balance", G=64, S=4096, E=128, k=8, dtype="f32", masked=True, step=True),
        # 100 experts, top-6, bf16 logits, ragged lengths
        dict(name="balance_step_odd", op="balance", G=3, S=3511, E=100, k=6, dtype="bf16", masked=True, step=True),
        # the activations of a decode batch
        dict(name="quantize_32", op="quantize", M=32, K=2048, dtype="bf16", swiglu=False),
        # the activations of a prompt
        dict(name="quantize_prompt", op="quantize", M=8192, K=4096, dtype="bf16", swiglu=False),
        # between the experts' two products: 4096 tokens x top-8 rows of gate and up
        dict(name="quantize_swiglu", op="quantize", M=32768, K=768, dtype="bf16", swiglu=True),
        # one token through one projection
        dict(name="matmul_token", op="matmul", M=1, N=4096, K=2048, E=0, k=0, out="bf16"),
        # a long prompt through one projection
        dict(name="matmul_prompt", op="matmul", M=8192, N=4096, K=4096, E=0, k=0, out="bf16"),
        # odd sizes, K ends inside a block of 128, FP32 result
        dict(name="matmul_odd", op="matmul", M=777, N=1003, K=1040, E=0, k=0, out="f32"),
        # gate and up of 128 experts for a decode batch of 32 tokens, top-8: two rows an expert
        dict(name="experts_decode", op="matmul", M=256, N=1536, K=2048, E=128, k=8, out="bf16"),
        # the same for a prompt of 4096 tokens, top-8
        dict(name="experts_prompt", op="matmul", M=32768, N=1536, K=2048, E=128, k=8, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["balance", "quantize", "matmul", "matmul", "experts"])
    if op == "balance":
        E = rng.choice([rng.randint(8, 256), 64, 128, 256])
        G = rng.choice([1, 1, rng.randint(2, 40)])
        S = _log(rng, 1, max(2, min(65536, 30_000_000 // (E * G))))
        return dict(op="balance", G=G, S=S, E=E, k=rng.randint(1, min(8, E)), dtype=rng.choice(["f32", "f32", "bf16"]),
                    masked=rng.random() < 0.5, step=rng.random() < 0.7)
    if op == "quantize":
        swiglu = rng.random() < 0.4
        K = 16 * _log(rng, 8, 512 if not swiglu else 256)
        return dict(op="quantize", M=_log(rng, 1, max(2, 30_000_000 // K)), K=K, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    swiglu=swiglu)
    out = rng.choice(["bf16", "bf16", "f32"])
    if op == "matmul":
        N, K = _log(rng, 100, 8192), 16 * _log(rng, 16, 512)
        M = _log(rng, 1, min(8192, 120_000_000_000 // (N * K)))
        return dict(op="matmul", M=M, N=N, K=K, E=0, k=0, out=out)
    E, k = rng.choice([16, 64, 100, 128]), rng.choice([2, 6, 8])
    N, K = _log(rng, 256, 2048), 16 * _log(rng, 32, 128)
    return dict(op="matmul", M=k * _log(rng, 1, 2048), N=N, K=K, E=E, k=k, out=out)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _codes(x):
    """E4M3 codes and FP32 scales of a weight [..., N, K] in blocks of 128 x 128."""
    *lead, n, k = x.shape
    nb, kb = -(-n // BLOCK), -(-k // BLOCK)
    p = torch.zeros(*lead, nb * BLOCK, kb * BLOCK, device=DEV)
    p[..., :n, :k] = x
    p = p.view(*lead, nb, BLOCK, kb, BLOCK)
    s = (p.abs().amax((-3, -1)) / 448).clamp_min(1e-30)
    q = (p / s[..., :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(*lead, nb * BLOCK, kb * BLOCK)[..., :n, :k].contiguous(), s.contiguous()


def prepare(case, seed):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    st = dict(case)
    if case["op"] == "balance":
        G, S, E, k = case["G"], case["S"], case["E"], case["k"]
        T = G * S
        # some experts are liked more than others, as early in training
        logits = (1.5 * rnd(T, E) + 0.5 * rnd(E)).to(TYPES[case["dtype"]])
        st["logits"] = logits
        st["ids"] = logits.float().topk(k, dim=1).indices.to(torch.int32)
        st["valid"] = None
        if case["masked"]:   # each sequence is padded behind its own length
            n = torch.randint(1, S + 1, (G,), generator=g, device=DEV)
            st["valid"] = (torch.arange(S, device=DEV)[None, :] < n[:, None]).reshape(T).contiguous()
        st["losses"] = torch.empty(2, device=DEV)
        st["counts"] = torch.empty(G, E, dtype=torch.int32, device=DEV)
        st["tokens"] = torch.empty(G + 1, dtype=torch.int32, device=DEV)   # of each group, then of all
        st["grad_losses"] = torch.tensor([1e-2, 1e-3], device=DEV) * (1 + torch.rand(2, generator=g, device=DEV))
        st["dlogits"] = torch.empty_like(logits)
    elif case["op"] == "quantize":
        M, K = case["M"], case["K"]
        cols = 2 * K if case["swiglu"] else K
        # a few channels are much larger than the others, as in trained models
        gain = torch.exp(0.5 * rnd(cols)) * (1 + 20 * (torch.rand(cols, generator=g, device=DEV) < 0.01))
        st["x"] = (rnd(M, cols) * gain).to(TYPES[case["dtype"]])
        st["q"] = torch.empty(M, K, dtype=torch.uint8, device=DEV)
        st["scales"] = torch.empty(M, -(-K // BLOCK), device=DEV)
    else:
        M, N, K, E, k = (case[n] for n in ("M", "N", "K", "E", "k"))
        rows = M // k if E else M   # experts: every token stands in k rows
        x = rnd(rows, K)
        xs = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(rows, -1, BLOCK)
        st["sx"] = (xs.abs().amax(-1) / 448).contiguous()
        st["x"] = (xs / st["sx"][..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(rows, -1)[:, :K].contiguous()
        st["w"], st["sw"] = _codes(rnd(*((E, N, K) if E else (N, K))) * K ** -0.5)
        st["y"] = torch.empty(M, N, dtype=TYPES[case["out"]], device=DEV)
        if E:
            ids = (rnd(rows, E) + 0.3 * rnd(E)).topk(k, dim=1).indices.reshape(-1)
            order = torch.argsort(ids, stable=True)
            st["x_rows"] = (order // k).to(torch.int32)
            st["counts"] = torch.bincount(ids, minlength=E).to(torch.int32)
            st["most"] = int(st["counts"].max())   # the plan: rows of the largest expert
    return st


# ---------------------------------------------------------------- the plain forms
def _balance(st):
    G, E, k = st["G"], st["E"], st["k"]
    x = st["logits"].float()
    T = x.shape[0]
    on = torch.ones(T, 1, device=DEV) if st["valid"] is None else st["valid"][:, None].float()
    counts = torch.zeros(G, E, dtype=torch.int32, device=DEV)
    counts.scatter_add_(1, st["ids"].view(G, -1).long(), on.int().expand(T, k).reshape(G, -1))
    valid = on.view(G, -1).sum(1, dtype=torch.int32)
    tokens = torch.cat([valid, valid.sum(0, keepdim=True, dtype=torch.int32)])
    m = x.amax(1, keepdim=True)
    ex = torch.exp(x - m)
    total = ex.sum(1, keepdim=True)
    p, lse = ex / total, m + torch.log(total)
    n = valid.double().clamp_min(1)
    share = (p * on).view(G, -1, E).sum(1, dtype=torch.float64)
    f = counts.double() * (E / (k * n))[:, None]
    balance = ((f * share).sum(1) / n).sum() / G
    z = (lse.square() * on).sum(dtype=torch.float64) / tokens[-1].double().clamp_min(1)
    losses = torch.stack([balance, z]).float()
    if not st["step"]:
        return losses, counts, tokens
    gb, gz = st["grad_losses"][0], st["grad_losses"][1]
    per = lambda v: v.float()[:, None].expand(G, T // G).reshape(T, 1)   # noqa: E731
    ft = f.float()[:, None, :].expand(G, T // G, E).reshape(T, E)
    dot = (p * ft).sum(1, keepdim=True)
    d = on * p * (gb * per(1 / (G * n)) * (ft - dot) + gz * (2 / tokens[-1].float().clamp_min(1)) * lse)
    return losses, counts, tokens, d.to(st["logits"].dtype)


def _quantize(st):
    x = st["x"].float()
    M, K = st["M"], st["K"]
    if st["swiglu"]:
        x = x[:, :K] / (1 + torch.exp(-x[:, :K])) * x[:, K:]
    v = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(M, -1, BLOCK)
    s = (v.abs().amax(-1) / torch.full((), 448.0, device=DEV)).clamp_min(2.0 ** -126)   # a number would be inverted and multiplied
    q = (v / s[..., None]).to(torch.float8_e4m3fn).reshape(M, -1)[:, :K].contiguous()
    return q, s


def _values(codes, scales, rows):
    """FP32 values of codes [..., n, k]; a scale for `rows` rows and 128 columns."""
    s = scales.repeat_interleave(BLOCK, -1)[..., : codes.shape[-1]]
    if rows > 1:
        s = s.repeat_interleave(rows, -2)[..., : codes.shape[-2], :]
    return codes.view(torch.float8_e4m3fn).float() * s


def _matmul(st):
    x = _values(st["x"], st["sx"], 1)
    w = _values(st["w"], st["sw"], BLOCK)
    out = TYPES[st["out"]]
    if not st["E"]:
        return torch.mm(x, w.t().contiguous()).to(out)
    counts = st["counts"].long()
    first = counts.cumsum(0) - counts
    m = torch.arange(st["M"], device=DEV)
    expert = torch.repeat_interleave(torch.arange(st["E"], device=DEV), counts, output_size=st["M"])
    at = expert * st["most"] + m - first[expert]
    padded = torch.zeros(st["E"] * st["most"], st["K"], device=DEV)
    padded[at] = x[st["x_rows"].long()]
    y = torch.bmm(padded.view(st["E"], st["most"], st["K"]), w.transpose(1, 2).contiguous())
    return y.view(-1, st["N"])[at].to(out)


# ---------------------------------------------------------------- this package's calls
def _own(st):
    import moe_gate_up_amd as mg
    if st["op"] == "balance":
        mg.moe_decode_balance(st["logits"], st["ids"], st["losses"], st["counts"], st["tokens"], valid=st["valid"])
        if not st["step"]:
            return st["losses"], st["counts"], st["tokens"]
        mg.moe_decode_balance_backward(st["logits"], st["counts"], st["tokens"], st["grad_losses"], st["dlogits"], st["k"],
                                       valid=st["valid"])
        return st["losses"], st["counts"], st["tokens"], st["dlogits"]
    if st["op"] == "quantize":
        mg.moe_decode_quantize_fp8(st["x"], st["q"], st["scales"], swiglu=st["swiglu"])
        return st["q"].view(torch.float8_e4m3fn), st["scales"]
    if st["E"]:
        return mg.moe_decode_matmul_fp8_experts(st["x"], st["sx"], st["counts"], st["w"], st["sw"], st["y"], x_rows=st["x_rows"])
    return mg.moe_decode_matmul_fp8(st["x"], st["sx"], st["w"], st["sw"], st["y"])


def run(state):
    if own:
        return _own(state)
    return {"balance": _balance, "quantize": _quantize, "matmul": _matmul}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "balance":
        T, E, k, G = case["G"] * case["S"], case["E"], case["k"], case["G"]
        tensor = T * E * size[case["dtype"]]
        mask = T if case["masked"] else 0
        b = tensor + 4 * T * k + mask + 4 * G * E + 4 * G + 8
        fl = 6 * T * E
        if case["step"]:   # the gradient needs the sums over all tokens: a second read of the logits
            b += tensor
            fl += 6 * T * E
        return {"bytes": b, "flops": fl}
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        n = 2 if case["swiglu"] else 1
        return {"bytes": n * M * K * size[case["dtype"]] + M * K + 4 * M * -(-K // BLOCK), "flops": (8 if n == 2 else 3) * M * K}
    M, N, K, E, k = (case[n] for n in ("M", "N", "K", "E", "k"))
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    if not E:
        rows, hit = M, 1
    else:
        rows, hit = M // k, min(E, E * (1 - (1 - k / E) ** (M // k)))   # experts that a routing reaches
    return {"bytes": int(rows * (K + 4 * kb) + hit * (N * K + 4 * nb * kb) + M * N * size[case["out"]] + (8 * M if E else 0)),
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "balance":
        G, S, E, k = case["G"], case["S"], case["E"], case["k"]
        losses, counts, tokens, grads = [0.0, 0.0], [], [], []
        valid = torch.ones(G * S, dtype=torch.bool, device=DEV) if st["valid"] is None else st["valid"].bool()
        N = max(1, int(valid.sum()))
        gb, gz = (float(v) for v in st["grad_losses"].double())
        for g in range(G):
            at = slice(g * S, (g + 1) * S)
            l = st["logits"][at].double()
            on = valid[at]
            n = int(on.sum())
            c = torch.bincount(st["ids"][at][on].reshape(-1).long(), minlength=E)
            p = torch.softmax(l, 1)
            z = torch.logsumexp(l, 1)
            f = c.double() * E / (k * max(1, n))
            losses[0] += float(p[on].mean(0).dot(f)) / G if n else 0.0
            losses[1] += float(z[on].square().sum()) / N
            counts.append(c.to(torch.int32))
            tokens.append(n)
            if case["step"]:
                # d p_e / d l_j = p_e (delta_ej - p_j);  d logsumexp / d l_j = p_j
                d = gb / (G * max(1, n)) * (p * f - p * (p @ f)[:, None]) + 2 * gz / N * z[:, None] * p
                grads.append(torch.where(on[:, None], d, torch.zeros_like(d)))
        got = (torch.tensor(losses, dtype=torch.float64, device=DEV), torch.stack(counts),
               torch.tensor(tokens + [sum(tokens)], dtype=torch.int32, device=DEV))
        return got + (torch.cat(grads),) if case["step"] else got
    if case["op"] == "quantize":
        M, K = case["M"], case["K"]
        x = st["x"].double()
        h = torch.sigmoid(x[:, :K]) * x[:, :K] * x[:, K:] if case["swiglu"] else x
        s = torch.empty(M, -(-K // BLOCK), dtype=torch.float64, device=DEV)
        q = torch.empty(M, K, dtype=torch.float64, device=DEV)
        for b in range(s.shape[1]):
            part = h[:, b * BLOCK:(b + 1) * BLOCK]
            s[:, b] = (part.abs().max(1).values / 448).clamp_min(2.0 ** -126).float()   # codes go by the stored scale
            r = (part / s[:, b:b + 1]).float().double()
            # E4M3: steps of 2^(exponent - 3), no exponent below -6; ties to even
            step = torch.exp2(torch.frexp(r).exponent.double().sub(1).clamp_min(-6) - 3)
            q[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(r / step) * step
        return q, s
    M, N, K, E = (case[n] for n in ("M", "N", "K", "E"))
    col = torch.arange(K, device=DEV) // BLOCK
    row = torch.arange(N, device=DEV) // BLOCK
    x = st["x"].view(torch.float8_e4m3fn).double() * st["sx"].double()[:, col]
    if not E:
        return x @ (st["w"].view(torch.float8_e4m3fn).double() * st["sw"].double()[row][:, col]).t()
    y, at = torch.empty(M, N, dtype=torch.float64, device=DEV), 0
    for e, c in enumerate(st["counts"].tolist()):
        if c:
            w = st["w"][e].view(torch.float8_e4m3fn).double() * st["sw"][e].double()[row][:, col]
            y[at:at + c] = x[st["x_rows"][at:at + c].long()] @ w.t()
            at += c
    return y
