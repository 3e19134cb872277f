"""Cases of what stands around the experts' products of a layer, with their plain forms.

route     scores s = softmax(l) or sigmoid(l) of the router's logits; choice c = s + bias; of `groups` groups of
          experts the `top` with the best group score (the largest c, or the sum of the two largest); of those the k
          largest c; weights s (with renorm over their sum) times a factor.  plan: the slots sorted by expert, as the
          experts' product takes them.  step: the gradient of the weights with respect to the logits.
norm      r = x + residual, y = r / sqrt(mean r^2 + eps) * w, and y in E4M3 codes with a scale for each 128 columns.
          step: the gradients with respect to x (the residual's is the same) and to w.
combine   y_t = add_t + sum_j w_tj rows[positions_tj], the experts' rows back to their tokens, and its gradients.
adapters  y_m = base_m + scaling_a B_a (A_a x_m): the low-rank adapter a of row m's request beside a projection.

H = 2048, I = 768, E = 128, k = 8 and H = 4096, I = 1536 are the layer shapes this repository measures.
"""
import math

import torch

own = False   # False: the plain forms; True: this package's calls

DEV = "cuda"
BLOCK = 128
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


def listed():
    return [
        # the router of one decode batch: sigmoid scores with a balance bias, 256 experts in 8 groups
        dict(name="route_decode", op="route", T=32, E=256, k=8, dtype="f32", sigmoid=True, bias=True, renorm=True,
             groups=8, top=4, top2=True, masked=False, plan=False, step=False),
        # a padded prompt of 4096 tokens, routed and laid out for the experts' product
        dict(name="route_prompt", op="route", T=4096, E=128, k=8, dtype="f32", sigmoid=False, bias=True, renorm=True,
             groups=1, top=1, top2=False, masked=True, plan=True, step=False),
        # 100 experts in 5 groups, top-6, bf16 logits, softmax as it is; forward, plan and gradient
        dict(name="route_step_odd", op="route", T=10533, E=100, k=6, dtype="bf16", sigmoid=False, bias=False, renorm=False,
             groups=5, top=3, top2=False, masked=False, plan=True, step=True),
        # one training batch of 262144 tokens, forward and gradient
        dict(name="route_step_256k", op="route", T=262144, E=128, k=8, dtype="f32", sigmoid=True, bias=True, renorm=True,
             groups=8, top=4, top2=True, masked=False, plan=False, step=True),
        # in front of the layer, one decode batch: latency
        dict(name="norm_decode", op="norm", M=32, H=2048, dtype="bf16", residual=True, q=True, step=False),
        # the same for a prompt
        dict(name="norm_prompt", op="norm", M=8192, H=4096, dtype="bf16", residual=True, q=True, step=False),
        # one training micro-batch, forward and gradients
        dict(name="norm_step", op="norm", M=16384, H=2048, dtype="bf16", residual=True, q=False, step=True),
        # odd rows in FP32, forward and gradients
        dict(name="norm_step_odd", op="norm", M=777, H=1003, dtype="f32", residual=False, q=False, step=True),
        # behind the experts, a short prompt's rows back to its tokens
        dict(name="combine_short", op="combine", T=200, k=8, N=2048, dtype="bf16", add=True, masked=False, step=False),
        # 4096 padded tokens, forward and gradients
        dict(name="combine_step", op="combine", T=4096, k=8, N=2048, dtype="bf16", add=True, masked=True, step=True),
        # a decode batch of 32 requests with adapters of their own beside one projection
        dict(name="adapters_decode", op="adapters", M=32, K=2048, N=4096, R=16, L=64, dtype="bf16", mixed=True),
        # 8 prompts, each with its adapter
        dict(name="adapters_prompt", op="adapters", M=8192, K=4096, N=4096, R=64, L=8, dtype="bf16", mixed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "norm", "norm", "combine", "adapters", "adapters"])
    half = rng.choice(["bf16", "bf16", "f16"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        top = rng.randint(max(1, groups // 2), groups)
        E = groups * rng.randint(max(2, 16 // groups), 256 // groups)
        k = rng.randint(1, min(8, top * (E // groups)))
        T = _log(rng, 1, 33_000_000 // E)
        return dict(op="route", T=T, E=E, k=k, dtype=rng.choice(["f32", "f32", "bf16"]), sigmoid=rng.random() < 0.5,
                    bias=rng.random() < 0.6, renorm=rng.random() < 0.7, groups=groups, top=top, top2=rng.random() < 0.5,
                    masked=rng.random() < 0.4, plan=rng.random() < 0.5, step=rng.random() < 0.5)
    if op == "norm":
        H = rng.choice([128 * rng.randint(2, 64), rng.randint(100, 8192)])
        M = _log(rng, 1, 33_000_000 // H)
        step = rng.random() < 0.5
        dtype = rng.choice([half, half, "f32"])
        return dict(op="norm", M=M if dtype != "f32" else -(-M // 2), H=H, dtype=dtype, residual=rng.random() < 0.7,
                    q=not step and rng.random() < 0.7, step=step)
    if op == "combine":
        N, k = rng.choice([128 * rng.randint(2, 48), rng.randint(100, 6000)]), rng.randint(1, 8)
        T = _log(rng, 1, 60_000_000 // (N * (k + 1)))
        dtype = rng.choice([half, half, "f32"])
        return dict(op="combine", T=T if dtype != "f32" else -(-T // 2), k=k, N=N, dtype=dtype, add=rng.random() < 0.5,
                    masked=rng.random() < 0.5, step=rng.random() < 0.6)
    K, N = 8 * _log(rng, 32, 768), rng.choice([16 * _log(rng, 16, 384), _log(rng, 200, 6000)])
    R, L = 8 * rng.choice([1, 2, 2, 4, 4, 6, 8]), rng.randint(1, 64)
    M = _log(rng, 1, min(8192, 100_000_000 // (K + 2 * N)))
    return dict(op="adapters", M=M, K=K, N=N, R=R, L=L, dtype=half, mixed=rng.random() < 0.5)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)   # noqa: E731
    uni = lambda *s: torch.rand(*s, generator=g, device=DEV)    # noqa: E731
    st = dict(case)
    new = lambda *s, t=torch.float32: torch.empty(*s, dtype=t, device=DEV)   # noqa: E731
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = (1.5 * rnd(T, E) + 0.5 * rnd(E)).to(TYPES[case["dtype"]])
        st["bias"] = 0.1 * rnd(E) if case["bias"] else None
        st["valid"] = uni(T) < 0.8 if case["masked"] else None
        st["scale"] = 2.5 if case["sigmoid"] else 1.0
        st["ids"], st["weights"] = new(T, k, t=torch.int32), new(T, k)
        st["counts"], st["x_rows"], st["positions"] = (new(*s, t=torch.int32) for s in ((E,), (T * k,), (T, k)))
        st["grad"], st["dlogits"] = rnd(T, k), torch.empty_like(st["logits"])
    elif case["op"] == "norm":
        M, H, t = case["M"], case["H"], TYPES[case["dtype"]]
        # a few channels are much larger than the others, as in trained models
        gain = torch.exp(0.5 * rnd(H)) * (1 + 20 * (uni(H) < 0.01))
        st["x"] = (rnd(M, H) * gain).to(t)
        st["residual"] = (2 * rnd(M, H) * gain).to(t) if case["residual"] else None
        st["weight"] = (1 + 0.2 * rnd(H)).to(t)
        st["y"], st["sum"], st["rstd"] = new(M, H, t=t), new(M, H, t=t) if case["residual"] else None, new(M)
        st["codes"], st["scales"] = new(M, H, t=torch.uint8), new(M, -(-H // BLOCK))
        if case["step"]:
            st["dy"] = rnd(M, H).to(t)
            st["dsum"] = rnd(M, H).to(t) if case["residual"] else None
            st["dx"], st["dweight"] = new(M, H, t=t), new(H)
    elif case["op"] == "combine":
        T, k, N, t = case["T"], case["k"], case["N"], TYPES[case["dtype"]]
        on = (uni(T) < 0.8) if case["masked"] else torch.ones(T, dtype=torch.bool, device=DEV)
        # the experts' rows lie in any order; those of padded tokens behind all others, never written
        key = torch.where(on[:, None], uni(T, k), torch.full((T, k), 2.0, device=DEV)).view(-1)
        order = torch.argsort(key, stable=True)
        at = torch.empty(T * k, dtype=torch.int32, device=DEV)
        at[order] = torch.arange(T * k, dtype=torch.int32, device=DEV)
        st["positions"] = torch.where(on[:, None], at.view(T, k), torch.full_like(at.view(T, k), -1))
        st["rows"] = rnd(T * k, N).to(t)
        w = uni(T, k) + 0.05
        st["weights"] = w / w.sum(1, keepdim=True)
        st["add"] = rnd(T, N).to(t) if case["add"] else None
        st["y"] = new(T, N, t=t)
        if case["step"]:
            st["dy"], st["dweights"] = rnd(T, N).to(t), new(T, k)
            st["drows"] = torch.zeros(T * k, N, dtype=t, device=DEV)
    else:
        M, K, N, R, L = (case[n] for n in ("M", "K", "N", "R", "L"))
        t = TYPES[case["dtype"]]
        if case["mixed"]:   # one token each of requests whose adapters differ; some have none
            ids = torch.randint(0, L, (M,), generator=g, device=DEV)
            ids = torch.where(uni(M) < 0.1, torch.full_like(ids, -1), ids)
        else:               # prompts one behind the other
            ids = torch.arange(M, device=DEV) * L // M
            ids = torch.randperm(L, generator=g, device=DEV)[ids]
        st["row_adapters"] = ids.to(torch.int32)
        st["x"], st["base"] = rnd(M, K).to(t), rnd(M, N).to(t)
        st["a"], st["b"] = (rnd(L, R, K) * K ** -0.5).to(t), (rnd(L, N, R) * R ** -0.5).to(t)
        st["scaling"] = 0.25 + uni(L)
        st["y"] = new(M, N, t=t)
        # the program's plan: which rows belong to which adapter
        st["rows_of"] = [(l, (ids == l).nonzero().view(-1)) for l in sorted(set(ids.tolist()) - {-1})]
    return st


# ---------------------------------------------------------------- the plain forms
def _first(v, n):
    """Indices of the n largest of each row, the lowest index first among equals."""
    return torch.sort(v, dim=1, descending=True, stable=True).indices[:, :n]


def _scores(x, sigmoid):
    if sigmoid:
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route(st):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    x = st["logits"].double()   # 64 bits: choices next to one another
    # without a bias the scores' order is the logits'
    c = x if st["bias"] is None else _scores(x, st["sigmoid"]) + st["bias"].double()
    if G > 1:
        if st["top2"]:
            best = (c if st["bias"] is not None else _scores(x, st["sigmoid"])).view(T, G, E // G)
            best = torch.sort(best, dim=2, descending=True).values[:, :, :2].sum(2)
        else:
            best = c.view(T, G, E // G).amax(2)
        keep = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        keep.scatter_(1, _first(best, st["top"]), True)
        c = c.masked_fill(~keep[:, :, None].expand(T, G, E // G).reshape(T, E), -math.inf)
    ids = _first(c, k)
    x = st["logits"].float()
    s = _scores(x, st["sigmoid"])
    p = s.gather(1, ids)
    if st["renorm"]:
        if not st["sigmoid"]:
            p = torch.exp(x.gather(1, ids) - x.gather(1, ids).amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    out = [ids.to(torch.int32), p * st["scale"]]
    if st["plan"]:
        key = ids if st["valid"] is None else torch.where(st["valid"][:, None], ids, torch.full_like(ids, E))
        key = key.reshape(-1)
        order = torch.argsort(key, stable=True)
        counts = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        counts.scatter_add_(0, key, torch.ones_like(key, dtype=torch.int32))
        behind = torch.arange(T * k, device=DEV) >= T * k - counts[E]
        at = torch.empty_like(order)
        at[order] = torch.where(behind, -1, torch.arange(T * k, device=DEV))
        out += [counts[:E], torch.where(behind, -1, order // k).to(torch.int32), at.to(torch.int32).view(T, k)]
    if st["step"]:
        gr = st["grad"] * st["scale"]
        if st["renorm"]:
            total = s.gather(1, ids).sum(1, keepdim=True)
            gr = gr - (gr * p).sum(1, keepdim=True)
            part = p * gr if not st["sigmoid"] else p * gr * (1 - s.gather(1, ids))
            d = torch.zeros_like(x).scatter_(1, ids, part)
        elif st["sigmoid"]:
            d = torch.zeros_like(x).scatter_(1, ids, gr * p * (1 - p))
        else:
            ds = torch.zeros_like(x).scatter_(1, ids, gr)
            d = s * (ds - (gr * p).sum(1, keepdim=True))
        out.append(d.to(st["logits"].dtype))
    return tuple(out)


def _norm(st):
    H, t = st["H"], st["x"].dtype
    r = st["x"] if st["residual"] is None else (st["x"].float() + st["residual"].float()).to(t)
    f, w = r.float(), st["weight"].float()
    rstd = 1 / torch.sqrt(f.square().mean(1, keepdim=True) + EPS)
    n = f * rstd
    y = n * w
    out = [y.to(t)] + ([r] if st["residual"] is not None else [])
    if st["q"]:
        v = torch.nn.functional.pad(y, (0, -H % BLOCK)).view(st["M"], -1, BLOCK)
        s = (v.abs().amax(-1) / torch.full((), 448.0, device=DEV)).clamp_min(2.0 ** -126)
        out += [(v / s[..., None]).to(torch.float8_e4m3fn).reshape(st["M"], -1)[:, :H].contiguous(), s]
    if st["step"]:
        dy = st["dy"].float()
        gr = dy * w
        dx = rstd * (gr - n * (gr * n).mean(1, keepdim=True))
        if st["dsum"] is not None:
            dx = dx + st["dsum"].float()
        out += [rstd[:, 0], dx.to(t), (dy * n).sum(0, dtype=torch.float64).float()]
    return tuple(out)


def _combine(st):
    T, k, N, t = st["T"], st["k"], st["N"], st["rows"].dtype
    on = (st["positions"] >= 0).view(-1, 1)
    at = st["positions"].view(-1).long().clamp_min(0)
    rows = torch.where(on, st["rows"][at].float(), torch.zeros((), device=DEV)).view(T, k, N)
    y = (rows * st["weights"][:, :, None]).sum(1)
    y = y if st["add"] is None else y + st["add"].float()
    if not st["step"]:
        return y.to(t)
    dy = st["dy"].float()
    dw = (rows * dy[:, None, :]).sum(2)
    part = (st["weights"][:, :, None] * dy[:, None, :]).to(t).view(T * k, N)
    # rows of padded tokens are left as they were: their slots go to a row behind the last
    drows = torch.zeros(T * k + 1, N, dtype=t, device=DEV)
    drows[torch.where(on[:, 0], at, T * k)] = part
    return y.to(t), drows[:-1], dw


def _adapters(st):
    M, K, N, R = (st[n] for n in ("M", "K", "N", "R"))
    t = st["x"].dtype
    y = st["base"].float()
    if M * R * (K + N) <= 1 << 27:   # few rows: each one's matrices gathered
        at = st["row_adapters"].long()
        on = (at >= 0)[:, None]
        at = at.clamp_min(0)
        v = torch.matmul(st["a"][at].float(), st["x"].float()[:, :, None])
        d = torch.matmul(st["b"][at].float(), v)[:, :, 0] * st["scaling"][at][:, None]
        return torch.where(on, y + d, y).to(t)
    for l, rows in st["rows_of"]:
        v = torch.mm(st["x"][rows].float(), st["a"][l].float().t().contiguous())
        y[rows] += torch.mm(v, st["b"][l].float().t().contiguous()) * st["scaling"][l]
    return y.to(t)


# ---------------------------------------------------------------- this package's calls
def _own(st):
    import moe_gate_up_amd as mg
    if st["op"] == "route":
        mg.moe_decode_route_experts(st["logits"], st["ids"], st["weights"], bias=st["bias"], sigmoid=st["sigmoid"],
                                    renorm=st["renorm"], groups=st["groups"], top_groups=st["top"], group_top2=st["top2"],
                                    scale=st["scale"])
        out = [st["ids"], st["weights"]]
        if st["plan"]:
            mg.moe_decode_sort_slots(st["ids"], st["counts"], st["x_rows"], st["positions"], valid=st["valid"])
            out += [st["counts"], st["x_rows"], st["positions"]]
        if st["step"]:
            mg.moe_decode_route_experts_backward(st["logits"], st["ids"], st["grad"], st["dlogits"], sigmoid=st["sigmoid"],
                                                 renorm=st["renorm"], scale=st["scale"])
            out.append(st["dlogits"])
        return tuple(out)
    if st["op"] == "norm":
        q = dict(q=st["codes"], scales=st["scales"]) if st["q"] else {}
        mg.moe_decode_rms_norm(st["x"], st["weight"], EPS, y=st["y"], residual=st["residual"], sum_out=st["sum"],
                               rstd=st["rstd"] if st["step"] else None, **q)
        out = [st["y"]] + ([st["sum"]] if st["residual"] is not None else [])
        if st["q"]:
            out += [st["codes"].view(torch.float8_e4m3fn), st["scales"]]
        if st["step"]:
            r = st["x"] if st["residual"] is None else st["sum"]
            mg.moe_decode_rms_norm_backward(st["dy"], r, st["weight"], st["rstd"], st["dx"], st["dweight"], dsum=st["dsum"])
            out += [st["rstd"], st["dx"], st["dweight"]]
        return tuple(out)
    if st["op"] == "combine":
        mg.moe_decode_combine(st["rows"], st["positions"], st["weights"], st["y"], add=st["add"])
        if not st["step"]:
            return st["y"]
        mg.moe_decode_combine_backward(st["dy"], st["rows"], st["positions"], st["weights"], st["drows"], st["dweights"])
        return st["y"], st["drows"], st["dweights"]
    return mg.moe_decode_adapters(st["x"], st["row_adapters"], st["a"], st["b"], st["scaling"], st["y"], base=st["base"])


def run(state):
    if own:
        return _own(state)
    return {"route": _route, "norm": _norm, "combine": _combine, "adapters": _adapters}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    n = SIZE[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b, fl = T * E * n + 8 * T * k + (4 * E if case["bias"] else 0), 6 * T * E
        if case["plan"]:
            b += 8 * T * k + 4 * E + (T if case["masked"] else 0)
        if case["step"]:
            b += T * E * n + 4 * T * k   # the logits are read once for both passes
            fl += 4 * T * E
        return {"bytes": b, "flops": fl}
    if case["op"] == "norm":
        M, H = case["M"], case["H"]
        b = M * H * n * (4 if case["residual"] else 2) + H * n
        if case["q"]:
            b += M * H + 4 * M * -(-H // BLOCK)
        if case["step"]:
            b += M * H * n * (3 if case["residual"] else 2) + 4 * M + 4 * H
        return {"bytes": b, "flops": M * H * (5 + (10 if case["step"] else 0))}
    if case["op"] == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        live = T * k * (0.8 if case["masked"] else 1)
        b = live * N * n + T * N * n * (2 if case["add"] else 1) + 8 * T * k
        if case["step"]:
            b += live * N * n + T * N * n + 4 * T * k
        return {"bytes": int(b), "flops": int(live * N * (6 if case["step"] else 2))}
    M, K, N, R, L = (case[i] for i in ("M", "K", "N", "R", "L"))
    rows = M * (0.9 if case["mixed"] else 1)
    hit = min(L, M) if not case["mixed"] else L * (1 - (1 - 1 / L) ** rows)   # adapters that some row has
    return {"bytes": int(M * (K + 2 * N) * n + hit * R * (K + N) * n + 4 * M), "flops": int(2 * rows * R * (K + N))}


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_route(st):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    l = st["logits"].double()
    s = torch.sigmoid(l) if st["sigmoid"] else torch.softmax(l, 1)
    c = s + st["bias"].double() if st["bias"] is not None else l
    col = torch.arange(E, device=DEV)
    if G > 1:
        v = (s if st["top2"] and st["bias"] is None else c).view(T, G, E // G)
        score = v.topk(2, dim=2).values.sum(2) if st["top2"] else v.max(2).values
        out = torch.ones(T, G, dtype=torch.bool, device=DEV)
        for _ in range(st["top"]):   # argmax by hand: the first of the largest
            live = score.masked_fill(~out, -math.inf)
            first = torch.where(live == live.max(1, keepdim=True).values, torch.arange(G, device=DEV), G).min(1).values
            out[torch.arange(T, device=DEV), first] = False
        c = c.masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
    ids = []
    for _ in range(k):
        first = torch.where(c == c.max(1, keepdim=True).values, col, E).min(1, keepdim=True).values
        ids.append(first)
        c = c.scatter(1, first, -math.inf)
    ids = torch.cat(ids, 1)
    chosen = s.gather(1, ids)
    w = chosen / chosen.sum(1, keepdim=True) if st["renorm"] else chosen
    got = [ids.to(torch.int32), w * st["scale"]]
    if st["plan"]:
        on = torch.ones(T, dtype=torch.bool, device=DEV) if st["valid"] is None else st["valid"]
        flat, live = ids.view(-1), on.repeat_interleave(k)
        counts = torch.bincount(flat[live], minlength=E)
        slot = torch.arange(T * k, device=DEV)[live]
        slot = slot[torch.sort(flat[live] * (T * k) + slot).indices]   # by expert, then by slot
        rows, at = torch.full((T * k,), -1, device=DEV), torch.full((T * k,), -1, device=DEV)
        rows[:slot.numel()] = slot // k
        at[slot] = torch.arange(slot.numel(), device=DEV)
        got += [counts.to(torch.int32), rows.to(torch.int32), at.view(T, k).to(torch.int32)]
    if st["step"]:
        d = st["grad"].double() * st["scale"]
        if st["renorm"]:   # d w_j / d s_i = (delta_ij - w_j) / sum
            d = (d - (d * w).sum(1, keepdim=True)) / chosen.sum(1, keepdim=True)
        ds = torch.zeros_like(l).scatter_(1, ids, d)
        got.append(ds * s * (1 - s) if st["sigmoid"] else s * ds - s * (s * ds).sum(1, keepdim=True))
    return tuple(got)


def _exact_norm(st):
    t = st["x"].dtype
    r = st["x"].double()
    if st["residual"] is not None:
        r = (r + st["residual"].double()).to(t).double()   # the sum that is stored is what the norm is of
    w = st["weight"].double()
    rstd = (r.pow(2).sum(1) / st["H"] + EPS).rsqrt()
    y = r * rstd[:, None] * w
    got = [y] + ([r] if st["residual"] is not None else [])
    if st["q"]:
        s = torch.empty(st["M"], -(-st["H"] // BLOCK), dtype=torch.float64, device=DEV)
        q = torch.empty_like(y)
        for b in range(s.shape[1]):
            part = y[:, b * BLOCK:(b + 1) * BLOCK]
            s[:, b] = (part.abs().max(1).values / 448).clamp_min(2.0 ** -126).float()   # codes go by the stored scale
            v = (part / s[:, b:b + 1]).float().double()
            # E4M3: steps of 2^(exponent - 3), no exponent below -6; ties to even
            step = torch.exp2(torch.frexp(v).exponent.double().sub(1).clamp_min(-6) - 3)
            q[:, b * BLOCK:(b + 1) * BLOCK] = torch.round(v / step) * step
        got += [q, s]
    if st["step"]:
        dy = st["dy"].double()
        # y_c = r_c w_c rstd(r): d rstd / d r_c = - rstd^3 r_c / H
        dot = (dy * w * r).sum(1)
        dx = dy * w * rstd[:, None] - r * (rstd.pow(3) * dot / st["H"])[:, None]
        if st["dsum"] is not None:
            dx = dx + st["dsum"].double()
        got += [rstd, dx, torch.mv((dy * r).t().contiguous(), rstd)]
    return tuple(got)


def _exact_combine(st):
    T, k, N = st["T"], st["k"], st["N"]
    y = torch.zeros(T, N, dtype=torch.float64, device=DEV) if st["add"] is None else st["add"].double()
    drows = torch.zeros(T * k, N, dtype=torch.float64, device=DEV) if st["step"] else None
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    for j in range(k):
        tok = (st["positions"][:, j] >= 0).nonzero().view(-1)
        at = st["positions"][tok, j].long()
        rows, w = st["rows"][at].double(), st["weights"][tok, j].double()[:, None]
        y.index_add_(0, tok, rows * w)
        if st["step"]:
            dy = st["dy"][tok].double()
            drows[at] = dy * w
            dw[tok, j] = (dy * rows).sum(1)
    return (y, drows, dw) if st["step"] else y


def _exact_adapters(st):
    y = st["base"].double()
    for l, rows in st["rows_of"]:
        v = st["x"][rows].double() @ st["a"][l].double().t()
        y[rows] = y[rows] + st["scaling"][l].double() * (v @ st["b"][l].double().t())
    return y


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "norm": _exact_norm, "combine": _exact_combine, "adapters": _exact_adapters}[case["op"]](st)
