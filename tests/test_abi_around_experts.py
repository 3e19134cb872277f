"""Host-side checks of the calls around the experts (routing by scores, sorted slots,
combine, norm, adapters) of the C ABI, CPU only: every case returns during argument
validation, before any HIP call; the pointers are addresses that are never dereferenced."""
import ctypes

import pytest

import moe_gate_up_amd as mg

A = 0x100000000000   # aligned stand-ins for device buffers, 64 GiB apart
S = 0x1000000000
MOST = 2 ** 31 - 1


def at(i, plus=0):
    return A + i * S + plus


def P(v):
    return ctypes.c_void_p(v or None)


def size_of(fn, *args):
    n = ctypes.c_size_t()
    fn(*args, ctypes.byref(n))   # leaves 0 where it refuses
    return n.value


def route(logits=at(0), ld=128, dtype=mg.MOE_F32, bias=at(1), ids=at(2), w=at(3), T=64, E=128, k=8, groups=1, top=1, flags=0):
    return mg.lib().moe_decode_route_experts(P(logits), ld, dtype, P(bias), P(ids), P(w), T, E, k, groups, top, flags, 1.0, None)


def route_backward(logits=at(0), ld=128, dtype=mg.MOE_F32, ids=at(1), grad=at(2), d=at(3), ld_d=128, T=64, E=128, k=8, flags=0):
    return mg.lib().moe_decode_route_experts_backward(P(logits), ld, dtype, P(ids), P(grad), P(d), ld_d, T, E, k, flags, 1.0, None)


def sort(ids=at(0), valid=0, counts=at(1), rows=at(2), pos=at(3), ws=at(4), ws_bytes=None, T=8192, E=128, k=8):
    if ws_bytes is None:
        ws_bytes = size_of(mg.lib().moe_decode_sort_slots_workspace, T, E, k)
    return mg.lib().moe_decode_sort_slots(P(ids), P(valid), P(counts), P(rows), P(pos), P(ws), ws_bytes, T, E, k, None)


def combine(rows=at(0), ld_rows=2048, dtype=mg.MOE_BF16, pos=at(1), w=at(2), add=at(3), ld_add=2048, y=at(4), ld_y=2048,
            M=512, T=64, N=2048, k=8):
    return mg.lib().moe_decode_combine(P(rows), ld_rows, dtype, P(pos), P(w), P(add), ld_add, P(y), ld_y, M, T, N, k, None)


def combine_backward(dy=at(0), ld_dy=2048, rows=at(1), ld_rows=2048, dtype=mg.MOE_BF16, pos=at(2), w=at(3), drows=at(4), ld_d=2048,
                     dw=at(5), M=512, T=64, N=2048, k=8):
    return mg.lib().moe_decode_combine_backward(P(dy), ld_dy, P(rows), ld_rows, dtype, P(pos), P(w), P(drows), ld_d, P(dw), M, T, N, k, None)


def norm(x=at(0), ld_x=2048, res=at(1), ld_res=2048, dtype=mg.MOE_BF16, weight=at(2), wt=mg.MOE_BF16, eps=1e-6, y=at(3), ld_y=2048,
         q=at(4), scales=at(5), total=at(6), ld_sum=2048, rstd=at(7), M=32, H=2048, flags=0):
    return mg.lib().moe_decode_rms_norm(P(x), ld_x, P(res), ld_res, dtype, P(weight), wt, eps, P(y), ld_y, P(q), P(scales), P(total), ld_sum,
                                        P(rstd), M, H, flags, None)


def norm_backward(dy=at(0), ld_dy=2048, r=at(1), ld_r=2048, dtype=mg.MOE_BF16, weight=at(2), wt=mg.MOE_BF16, rstd=at(3), dsum=at(4),
                  ld_dsum=2048, dx=at(5), ld_dx=2048, dweight=at(6), ws=at(7), ws_bytes=None, M=32, H=2048):
    if ws_bytes is None:
        ws_bytes = size_of(mg.lib().moe_decode_rms_norm_backward_workspace, M, H)
    return mg.lib().moe_decode_rms_norm_backward(P(dy), ld_dy, P(r), ld_r, dtype, P(weight), wt, P(rstd), P(dsum), ld_dsum, P(dx), ld_dx,
                                                 P(dweight), P(ws), ws_bytes, M, H, None)


def adapters(x=at(0), ld_x=2048, dtype=mg.MOE_BF16, ids=at(1), a=at(2), b=at(3), s=at(4), base=at(5), ld_base=4096, y=at(6), ld_y=4096,
             ws=at(7), ws_bytes=None, M=2000, K=2048, N=4096, R=16, L=64):
    if ws_bytes is None:
        ws_bytes = size_of(mg.lib().moe_decode_adapters_workspace, M, K, N, R, L)
    return mg.lib().moe_decode_adapters(P(x), ld_x, dtype, P(ids), P(a), P(b), P(s), P(base), ld_base, P(y), ld_y, P(ws), ws_bytes, M, K, N,
                                        R, L, None)


SHAPES = {
    route: [dict(T=-1), dict(T=1 << 26), dict(E=0), dict(E=1025, ld=1025), dict(k=0), dict(k=65), dict(k=9, E=8, ld=8), dict(ld=127),
            dict(ld=(1 << 30) + 1), dict(groups=0), dict(groups=3), dict(groups=128), dict(groups=65), dict(groups=-1), dict(top=0), dict(top=2),
            dict(groups=32, top=1), dict(T=(1 << 26) - 1, k=64)],
    route_backward: [dict(T=-1), dict(T=1 << 26), dict(E=0), dict(E=1025, ld=1025, ld_d=1025), dict(k=0), dict(k=65), dict(ld=127), dict(ld_d=100)],
    sort: [dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(T=1 << 21), dict(T=MOST)],
    combine: [dict(M=-1), dict(T=-1), dict(N=0), dict(k=0), dict(k=65), dict(T=1 << 21), dict(M=(1 << 24) + 1), dict(ld_rows=2047), dict(ld_add=1),
              dict(ld_y=2047), dict(ld_y=(1 << 30) + 1), dict(N=MOST, ld_rows=MOST), dict(T=1 << 20, k=1, N=1 << 17, ld_rows=1 << 17, ld_y=1 << 17)],
    combine_backward: [dict(M=-1), dict(T=-1), dict(N=0), dict(k=0), dict(k=65), dict(T=1 << 21), dict(ld_rows=2047), dict(ld_dy=1), dict(ld_d=2047)],
    norm: [dict(M=-1), dict(H=0), dict(H=32769), dict(M=1 << 26), dict(M=1 << 24, H=4097), dict(M=1 << 22, H=16385), dict(ld_x=2047), dict(ld_res=0),
           dict(ld_y=2047), dict(ld_sum=2047), dict(ld_x=(1 << 30) + 1)],
    norm_backward: [dict(M=-1), dict(H=0), dict(H=32769), dict(M=1 << 26), dict(ld_dy=2047), dict(ld_r=0), dict(ld_dsum=2047), dict(ld_dx=2047)],
    adapters: [dict(M=-1), dict(M=1 << 22), dict(K=0), dict(K=2044), dict(K=(1 << 20) + 8), dict(N=0), dict(N=(1 << 20) + 1), dict(R=0), dict(R=12),
               dict(R=264), dict(L=0), dict(L=1024), dict(ld_x=2040), dict(ld_x=2052), dict(ld_base=4095), dict(ld_y=4095)],
}


@pytest.mark.parametrize("fn", SHAPES, ids=lambda f: f.__name__)
def test_shapes(fn):
    for bad in SHAPES[fn]:
        assert fn(**bad) == mg.MOE_ERR_SHAPE, bad


def test_arguments():
    for fn in (route, route_backward):
        assert fn(dtype=mg.MOE_F16) == fn(dtype=7) == fn(flags=8) == fn(flags=-1) == mg.MOE_ERR_ARG
    for fn in (combine, combine_backward, norm, norm_backward):
        assert fn(dtype=3) == mg.MOE_ERR_ARG
    for fn in (norm, norm_backward):
        assert fn(wt=mg.MOE_F16) == fn(dtype=mg.MOE_F32) == mg.MOE_ERR_ARG
    for eps in (0.0, -1e-6, 1e-45, float("nan"), float("inf")):
        assert norm(eps=eps) == mg.MOE_ERR_ARG
    assert norm(flags=mg.MOE_QUANT_SWIGLU) == mg.MOE_ERR_ARG
    assert adapters(dtype=mg.MOE_F32) == mg.MOE_ERR_ARG
    assert sort(ws_bytes=256) == norm_backward(ws_bytes=256) == adapters(ws_bytes=256) == mg.MOE_ERR_ARG


REQUIRED = {route: "logits ids w", route_backward: "logits ids grad d", sort: "ids counts rows pos ws", combine: "rows pos y",
            combine_backward: "dy rows pos drows", norm: "x weight", norm_backward: "dy r weight rstd dx dweight ws",
            adapters: "x ids a b s y ws"}
OPTIONAL = {route: "bias", sort: "valid", combine: "w add", combine_backward: "w dw", norm: "rstd total", norm_backward: "dsum", adapters: "base"}


@pytest.mark.parametrize("fn", REQUIRED, ids=lambda f: f.__name__)
def test_pointers(fn):
    for name in REQUIRED[fn].split():
        assert fn(**{name: 0}) == mg.MOE_ERR_NULL, name
        assert fn(**{name: at(9, 1)}) == mg.MOE_ERR_ALIGN, name
    for name in OPTIONAL.get(fn, "").split():
        if name not in ("valid",):
            assert fn(**{name: at(9, 1)}) == mg.MOE_ERR_ALIGN, name


def test_what_goes_together():
    assert norm(y=0, q=0, scales=0) == mg.MOE_ERR_NULL       # nothing is asked for
    assert norm(q=0) == norm(scales=0) == mg.MOE_ERR_NULL
    assert norm(res=0) == mg.MOE_ERR_NULL                    # a sum of one
    for name in ("x", "a", "b"):
        assert adapters(**{name: at(9, 8)}) == mg.MOE_ERR_ALIGN, name


OUTPUTS = {route: ("ids w", "logits bias"), route_backward: ("d", "logits ids grad"), sort: ("counts rows pos ws", "ids"),
           combine: ("y", "rows pos w"), combine_backward: ("drows dw", "dy rows pos w"), norm: ("y q scales total rstd", "x weight"),
           norm_backward: ("dx dweight ws", "dy r weight rstd"), adapters: ("y ws", "x ids a b s")}


@pytest.mark.parametrize("fn", OUTPUTS, ids=lambda f: f.__name__)
def test_overlaps(fn):
    import inspect
    where = {n: p.default for n, p in inspect.signature(fn).parameters.items()}
    outs, ins = (v.split() for v in OUTPUTS[fn])
    for o in outs:
        for other in ins + [p for p in outs if p != o]:
            assert fn(**{o: where[other]}) == mg.MOE_ERR_ALIAS, (o, other)


def test_in_place_is_exact():
    """An output may be the input that is added to it, not a part of it or at another stride."""
    assert combine(y=at(3, 4096)) == combine(y=at(3), ld_y=2056) == mg.MOE_ERR_ALIAS
    assert norm(total=at(1, 4096)) == norm(total=at(1), ld_sum=2056) == norm(y=at(1)) == mg.MOE_ERR_ALIAS
    assert norm_backward(dx=at(4, 4096)) == norm_backward(dx=at(4), ld_dx=2056) == mg.MOE_ERR_ALIAS
    assert adapters(y=at(5, 8192)) == adapters(y=at(5), ld_y=4104) == mg.MOE_ERR_ALIAS
    # in place, with one more output on top of it: the check behind the one that lets it pass
    assert norm(total=at(1), rstd=at(1, 8)) == mg.MOE_ERR_ALIAS
    assert norm_backward(dx=at(4), dweight=at(4, 8)) == mg.MOE_ERR_ALIAS
    assert adapters(y=at(5), ws=at(5)) == mg.MOE_ERR_ALIAS


def test_empty_calls_do_nothing():
    assert route(T=0, logits=0, ids=0, w=0) == mg.MOE_OK
    assert route_backward(T=0, logits=0, ids=0, grad=0, d=0) == mg.MOE_OK
    assert sort(T=0, ids=0, counts=0, rows=0, pos=0, ws=0) == mg.MOE_OK
    assert combine(T=0, rows=0, pos=0, y=0) == mg.MOE_OK
    assert combine_backward(T=0, dy=0, rows=0, pos=0, drows=0) == mg.MOE_OK
    assert norm(M=0, x=0, weight=0, y=0) == mg.MOE_OK
    assert norm_backward(M=0, dy=0, r=0, weight=0, rstd=0, dx=0, dweight=0, ws=0) == mg.MOE_OK
    assert adapters(M=0, x=0, ids=0, a=0, b=0, s=0, y=0, ws=0) == mg.MOE_OK


def test_workspaces():
    assert mg.moe_decode_sort_slots_workspace(1024, 1024, 8) == 0 < mg.moe_decode_sort_slots_workspace(1025, 1024, 8)
    assert mg.moe_decode_adapters_workspace(384, 64, 64, 8, 4) == 0 < mg.moe_decode_adapters_workspace(385, 64, 64, 8, 4)
    assert mg.moe_decode_adapters_workspace(96, 8192, 64, 16, 4) == 0 < mg.moe_decode_adapters_workspace(97, 8192, 64, 16, 4)
    assert mg.moe_decode_adapters_workspace(1, 2048, 64, 64, 4) == 0 < mg.moe_decode_adapters_workspace(1, 2056, 64, 64, 4)
    assert mg.moe_decode_rms_norm_backward_workspace(1, 100) >= 400
    for fn, args in ((mg.moe_decode_sort_slots_workspace, (1 << 24, 8, 1)), (mg.moe_decode_adapters_workspace, (1, 4, 1, 8, 1)),
                     (mg.moe_decode_rms_norm_backward_workspace, (1, 0))):
        with pytest.raises(mg.MoeDecodeError):
            fn(*args)


def test_binding_refuses_cpu_tensors():
    import torch
    f, i32, u8 = torch.zeros, dict(dtype=torch.int32), dict(dtype=torch.uint8)
    h = dict(dtype=torch.bfloat16)
    for call in (lambda: mg.moe_decode_route_experts(f(4, 8), f(4, 2, **i32), f(4, 2)),
                 lambda: mg.moe_decode_route_experts_backward(f(4, 8), f(4, 2, **i32), f(4, 2), f(4, 8)),
                 lambda: mg.moe_decode_sort_slots(f(4, 2, **i32), f(8, **i32), f(8, **i32), f(4, 2, **i32)),
                 lambda: mg.moe_decode_combine(f(8, 16), f(4, 2, **i32), f(4, 2), f(4, 16)),
                 lambda: mg.moe_decode_combine_backward(f(4, 16), f(8, 16), f(4, 2, **i32), f(4, 2), f(8, 16), f(4, 2)),
                 lambda: mg.moe_decode_rms_norm(f(4, 16), f(16), 1e-6, y=f(4, 16)),
                 lambda: mg.moe_decode_rms_norm(f(4, 16), f(16), 1e-6, q=f(4, 16, **u8), scales=f(4, 1)),
                 lambda: mg.moe_decode_rms_norm_backward(f(4, 16), f(4, 16), f(16), f(4), f(4, 16), f(16)),
                 lambda: mg.moe_decode_adapters(f(4, 16, **h), f(4, **i32), f(2, 8, 16, **h), f(2, 8, 8, **h), f(2), f(4, 8, **h))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("K,R", [(8, 8), (4096, 64), (4096, 256), (1 << 20, 256)])
def test_adapters_of_no_rows(K, R):
    assert mg.moe_decode_adapters_workspace(0, K, 4096, R, 64) == 0
    assert adapters(M=0, K=K, R=R, ws=None, ws_bytes=0) == mg.MOE_OK
