"""Host-side checks of the router training and block-scaled 8-bit calls of the C
ABI (CPU only: every case returns during argument validation, before any HIP
call; the pointers are addresses that are never dereferenced)."""
import ctypes

import pytest

import moe_gate_up_amd as mg

A = 0x100000000000   # aligned stand-ins for device buffers, 64 GiB apart
S = 0x1000000000


def at(i, plus=0):
    return A + i * S + plus


def P(v):
    return ctypes.c_void_p(v or None)


def balance(logits=at(0), ld=128, dtype=mg.MOE_F32, ids=at(1), valid=0, losses=at(2), counts=at(3), tokens=at(4),
            ws=at(5), ws_bytes=None, T=640, E=128, k=8, G=1):
    if ws_bytes is None:
        n = ctypes.c_size_t()
        mg.lib().moe_decode_balance_workspace(T, E, k, G, ctypes.byref(n))   # leaves 0 where it refuses
        ws_bytes = n.value
    return mg.lib().moe_decode_balance(P(logits), ld, dtype, P(ids), P(valid), P(losses), P(counts), P(tokens), P(ws),
                                       ws_bytes, T, E, k, G, None)


def backward(logits=at(0), ld=128, dtype=mg.MOE_F32, valid=0, counts=at(1), tokens=at(2), grad=at(3), d=at(4), ld_d=128,
             T=640, E=128, k=8, G=1):
    return mg.lib().moe_decode_balance_backward(P(logits), ld, dtype, P(valid), P(counts), P(tokens), P(grad), P(d), ld_d,
                                                T, E, k, G, None)


def quantize(x=at(0), ldx=2048, dtype=mg.MOE_BF16, q=at(1), s=at(2), M=32, K=2048, flags=0):
    return mg.lib().moe_decode_quantize_fp8(P(x), ldx, dtype, P(q), P(s), M, K, flags, None)


def matmul(x=at(0), ldx=2048, sx=at(1), w=at(2), sw=at(3), y=at(4), ldy=4096, dtype=mg.MOE_BF16, M=32, N=4096, K=2048,
           variant=None):
    args = [P(x), ldx, P(sx), P(w), P(sw), P(y), ldy, dtype, M, N, K]
    if variant is None:
        return mg.lib().moe_decode_matmul_fp8(*args, None)
    return mg.lib().moe_decode_matmul_fp8_ex(*args, variant, None)


def experts(x=at(0), ldx=2048, sx=at(1), rows=at(5), counts=at(6), w=at(2), sw=at(3), y=at(4), ldy=1536,
            dtype=mg.MOE_BF16, X=32, M=256, N=1536, K=2048, E=128, variant=None):
    args = [P(x), ldx, P(sx), P(rows), P(counts), P(w), P(sw), P(y), ldy, dtype, X, M, N, K, E]
    if variant is None:
        return mg.lib().moe_decode_matmul_fp8_experts(*args, None)
    return mg.lib().moe_decode_matmul_fp8_experts_ex(*args, variant, None)


@pytest.mark.parametrize("fn", [balance, backward])
def test_balance_shapes(fn):
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=65, E=128), dict(k=9, E=8, ld=8), dict(E=1025, ld=1025), dict(G=0),
                dict(G=7), dict(ld=127), dict(T=1 << 30, k=2), dict(T=1 << 21, G=1 << 21), dict(T=1 << 19, G=1 << 19, E=512, ld=512),
                dict(ld=(1 << 30) + 128)):
        if fn is backward and "ld" in bad:
            bad.setdefault("ld_d", max(bad["ld"], 0))
        assert fn(**bad) == mg.MOE_ERR_SHAPE, bad
    assert fn(dtype=mg.MOE_F16) == mg.MOE_ERR_ARG
    assert fn(dtype=7) == mg.MOE_ERR_ARG


def test_balance_pointers():
    for n in ("logits", "ids", "losses", "counts", "tokens", "ws"):
        assert balance(**{n: 0}) == mg.MOE_ERR_NULL, n
    for n, off in (("logits", 2), ("ids", 2), ("losses", 1), ("counts", 2), ("tokens", 3), ("ws", 128)):
        assert balance(**{n: at(8, off)}) == mg.MOE_ERR_ALIGN, n
    assert balance(logits=at(8, 1), dtype=mg.MOE_BF16) == mg.MOE_ERR_ALIGN
    for n in ("logits", "counts", "tokens", "grad", "d"):
        assert backward(**{n: 0}) == mg.MOE_ERR_NULL, n
    for n, off in (("logits", 2), ("counts", 2), ("tokens", 3), ("grad", 1), ("d", 2)):
        assert backward(**{n: at(8, off)}) == mg.MOE_ERR_ALIGN, n


def test_balance_overlaps():
    assert balance(counts=at(0, 64)) == mg.MOE_ERR_ALIAS
    assert balance(losses=at(1, 64)) == mg.MOE_ERR_ALIAS
    assert balance(valid=at(4)) == mg.MOE_ERR_ALIAS
    assert balance(tokens=at(3, 508)) == mg.MOE_ERR_ALIAS       # the last count
    assert balance(ws=at(0)) == mg.MOE_ERR_ALIAS
    assert balance(ws_bytes=64) == mg.MOE_ERR_ARG
    assert backward(d=at(0, 16)) == mg.MOE_ERR_ALIAS
    assert backward(d=at(1)) == mg.MOE_ERR_ALIAS
    assert backward(valid=at(4, 100)) == mg.MOE_ERR_ALIAS


def test_empty_calls_do_nothing():
    assert balance(T=0, logits=0, ids=0, losses=0, counts=0, tokens=0, ws=0) == mg.MOE_OK
    assert backward(T=0, logits=0, counts=0, tokens=0, grad=0, d=0) == mg.MOE_OK
    assert quantize(M=0, x=0, q=0, s=0) == mg.MOE_OK
    assert matmul(M=0, x=0, sx=0, w=0, sw=0, y=0) == mg.MOE_OK
    assert experts(M=0, X=0, x=0, sx=0, rows=0, counts=0, w=0, sw=0, y=0) == mg.MOE_OK
    assert mg.moe_decode_balance_workspace(0, 128, 8) == 0
    assert mg.moe_decode_balance_workspace(256, 128, 8) == 0 < mg.moe_decode_balance_workspace(257, 128, 8)
    assert mg.moe_decode_balance_workspace(256, 128, 8, 2) > 0


def test_quantize_refusals():
    for bad in (dict(M=-1), dict(K=0), dict(K=-16), dict(ldx=2047), dict(flags=mg.MOE_QUANT_SWIGLU), dict(M=1 << 26),
                dict(ldx=(1 << 30) + 1), dict(K=(1 << 28) + 1, ldx=1 << 29)):
        assert quantize(**bad) == mg.MOE_ERR_SHAPE, bad       # SwiGLU: a row of x is 2 K long
    assert quantize(flags=4) == mg.MOE_ERR_ARG
    assert quantize(flags=-1) == mg.MOE_ERR_ARG
    assert quantize(dtype=3) == mg.MOE_ERR_ARG
    for n in ("x", "q", "s"):
        assert quantize(**{n: 0}) == mg.MOE_ERR_NULL
    assert quantize(x=at(8, 1)) == mg.MOE_ERR_ALIGN
    assert quantize(x=at(8, 2), dtype=mg.MOE_F32) == mg.MOE_ERR_ALIGN
    assert quantize(s=at(8, 2)) == mg.MOE_ERR_ALIGN
    assert quantize(q=at(0, 4096)) == mg.MOE_ERR_ALIAS
    assert quantize(s=at(1, 65532)) == mg.MOE_ERR_ALIAS
    assert quantize(s=at(0, 131068)) == mg.MOE_ERR_ALIAS


@pytest.mark.parametrize("fn", [matmul, experts])
def test_matmul_refusals(fn):
    for bad in (dict(M=-1), dict(N=0), dict(K=0), dict(K=2040), dict(ldx=2032), dict(ldx=2056), dict(ldy=100),
                dict(N=1 << 20, ldy=1 << 20), dict(ldx=(1 << 30) + 16), dict(ldy=(1 << 30) + 4)):
        assert fn(**bad) == mg.MOE_ERR_SHAPE, bad
    assert fn(dtype=3) == mg.MOE_ERR_ARG
    assert fn(variant=99) == mg.MOE_ERR_ARG
    assert fn(variant=-1) == mg.MOE_ERR_ARG
    for n in ("x", "sx", "w", "sw", "y"):
        assert fn(**{n: 0}) == mg.MOE_ERR_NULL, n
    for n, off in (("x", 8), ("w", 8), ("sx", 2), ("sw", 2), ("y", 1)):
        assert fn(**{n: at(8, off)}) == mg.MOE_ERR_ALIGN, n
    assert fn(y=at(8, 2), dtype=mg.MOE_F32) == mg.MOE_ERR_ALIGN
    for i in range(4):
        assert fn(y=at(i, 16)) == mg.MOE_ERR_ALIAS, i


def test_experts_refusals():
    assert experts(counts=0) == mg.MOE_ERR_NULL
    assert experts(counts=at(8, 2)) == mg.MOE_ERR_ALIGN
    assert experts(rows=at(8, 2)) == mg.MOE_ERR_ALIGN
    assert experts(y=at(5)) == mg.MOE_ERR_ALIAS
    assert experts(y=at(6)) == mg.MOE_ERR_ALIAS
    for bad in (dict(E=0), dict(E=1025), dict(M=1 << 24), dict(X=-1), dict(X=0), dict(rows=0, X=255)):
        assert experts(**bad) == mg.MOE_ERR_SHAPE, bad


def test_variants_refuse_what_they_cannot_reach():
    far = dict(ldx=1 << 29)                        # 128 such rows pass 32-bit offsets
    for v in (mg.MOE_MATMUL_TILE_64X64, mg.MOE_MATMUL_TILE_64X128, mg.MOE_MATMUL_TILE_64X128_STREAM,
              mg.MOE_MATMUL_TILE_128X128, mg.MOE_MATMUL_TILE_256X256):
        assert matmul(variant=v, M=300, **far) == mg.MOE_ERR_ARG
        assert experts(variant=v, X=1 << 21) == mg.MOE_ERR_ARG      # 2^21 rows of 2048 bytes to pick from
    assert matmul(variant=mg.MOE_MATMUL_TILE_256X256, dtype=mg.MOE_F32) == mg.MOE_ERR_ARG


def test_plan_names_a_variant():
    for M, N, K, E in ((1, 4096, 2048, 0), (8192, 4096, 4096, 0), (256, 1536, 2048, 128), (32768, 1536, 2048, 128), (0, 128, 128, 0)):
        v, g = mg.moe_decode_matmul_fp8_plan(M, N, K, E)
        assert v >= 1 and g >= 0
    with pytest.raises(mg.MoeDecodeError):
        mg.moe_decode_matmul_fp8_plan(1, 128, 100)


def test_binding_refuses_cpu_tensors():
    import torch
    f = torch.zeros
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError):
        mg.moe_decode_balance(f(4, 8), f(4, 2, **i32), f(2), f(1, 8, **i32), f(2, **i32))
    with pytest.raises(ValueError):
        mg.moe_decode_balance_backward(f(4, 8), f(1, 8, **i32), f(2, **i32), f(2), f(4, 8), 2)
    u8 = dict(dtype=torch.uint8)
    with pytest.raises(ValueError):
        mg.moe_decode_quantize_fp8(f(4, 128), f(4, 128, **u8), f(4, 1))
    with pytest.raises(ValueError):
        mg.moe_decode_matmul_fp8(f(4, 128, **u8), f(4, 1), f(8, 128, **u8), f(1, 1), f(4, 8))
    with pytest.raises(ValueError):
        mg.moe_decode_matmul_fp8_experts(f(4, 128, **u8), f(4, 1), f(2, **i32), f(2, 8, 128, **u8), f(2, 1, 1), f(4, 8))


def test_largest_sizes():
    """The documented limits hold: beyond them 32-bit indices or a launch's 2^32 threads would not."""
    most = 2 ** 31 - 1
    n = ctypes.c_size_t()
    assert mg.lib().moe_decode_balance_workspace(1 << 30, 1, 1, 1, ctypes.byref(n)) == mg.MOE_OK and n.value > 0
    for T in ((1 << 30) + 1, most):
        assert mg.lib().moe_decode_balance_workspace(T, 1, 1, 1, ctypes.byref(n)) == mg.MOE_ERR_SHAPE
        assert balance(T=T, E=1, k=1, ld=1) == mg.MOE_ERR_SHAPE
        assert backward(T=T, E=1, k=1, ld=1, ld_d=1) == mg.MOE_ERR_SHAPE
    for bad in (dict(M=1 << 24), dict(M=1 << 28, K=1, ldx=1), dict(M=most, K=1, ldx=1), dict(M=1, K=most, ldx=most)):
        assert quantize(**bad) == mg.MOE_ERR_SHAPE, bad
    for bad in (dict(M=most, N=1, K=16, ldx=16, ldy=1), dict(M=1 << 30, N=1, K=16, ldx=16, ldy=1),
                dict(M=1, N=1, K=most - 15, ldx=most - 15)):
        for fn in (matmul, experts):
            assert fn(**bad) == mg.MOE_ERR_SHAPE, bad
    assert matmul(M=1, N=1 << 26, K=16, ldx=16, ldy=1 << 26) == mg.MOE_ERR_SHAPE
    for M, N, K, E in ((most, 1, 16, 0), (1 << 30, 1, 16, 0), (1, 1, most - 15, 0), (1, 1 << 26, 16, 0)):
        v, g = ctypes.c_int(), ctypes.c_int()
        assert mg.lib().moe_decode_matmul_fp8_plan(M, N, K, E, ctypes.byref(v), ctypes.byref(g)) == mg.MOE_ERR_SHAPE


def test_built_in_choice_on_both_sides_of_each_threshold():
    v = lambda *a: mg.moe_decode_matmul_fp8_plan(*a)[0]   # noqa: E731
    rows, t64, t128, stream, big = (mg.MOE_MATMUL_ROWS_16, mg.MOE_MATMUL_TILE_64X64, mg.MOE_MATMUL_TILE_64X128,
                                    mg.MOE_MATMUL_TILE_64X128_STREAM, mg.MOE_MATMUL_TILE_128X128)
    for size, want in (((16, 1 << 20, 128), rows), ((32, 4096, 2048), rows), ((33, 4096, 2048), t64), ((32, 4112, 2048), t64),
                       ((768, 4096, 2048), t64), ((769, 4096, 2048), t128), ((49152, 64, 2048), t64), ((49153, 64, 2048), big),
                       ((1536, 4096, 2048), t128), ((1537, 4096, 2048), big), ((8192, 4096, 4096), big)):
        assert v(*size) == want, size
    for size, want in (((21, 1536, 2048, 128), t64), ((22, 1536, 2048, 128), stream), ((256, 1536, 2048, 128), stream),
                       ((4223, 1536, 2048, 128), stream), ((4224, 1536, 2048, 128), t128), ((10239, 1536, 2048, 128), t128),
                       ((10240, 1536, 2048, 128), big), ((4416, 768, 2048, 16), t128), ((4480, 768, 2048, 16), big)):
        assert v(*size) == want, size


def test_sums_asked_for_with_the_variant():
    f = mg.MOE_MATMUL_FP8_SUMS
    for fn in (matmul, experts):
        assert fn(variant=f | 99) == mg.MOE_ERR_ARG
        assert fn(variant=2 * f) == mg.MOE_ERR_ARG
        assert fn(variant=f | mg.MOE_MATMUL_TILE_256X256, dtype=mg.MOE_F32) == mg.MOE_ERR_ARG
        for v in (0, f, f | mg.MOE_MATMUL_TILE_64X64, mg.MOE_MATMUL_TILE_256X256):
            assert fn(variant=v, y=at(2, 16)) == mg.MOE_ERR_ALIAS


def test_a_launch_holds_fewer_than_2_to_32_threads():
    """One column of tiles for up to 2^30 - 1 rows, in workgroups of 256 threads."""
    for M, N in (((1 << 30) - 1, 1), ((1 << 30) - 1, 128), (1 << 29, 128)):
        variant, blocks = mg.moe_decode_matmul_fp8_plan(M, N, 16)
        assert variant == mg.MOE_MATMUL_TILE_128X128 and 256 * blocks < 2 ** 32
    for M, N in ((1 << 30, 1), ((1 << 30) - 1, 300)):
        with pytest.raises(mg.MoeDecodeError):
            mg.moe_decode_matmul_fp8_plan(M, N, 16)


def test_binding_refuses_other_orders_of_the_same_elements(monkeypatch):
    """Scales block by block instead of row by row, transposed or regrouped matrices, counts expert by expert: as many
    elements in another order.  (CPU tensors stand in: every call is refused before it reaches the library.)"""
    import torch
    mg._load()
    monkeypatch.setattr(mg, "_gpu", lambda t, name: t.get_device())
    monkeypatch.setattr(mg, "_call", lambda where, fn, device, stream, *args: pytest.fail(f"{where} was called"))
    f, u8, i32 = torch.zeros, dict(dtype=torch.uint8), dict(dtype=torch.int32)
    x, sx, w, sw, y = f(4, 384, **u8), f(4, 3), f(256, 384, **u8), f(2, 3), f(4, 256)
    ok = [x, sx, w, sw, y]
    for i, bad in ((1, f(3, 4)), (1, f(12)), (2, f(384, 256, **u8)), (2, f(256, 3, 128, **u8)), (3, f(3, 2)), (3, f(6))):
        with pytest.raises(ValueError):
            mg.moe_decode_matmul_fp8(*ok[:i], bad, *ok[i + 1:])
    ok = [x, sx, f(2, **i32), f(2, 256, 384, **u8), f(2, 2, 3), y]
    for i, bad in ((1, f(3, 4)), (2, f(2, 1, **i32)), (3, f(2, 256, 3, 128, **u8)), (4, f(2, 3, 2)), (4, f(4, 3)), (4, f(2, 6))):
        with pytest.raises(ValueError):
            mg.moe_decode_matmul_fp8_experts(*ok[:i], bad, *ok[i + 1:])
    with pytest.raises(ValueError):
        mg.moe_decode_quantize_fp8(f(4, 384), f(4, 384, **u8), f(3, 4))
    with pytest.raises(ValueError):
        mg.moe_decode_balance(f(6, 8), f(6, 2, **i32), f(2), f(2, 2, 4, **i32), f(3, **i32))
    with pytest.raises(ValueError):
        mg.moe_decode_balance_backward(f(6, 8), f(2, 2, 4, **i32), f(3, **i32), f(2), f(6, 8), 2)


def test_binding_takes_what_has_one_meaning(monkeypatch):
    """A mask by group, ids by group and token, counts of one group as a row."""
    import torch
    mg._load()
    calls = []
    monkeypatch.setattr(mg, "_gpu", lambda t, name: t.get_device())
    monkeypatch.setattr(mg, "_call", lambda where, fn, device, stream, *args: calls.append(where))
    f, u8, i32 = torch.zeros, dict(dtype=torch.uint8), dict(dtype=torch.int32)
    mg.moe_decode_balance(f(6, 8), f(2, 3, 2, **i32), f(2), f(2, 8, **i32), f(3, **i32), valid=f(2, 3, dtype=torch.bool))
    for counts in (f(2, **i32), f(1, 2, **i32)):
        mg.moe_decode_matmul_fp8_experts(f(4, 384, **u8), f(4, 3), counts, f(2, 256, 384, **u8), f(2, 2, 3), f(4, 256),
                                         x_rows=f(2, 2, **i32))
    assert len(calls) == 3


def test_quantising_launches_fewer_than_2_to_32_threads():
    """16 threads a block of 128, in workgroups of 256: 2^28 - 16 blocks are the most.  (One more argument is wrong in the
    calls that the sizes allow, so nothing is launched.)"""
    for M, K, want in (((1 << 28) - 16, 1, mg.MOE_ERR_ALIAS), ((1 << 28) - 15, 1, mg.MOE_ERR_SHAPE), ((1 << 28) - 1, 128, mg.MOE_ERR_SHAPE),
                       ((1 << 27) - 8, 129, mg.MOE_ERR_ALIAS), ((1 << 27) - 7, 129, mg.MOE_ERR_SHAPE)):
        assert quantize(M=M, K=K, ldx=K, q=at(0)) == want, (M, K)
