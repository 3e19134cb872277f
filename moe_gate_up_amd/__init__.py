"""Python binding of the warp-decode MoE decode layer's C ABI (include/moe_decode.h).

Argument marshalling only: every step of the layer runs in the HIP kernels of
``libmoe_decode.so``.  PyTorch supplies device memory and streams.  There is no
fallback: if the library is missing, or a tensor is not on the GPU, the calls
raise.

The functions keep the C names and argument order; tensor shapes are checked
against the declared sizes before anything is launched, so a mis-sized tensor
raises here instead of being read out of bounds on the device.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_decode.so")

MOE_OK = 0
MOE_ERR_NULL = -1
MOE_ERR_SHAPE = -2
MOE_ERR_ALIGN = -3
MOE_ERR_LAUNCH = -4
MOE_ERR_ALIAS = -5
MOE_ERR_ARG = -6
MOE_ERR_SCRATCH = -7
MOE_GATE_UP_PER_SLOT = 1
MOE_GATE_UP_EXPERT_GROUPED = 2
MOE_GATE_UP_EXPERT_GROUPED_MFMA = 3
MOE_DOWN_PER_TOKEN = 1
MOE_DOWN_EXPERT_GROUPED = 2
MOE_DOWN_EXPERT_GROUPED_MFMA = 3
MOE_F32 = 0
MOE_BF16 = 1
MOE_F16 = 2
MOE_QUANT_SWIGLU = 1
MOE_QUANT_POW2 = 2
MOE_MATMUL_ROWS_16 = 1
MOE_MATMUL_TILE_64X64 = 2
MOE_MATMUL_TILE_64X128 = 3
MOE_MATMUL_TILE_64X128_STREAM = 4
MOE_MATMUL_TILE_128X128 = 5
MOE_MATMUL_TILE_256X256 = 6
MOE_MATMUL_FAR_ROWS = 7
MOE_MATMUL_FP8_SUMS = 256
MOE_ROUTE_SIGMOID = 1
MOE_ROUTE_RENORM = 2
MOE_ROUTE_GROUP_TOP2 = 4

EXPORTS = (
    "moe_decode_gate_up", "moe_decode_down", "moe_decode_gate_up_ex", "moe_decode_down_ex",
    "moe_decode_gate_up_plan", "moe_decode_down_plan", "moe_decode_conventional_workspace",
    "moe_decode_conventional", "moe_decode_conventional_noalloc", "moe_decode_route", "moe_decode_gate_up_routed", "moe_decode_gate_up_routed_ex",
    "moe_decode_balance_workspace", "moe_decode_balance", "moe_decode_balance_backward", "moe_decode_quantize_fp8",
    "moe_decode_matmul_fp8", "moe_decode_matmul_fp8_ex", "moe_decode_matmul_fp8_experts",
    "moe_decode_matmul_fp8_experts_ex", "moe_decode_matmul_fp8_plan",
    "moe_decode_route_experts", "moe_decode_route_experts_backward", "moe_decode_sort_slots_workspace",
    "moe_decode_sort_slots", "moe_decode_combine", "moe_decode_combine_backward", "moe_decode_rms_norm",
    "moe_decode_rms_norm_backward_workspace", "moe_decode_rms_norm_backward", "moe_decode_adapters_workspace",
    "moe_decode_adapters",
    "moe_decode_copy_peak", "moe_decode_read_peak",
    "moe_decode_strerror",
)

_lock = threading.Lock()
_lib = None


class MoeDecodeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} (code {code})")


def lib() -> ctypes.CDLL:
    """Load libmoe_decode.so (built by __graft_entry__.build() / moe_gate_up_amd.build)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing (run __graft_entry__.build())")
            L = ctypes.CDLL(LIB_PATH)
            P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
            IP = ctypes.POINTER(ctypes.c_int)
            L.moe_decode_gate_up.argtypes = [P] * 7 + [I] * 5 + [P]
            L.moe_decode_down.argtypes = [P] * 6 + [I] * 5 + [P]
            L.moe_decode_gate_up_ex.argtypes = [P] * 7 + [I] * 7 + [P]
            L.moe_decode_down_ex.argtypes = [P] * 6 + [I] * 7 + [P]
            L.moe_decode_gate_up_plan.argtypes = [I] * 5 + [IP, IP, IP]
            L.moe_decode_down_plan.argtypes = [I] * 5 + [IP, IP, IP]
            L.moe_decode_conventional_workspace.argtypes = [I] * 5 + [ctypes.POINTER(ctypes.c_size_t)]
            L.moe_decode_conventional.argtypes = [P] * 11 + [S] + [I] * 5 + [P]
            L.moe_decode_conventional_noalloc.argtypes = [P] * 10 + [I] * 5 + [P]
            L.moe_decode_route.argtypes = [P] * 3 + [I] * 3 + [P]
            L.moe_decode_gate_up_routed.argtypes = [P] * 9 + [I] * 5 + [P]
            L.moe_decode_gate_up_routed_ex.argtypes = [P] * 9 + [I] * 7 + [P]
            LL = ctypes.c_longlong
            L.moe_decode_balance_workspace.argtypes = [I] * 4 + [ctypes.POINTER(S)]
            L.moe_decode_balance.argtypes = [P, LL, I] + [P] * 6 + [S] + [I] * 4 + [P]
            L.moe_decode_balance_backward.argtypes = [P, LL, I] + [P] * 5 + [LL] + [I] * 4 + [P]
            L.moe_decode_quantize_fp8.argtypes = [P, LL, I, P, P, I, I, I, P]
            L.moe_decode_matmul_fp8.argtypes = [P, LL, P, P, P, P, LL] + [I] * 4 + [P]
            L.moe_decode_matmul_fp8_ex.argtypes = [P, LL, P, P, P, P, LL] + [I] * 5 + [P]
            L.moe_decode_matmul_fp8_experts.argtypes = [P, LL] + [P] * 6 + [LL] + [I] * 6 + [P]
            L.moe_decode_matmul_fp8_experts_ex.argtypes = [P, LL] + [P] * 6 + [LL] + [I] * 7 + [P]
            L.moe_decode_matmul_fp8_plan.argtypes = [I] * 4 + [IP, IP]
            SP, F = ctypes.POINTER(S), ctypes.c_float
            L.moe_decode_route_experts.argtypes = [P, LL, I, P, P, P] + [I] * 6 + [F, P]
            L.moe_decode_route_experts_backward.argtypes = [P, LL, I, P, P, P, LL] + [I] * 4 + [F, P]
            L.moe_decode_sort_slots_workspace.argtypes = [I] * 3 + [SP]
            L.moe_decode_sort_slots.argtypes = [P] * 6 + [S] + [I] * 3 + [P]
            L.moe_decode_combine.argtypes = [P, LL, I, P, P, P, LL, P, LL] + [I] * 4 + [P]
            L.moe_decode_combine_backward.argtypes = [P, LL, P, LL, I, P, P, P, LL, P] + [I] * 4 + [P]
            L.moe_decode_rms_norm.argtypes = [P, LL, P, LL, I, P, I, F, P, LL, P, P, P, LL, P, I, I, I, P]
            L.moe_decode_rms_norm_backward_workspace.argtypes = [I, I, SP]
            L.moe_decode_rms_norm_backward.argtypes = [P, LL, P, LL, I, P, I, P, P, LL, P, LL, P, P, S, I, I, P]
            L.moe_decode_adapters_workspace.argtypes = [I] * 5 + [SP]
            L.moe_decode_adapters.argtypes = [P, LL, I, P, P, P, P, P, LL, P, LL, P, S] + [I] * 5 + [P]
            L.moe_decode_copy_peak.argtypes = [P, P, S, P]
            L.moe_decode_read_peak.argtypes = [P, S, P, P]
            L.moe_decode_strerror.argtypes = [I]
            L.moe_decode_strerror.restype = ctypes.c_char_p
            for n in EXPORTS[:-1]:
                getattr(L, n).restype = I
            _lib = L
        return _lib


def strerror(code: int) -> str:
    return lib().moe_decode_strerror(int(code)).decode()


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _dev(t, name, numel=None, dtypes=None):
    if t is None:
        return None
    if not getattr(t, "is_cuda", False):
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    return ctypes.c_void_p(t.data_ptr())


def _types():
    import torch
    return dict(bf16=(torch.bfloat16, torch.int16, torch.uint16), i32=(torch.int32,), f32=(torch.float32,),
                u8=(torch.uint8,))


def moe_decode_gate_up(x, topk_ids, w_gate, s_gate, w_up, s_up, h_out, B=None, H=None, I=None, E=None, k=None,
                       stream=None, rows_per_wave=None, variant=None):
    """h_out[b,j,n] = bf16(SiLU(gate) * up) for expert topk_ids[b,j] (see include/moe_decode.h)."""
    T = _types()
    B = x.shape[0] if B is None else B
    H = x.shape[-1] if H is None else H
    k = topk_ids.shape[-1] if k is None else k
    E = w_gate.shape[0] if E is None else E
    I = w_gate.shape[1] if I is None else I
    args = [
        _dev(x, "x", B * H, T["bf16"]), _dev(topk_ids, "topk_ids", B * k, T["i32"]),
        _dev(w_gate, "w_gate", E * I * H, T["u8"]), _dev(s_gate, "s_gate", E * I * (H // 32), T["u8"]),
        _dev(w_up, "w_up", E * I * H, T["u8"]), _dev(s_up, "s_up", E * I * (H // 32), T["u8"]),
        _dev(h_out, "h_out", B * k * I, T["bf16"]), B, H, I, E, k,
    ]
    if rows_per_wave is None and variant is None:
        rc = lib().moe_decode_gate_up(*args, _stream(stream))
    else:
        rc = lib().moe_decode_gate_up_ex(*args, int(variant or 0), int(rows_per_wave or 0), _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_gate_up")
    return h_out


def moe_decode_route(logits, topk_ids, topk_weights, B=None, E=None, k=None, stream=None):
    """Top-k router: topk_ids / topk_weights [B,k] from logits fp32 [B,E] (see include/moe_decode.h)."""
    T = _types()
    B = logits.shape[0] if B is None else B
    E = logits.shape[-1] if E is None else E
    k = topk_ids.shape[-1] if k is None else k
    rc = lib().moe_decode_route(
        _dev(logits, "logits", B * E, T["f32"]), _dev(topk_ids, "topk_ids", B * k, T["i32"]),
        _dev(topk_weights, "topk_weights", B * k, T["f32"]), B, E, k, _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_route")
    return topk_ids, topk_weights


def moe_decode_gate_up_routed(x, logits, w_gate, s_gate, w_up, s_up, h_out, topk_ids_out, topk_weights_out,
                              B=None, H=None, I=None, E=None, k=None, stream=None, rows_per_wave=None, variant=None):
    """gate/up with the top-k router step fused in: h_out, topk_ids_out and topk_weights_out
    from x and the router logits (see include/moe_decode.h)."""
    T = _types()
    B = x.shape[0] if B is None else B
    H = x.shape[-1] if H is None else H
    k = topk_ids_out.shape[-1] if k is None else k
    E = w_gate.shape[0] if E is None else E
    I = w_gate.shape[1] if I is None else I
    args = [
        _dev(x, "x", B * H, T["bf16"]), _dev(logits, "logits", B * E, T["f32"]),
        _dev(w_gate, "w_gate", E * I * H, T["u8"]), _dev(s_gate, "s_gate", E * I * (H // 32), T["u8"]),
        _dev(w_up, "w_up", E * I * H, T["u8"]), _dev(s_up, "s_up", E * I * (H // 32), T["u8"]),
        _dev(h_out, "h_out", B * k * I, T["bf16"]), _dev(topk_ids_out, "topk_ids_out", B * k, T["i32"]),
        _dev(topk_weights_out, "topk_weights_out", B * k, T["f32"]), B, H, I, E, k,
    ]
    if rows_per_wave is None and variant is None:
        rc = lib().moe_decode_gate_up_routed(*args, _stream(stream))
    else:
        rc = lib().moe_decode_gate_up_routed_ex(*args, int(variant or 0), int(rows_per_wave or 0), _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_gate_up_routed")
    return h_out, topk_ids_out, topk_weights_out


def moe_decode_down(h, topk_ids, topk_weights, w_down, s_down, y_out, B=None, H=None, I=None, E=None, k=None,
                    stream=None, rows_per_wave=None, variant=None):
    """y_out[b,o] = bf16(sum_j w[b,j] * down row . h[b,j,:]) (see include/moe_decode.h)."""
    T = _types()
    B = h.shape[0] if B is None else B
    k = topk_ids.shape[-1] if k is None else k
    E = w_down.shape[0] if E is None else E
    H = w_down.shape[1] if H is None else H
    I = w_down.shape[2] if I is None else I
    args = [
        _dev(h, "h", B * k * I, T["bf16"]), _dev(topk_ids, "topk_ids", B * k, T["i32"]),
        _dev(topk_weights, "topk_weights", B * k, T["f32"]),
        _dev(w_down, "w_down", E * H * I, T["u8"]), _dev(s_down, "s_down", E * H * (I // 32), T["u8"]),
        _dev(y_out, "y_out", B * H, T["bf16"]), B, H, I, E, k,
    ]
    if rows_per_wave is None and variant is None:
        rc = lib().moe_decode_down(*args, _stream(stream))
    else:
        rc = lib().moe_decode_down_ex(*args, int(variant or 0), int(rows_per_wave or 0), _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_down")
    return y_out


def moe_decode_gate_up_plan(B, H, I, E, k):
    """(variant, rows_per_wave, workgroups) the built-in table picks."""
    v, r, g = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = lib().moe_decode_gate_up_plan(B, H, I, E, k, ctypes.byref(v), ctypes.byref(r), ctypes.byref(g))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_gate_up_plan")
    return v.value, r.value, g.value


def moe_decode_down_plan(B, H, I, E, k):
    """(variant, rows_per_wave, workgroups) the built-in table picks."""
    v, r, g = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = lib().moe_decode_down_plan(B, H, I, E, k, ctypes.byref(v), ctypes.byref(r), ctypes.byref(g))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_down_plan")
    return v.value, r.value, g.value


def moe_decode_conventional_workspace(B, H, I, E, k):
    """Bytes of device workspace moe_decode_conventional needs."""
    n = ctypes.c_size_t()
    rc = lib().moe_decode_conventional_workspace(B, H, I, E, k, ctypes.byref(n))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_conventional_workspace")
    return n.value


def moe_decode_conventional(x, topk_ids, topk_weights, w_gate, s_gate, w_up, s_up, w_down, s_down, y_out, workspace,
                            stream=None):
    """The expert-centric path (see include/moe_decode.h); workspace: a uint8 GPU tensor."""
    T = _types()
    B, H = x.shape
    k = topk_ids.shape[-1]
    E, I = w_gate.shape[0], w_gate.shape[1]
    wb = E * I * H
    args = [
        _dev(x, "x", B * H, T["bf16"]), _dev(topk_ids, "topk_ids", B * k, T["i32"]),
        _dev(topk_weights, "topk_weights", B * k, T["f32"]),
        _dev(w_gate, "w_gate", wb, T["u8"]), _dev(s_gate, "s_gate", wb // 32, T["u8"]),
        _dev(w_up, "w_up", wb, T["u8"]), _dev(s_up, "s_up", wb // 32, T["u8"]),
        _dev(w_down, "w_down", wb, T["u8"]), _dev(s_down, "s_down", wb // 32, T["u8"]),
        _dev(y_out, "y_out", B * H, T["bf16"]), _dev(workspace, "workspace", None, T["u8"]),
        workspace.numel(), B, H, I, E, k,
    ]
    rc = lib().moe_decode_conventional(*args, _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_conventional")
    return y_out


def moe_decode_conventional_noalloc(x, topk_ids, topk_weights, w_gate, s_gate, w_up, s_up, w_down, s_down, y_out,
                                    stream=None):
    """The expert-centric path on the library's fixed scratch buffer, with no
    workspace and no allocation (see include/moe_decode.h)."""
    T = _types()
    B, H = x.shape
    k = topk_ids.shape[-1]
    E, I = w_gate.shape[0], w_gate.shape[1]
    wb = E * I * H
    args = [
        _dev(x, "x", B * H, T["bf16"]), _dev(topk_ids, "topk_ids", B * k, T["i32"]),
        _dev(topk_weights, "topk_weights", B * k, T["f32"]),
        _dev(w_gate, "w_gate", wb, T["u8"]), _dev(s_gate, "s_gate", wb // 32, T["u8"]),
        _dev(w_up, "w_up", wb, T["u8"]), _dev(s_up, "s_up", wb // 32, T["u8"]),
        _dev(w_down, "w_down", wb, T["u8"]), _dev(s_down, "s_down", wb // 32, T["u8"]),
        _dev(y_out, "y_out", B * H, T["bf16"]), B, H, I, E, k,
    ]
    rc = lib().moe_decode_conventional_noalloc(*args, _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_conventional_noalloc")
    return y_out


# ---------------------------------------------------------------- router training and block-scaled 8-bit products
_torch = None   # the module and what is looked up in it once, by _load()
_codes = {}     # tensor type -> MOE_F32 / MOE_BF16 / MOE_F16; 16-bit integer tensors hold bf16 patterns


def _load():
    """The library, with torch's lookups done once: a small call costs more on the host than on the GPU."""
    global _torch, _u8, _i32, _f32, _flags, _raw_stream, _raw_device
    if _torch is None:
        import torch
        _codes.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.int16: MOE_BF16,
                       torch.uint16: MOE_BF16, torch.float16: MOE_F16})
        _u8, _i32, _f32, _flags = torch.uint8, torch.int32, torch.float32, (torch.bool, torch.uint8)
        # the current stream's handle and the current device without a Python object around them
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
        _raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _torch = torch
    return _lib or lib()


def _dtype_code(t, name, allowed):
    c = _codes.get(t.dtype)
    if c is None or c not in allowed:
        raise ValueError(f"{name} has dtype {t.dtype}, which this call does not take")
    return c


def _rows(t, name, device, rows, cols):
    """Row stride of a GPU matrix [rows, cols] whose rows are contiguous (they may lie apart)."""
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on GPU {device}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, cols)}")
    if rows < 2 or cols < 2:
        ld, one = t.stride()
        if one != 1 and cols > 1:
            raise ValueError(f"{name}: the elements of a row must be contiguous")
        return ld if rows > 1 else cols
    ld, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return ld


def _mat(t, name, device, like, rows, cols):
    """Address and row stride of a GPU matrix of the type of `like`, as _rows() checks it, in few lookups."""
    if t.dtype is not like and _codes.get(t.dtype) != _codes[like]:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {like}")
    if t.shape == (rows, cols) and t.get_device() == device:
        ld, one = t.stride()
        if one == 1:
            return t.data_ptr(), ld if rows > 1 else cols
    return t.data_ptr(), _rows(t, name, device, rows, cols)


def _flat(t, name, device, size, dtype):
    """Address of a contiguous GPU tensor of that shape (a tuple), or of that many elements (a number) where its rows
    have one meaning only."""
    if t.get_device() != device:
        raise ValueError(f"{name} is on {t.device}, not on GPU {device}")
    if t.dtype is not dtype and (dtype is not _flags or t.dtype not in _flags):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if (t.numel() if isinstance(size, int) else t.shape) != size or not t.is_contiguous():
        raise ValueError(f"{name}: expected {size} contiguous elements, got shape {tuple(t.shape)}, strides {t.stride()}")
    return t.data_ptr()


def _gpu(t, name):
    """The GPU that holds `t`."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    return i


def _call(where, fn, device, stream, *args):
    """fn(*args, stream) with the GPU `device` current: on its current stream where none is given."""
    s = _raw_stream(device) if stream is None else stream if isinstance(stream, int) else stream.cuda_stream
    if device == _raw_device():
        rc = fn(*args, s)
    else:
        with _torch.cuda.device(device):
            rc = fn(*args, s)
    if rc:
        raise MoeDecodeError(rc, where)


@functools.lru_cache(maxsize=256)
def moe_decode_balance_workspace(T, E, k, G=1):
    """Bytes of device workspace moe_decode_balance needs."""
    n = ctypes.c_size_t()
    rc = lib().moe_decode_balance_workspace(T, E, k, G, ctypes.byref(n))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_balance_workspace")
    return n.value


def moe_decode_balance(logits, topk_ids, losses, counts, tokens, valid=None, workspace=None, stream=None):
    """Per-expert counts [G,E], valid tokens [G+1], and the balance and z losses [2] of the router's
    logits [T,E] (fp32 or bf16) and choices topk_ids [T,k] (see include/moe_decode.h).

    valid: [T] bool or uint8, the tokens that count.  Without a workspace one is taken from torch's
    allocator for the call (which then runs on the current stream)."""
    L = _load()
    d = _gpu(logits, "logits")
    T, E = logits.shape
    k, G = topk_ids.shape[-1], counts.shape[0]
    dt = _dtype_code(logits, "logits", (MOE_F32, MOE_BF16))
    ld = _rows(logits, "logits", d, T, E)
    n = moe_decode_balance_workspace(T, E, k, G) if workspace is None else workspace.numel()
    if workspace is None and n:
        if stream is not None:
            raise ValueError("moe_decode_balance on a given stream needs a workspace")
        workspace = _torch.empty(n, dtype=_u8, device=logits.device)
    _call("moe_decode_balance", L.moe_decode_balance, d, stream, logits.data_ptr(), ld, dt,
          _flat(topk_ids, "topk_ids", d, T * k, _i32), None if valid is None else _flat(valid, "valid", d, T, _flags),
          _flat(losses, "losses", d, 2, _f32), _flat(counts, "counts", d, (G, E), _i32),
          _flat(tokens, "tokens", d, G + 1, _i32),
          None if workspace is None else _flat(workspace, "workspace", d, n, _u8), n, T, E, k, G)
    return losses, counts, tokens


def moe_decode_balance_backward(logits, counts, tokens, grad_losses, dlogits, k, valid=None, stream=None):
    """dlogits [T,E] = the gradient of grad_losses . losses of moe_decode_balance with respect to the logits, from
    the counts and tokens that call left (see include/moe_decode.h)."""
    L = _load()
    d = _gpu(logits, "logits")
    T, E = logits.shape
    G = counts.shape[0]
    dt = _dtype_code(logits, "logits", (MOE_F32, MOE_BF16))
    if _codes.get(dlogits.dtype) != dt:
        raise ValueError("dlogits must have the type of logits")
    _call("moe_decode_balance_backward", L.moe_decode_balance_backward, d, stream, logits.data_ptr(),
          _rows(logits, "logits", d, T, E), dt, None if valid is None else _flat(valid, "valid", d, T, _flags),
          _flat(counts, "counts", d, (G, E), _i32), _flat(tokens, "tokens", d, G + 1, _i32),
          _flat(grad_losses, "grad_losses", d, 2, _f32), dlogits.data_ptr(), _rows(dlogits, "dlogits", d, T, E),
          T, E, k, G)
    return dlogits


def moe_decode_quantize_fp8(x, q, scales, swiglu=False, pow2=False, stream=None):
    """q [M,K] E4M3 codes (uint8) and scales fp32 [M, ceil(K/128)] of x [M,K], or with swiglu of
    SiLU(x[:, :K]) * x[:, K:] of x [M,2K]; pow2: scales are powers of two (see include/moe_decode.h)."""
    L = _load()
    d = _gpu(x, "x")
    M, K = q.shape
    _call("moe_decode_quantize_fp8", L.moe_decode_quantize_fp8, d, stream, x.data_ptr(),
          _rows(x, "x", d, M, 2 * K if swiglu else K), _dtype_code(x, "x", (MOE_F32, MOE_BF16, MOE_F16)),
          _flat(q, "q", d, M * K, _u8), _flat(scales, "scales", d, (M, -(-K // 128)), _f32), M, K,
          (MOE_QUANT_SWIGLU if swiglu else 0) | (MOE_QUANT_POW2 if pow2 else 0))
    return q, scales


def moe_decode_matmul_fp8(x, sx, w, sw, y, stream=None, variant=None, fp8_sums=False):
    """y [M,N] = the product of x [M,K] and w [N,K] (E4M3 codes, uint8) with scales sx [M, ceil(K/128)] and
    sw [ceil(N/128), ceil(K/128)]; fp8_sums lets a 16-bit y have the FP8 instruction's sums, faster and less exact
    (see include/moe_decode.h)."""
    L = _load()
    d = _gpu(x, "x")
    M, K = x.shape
    N = w.shape[0]
    kb = -(-K // 128)
    if x.dtype is not _u8:
        raise ValueError(f"x has dtype {x.dtype}, expected torch.uint8 (E4M3 codes)")
    args = (x.data_ptr(), _rows(x, "x", d, M, K), _flat(sx, "sx", d, (M, kb), _f32), _flat(w, "w", d, (N, K), _u8),
            _flat(sw, "sw", d, (-(-N // 128), kb), _f32), y.data_ptr(), _rows(y, "y", d, M, N),
            _dtype_code(y, "y", (MOE_F32, MOE_BF16, MOE_F16)), M, N, K)
    if variant is None and not fp8_sums:
        _call("moe_decode_matmul_fp8", L.moe_decode_matmul_fp8, d, stream, *args)
    else:
        _call("moe_decode_matmul_fp8", L.moe_decode_matmul_fp8_ex, d, stream, *args, int(variant or 0) | (MOE_MATMUL_FP8_SUMS if fp8_sums else 0))
    return y


def moe_decode_matmul_fp8_experts(x, sx, counts, w, sw, y, x_rows=None, stream=None, variant=None, fp8_sums=False):
    """The product of moe_decode_matmul_fp8 for E matrices w [E,N,K] on rows sorted by expert, counts [E] (int32) of
    them each; x_rows [M] (int32): the row of x that each row of y comes from (see include/moe_decode.h).

    With moe_decode_balance's counts, added up over its groups, the sorted rows are the slots of valid tokens with ids in
    [0, E); all other slots go behind them."""
    L = _load()
    d = _gpu(x, "x")
    X, K = x.shape
    E, N, M = w.shape[0], w.shape[1], y.shape[0]
    kb = -(-K // 128)
    if x.dtype is not _u8:
        raise ValueError(f"x has dtype {x.dtype}, expected torch.uint8 (E4M3 codes)")
    args = (x.data_ptr(), _rows(x, "x", d, X, K), _flat(sx, "sx", d, (X, kb), _f32),
            None if x_rows is None else _flat(x_rows, "x_rows", d, M, _i32),
            _flat(counts, "counts", d, (E,) if counts.dim() == 1 else (1, E), _i32),
            _flat(w, "w", d, (E, N, K), _u8), _flat(sw, "sw", d, (E, -(-N // 128), kb), _f32), y.data_ptr(),
            _rows(y, "y", d, M, N), _dtype_code(y, "y", (MOE_F32, MOE_BF16, MOE_F16)), X, M, N, K, E)
    if variant is None and not fp8_sums:
        _call("moe_decode_matmul_fp8_experts", L.moe_decode_matmul_fp8_experts, d, stream, *args)
    else:
        _call("moe_decode_matmul_fp8_experts", L.moe_decode_matmul_fp8_experts_ex, d, stream, *args, int(variant or 0) | (MOE_MATMUL_FP8_SUMS if fp8_sums else 0))
    return y


def moe_decode_matmul_fp8_plan(M, N, K, E=0):
    """(variant, workgroups) the built-in choice for these sizes (E = 0: one matrix)."""
    v, g = ctypes.c_int(), ctypes.c_int()
    rc = lib().moe_decode_matmul_fp8_plan(M, N, K, E, ctypes.byref(v), ctypes.byref(g))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_matmul_fp8_plan")
    return v.value, g.value


# ---------------------------------------------------------------- around the experts: router, slots, norm, adapters
def moe_decode_route_experts(logits, topk_ids, topk_weights, bias=None, sigmoid=False, renorm=True, groups=1, top_groups=1,
                             group_top2=False, scale=1.0, stream=None):
    """topk_ids (int32) and topk_weights (fp32) [T,k] from the router's logits [T,E] (fp32 or bf16): the k largest of
    softmax (or sigmoid) scores + bias [E] within the top_groups best groups of experts, weighted with the scores, over
    their sum with renorm, times scale (see include/moe_decode.h)."""
    L = _load()
    d = _gpu(logits, "logits")
    T, E = logits.shape
    k = topk_ids.shape[-1]
    _call("moe_decode_route_experts", L.moe_decode_route_experts, d, stream, logits.data_ptr(),
          _rows(logits, "logits", d, T, E), _dtype_code(logits, "logits", (MOE_F32, MOE_BF16)),
          None if bias is None else _flat(bias, "bias", d, E, _f32), _flat(topk_ids, "topk_ids", d, T * k, _i32),
          _flat(topk_weights, "topk_weights", d, (T, k), _f32), T, E, k, groups, top_groups,
          (MOE_ROUTE_SIGMOID if sigmoid else 0) | (MOE_ROUTE_RENORM if renorm else 0) |
          (MOE_ROUTE_GROUP_TOP2 if group_top2 else 0), scale)
    return topk_ids, topk_weights


def moe_decode_route_experts_backward(logits, topk_ids, grad_weights, dlogits, sigmoid=False, renorm=True, scale=1.0,
                                      stream=None):
    """dlogits [T,E] = the gradient of grad_weights [T,k] . topk_weights of moe_decode_route_experts with respect to the
    logits, for the choices topk_ids it made (see include/moe_decode.h)."""
    L = _load()
    d = _gpu(logits, "logits")
    T, E = logits.shape
    k = topk_ids.shape[-1]
    dt = _dtype_code(logits, "logits", (MOE_F32, MOE_BF16))
    if _codes.get(dlogits.dtype) != dt:
        raise ValueError("dlogits must have the type of logits")
    _call("moe_decode_route_experts_backward", L.moe_decode_route_experts_backward, d, stream, logits.data_ptr(),
          _rows(logits, "logits", d, T, E), dt, _flat(topk_ids, "topk_ids", d, T * k, _i32),
          _flat(grad_weights, "grad_weights", d, (T, k), _f32), dlogits.data_ptr(), _rows(dlogits, "dlogits", d, T, E),
          T, E, k, (MOE_ROUTE_SIGMOID if sigmoid else 0) | (MOE_ROUTE_RENORM if renorm else 0), scale)
    return dlogits


@functools.lru_cache(maxsize=256)
def moe_decode_sort_slots_workspace(T, E, k):
    """Bytes of device workspace moe_decode_sort_slots needs."""
    n = ctypes.c_size_t()
    rc = lib().moe_decode_sort_slots_workspace(T, E, k, ctypes.byref(n))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_sort_slots_workspace")
    return n.value


def _workspace(workspace, need, device, stream, where):
    """(tensor or None, its bytes): the caller's workspace, or `need` bytes of torch's allocator on the current stream."""
    if workspace is not None:
        return _flat(workspace, "workspace", device, workspace.numel(), _u8), workspace.numel(), workspace
    if not need:
        return None, 0, None
    if stream is not None:
        raise ValueError(f"{where} on a given stream needs a workspace")
    t = _torch.empty(need, dtype=_u8, device=device)
    return t.data_ptr(), need, t


def moe_decode_sort_slots(topk_ids, counts, x_rows, positions, valid=None, workspace=None, stream=None):
    """The slots of topk_ids [T,k] sorted by expert, all int32: counts [E], x_rows [T*k] (the token of each sorted row, as
    moe_decode_matmul_fp8_experts takes it) and positions [T,k] (the sorted row of each slot, as moe_decode_combine takes
    it); -1 for slots of tokens that are not valid and for ids outside [0,E) (see include/moe_decode.h).  With no tokens
    nothing is written, counts neither.

    Without a workspace one is taken from torch's allocator for the call (which then runs on the current stream)."""
    L = _load()
    d = _gpu(topk_ids, "topk_ids")
    T, k = topk_ids.shape
    E = counts.shape[-1]
    ws, n, keep = _workspace(workspace, moe_decode_sort_slots_workspace(T, E, k), d, stream, "moe_decode_sort_slots")
    _call("moe_decode_sort_slots", L.moe_decode_sort_slots, d, stream, _flat(topk_ids, "topk_ids", d, (T, k), _i32),
          None if valid is None else _flat(valid, "valid", d, T, _flags), _flat(counts, "counts", d, E, _i32),
          _flat(x_rows, "x_rows", d, T * k, _i32), _flat(positions, "positions", d, (T, k), _i32), ws, n, T, E, k)
    return counts, x_rows, positions


def moe_decode_combine(rows, positions, weights, y, add=None, stream=None):
    """y [T,N] = add + sum_j weights[:,j] * rows[positions[:,j]] of rows [M,N] (fp32, bf16 or fp16), positions int32 [T,k];
    weights fp32 [T,k] or None (1); add may be y (see include/moe_decode.h)."""
    L = _load()
    d = _gpu(rows, "rows")
    M, N = rows.shape
    T, k = positions.shape
    t = rows.dtype
    dt = _dtype_code(rows, "rows", (MOE_F32, MOE_BF16, MOE_F16))
    _call("moe_decode_combine", L.moe_decode_combine, d, stream, *_mat(rows, "rows", d, t, M, N), dt,
          _flat(positions, "positions", d, (T, k), _i32),
          None if weights is None else _flat(weights, "weights", d, (T, k), _f32),
          *((None, 0) if add is None else _mat(add, "add", d, t, T, N)), *_mat(y, "y", d, t, T, N), M, T, N, k)
    return y


def moe_decode_combine_backward(dy, rows, positions, weights, drows, dweights, stream=None):
    """drows [M,N] (rows that no slot names stay as they were) and dweights fp32 [T,k], the gradients of
    moe_decode_combine from dy [T,N]; without dweights (None) rows may be None too (see include/moe_decode.h)."""
    L = _load()
    d = _gpu(dy, "dy")
    T, N = dy.shape
    M, k = drows.shape[0], positions.shape[-1]
    t = dy.dtype
    dt = _dtype_code(dy, "dy", (MOE_F32, MOE_BF16, MOE_F16))
    if dweights is not None and rows is None:
        raise ValueError("dweights need rows")
    _call("moe_decode_combine_backward", L.moe_decode_combine_backward, d, stream, *_mat(dy, "dy", d, t, T, N),
          *((None, 0) if rows is None else _mat(rows, "rows", d, t, M, N)), dt, _flat(positions, "positions", d, (T, k), _i32),
          None if weights is None else _flat(weights, "weights", d, (T, k), _f32), *_mat(drows, "drows", d, t, M, N),
          None if dweights is None else _flat(dweights, "dweights", d, (T, k), _f32), M, T, N, k)
    return drows, dweights


def moe_decode_rms_norm(x, weight, eps, y=None, q=None, scales=None, residual=None, sum_out=None, rstd=None, pow2=False,
                        stream=None):
    """The root-mean-square norm of x [M,H] (+ residual) times weight [H] (x's type or fp32): y [M,H], and / or q [M,H]
    E4M3 codes (uint8) with scales fp32 [M, ceil(H/128)]; sum_out [M,H]: x + residual (it may be the residual); rstd
    fp32 [M] (see include/moe_decode.h).  Returns (y, q, scales, sum_out, rstd), None where none was given."""
    L = _load()
    d = _gpu(x, "x")
    M, H = x.shape
    t = x.dtype
    dt = _dtype_code(x, "x", (MOE_F32, MOE_BF16, MOE_F16))
    xp, xl = _mat(x, "x", d, t, M, H)
    rp, rl = (None, 0) if residual is None else _mat(residual, "residual", d, t, M, H)
    yp, yl = (None, 0) if y is None else _mat(y, "y", d, t, M, H)
    sp, sl = (None, 0) if sum_out is None else _mat(sum_out, "sum_out", d, t, M, H)
    _call("moe_decode_rms_norm", L.moe_decode_rms_norm, d, stream, xp, xl, rp, rl, dt,
          _flat(weight, "weight", d, (H,), weight.dtype), dt if weight.dtype is t else _dtype_code(weight, "weight", (MOE_F32, dt)),
          eps, yp, yl, None if q is None else _flat(q, "q", d, (M, H), _u8),
          None if scales is None else _flat(scales, "scales", d, (M, -(-H // 128)), _f32), sp, sl,
          None if rstd is None else _flat(rstd, "rstd", d, (M,), _f32), M, H, MOE_QUANT_POW2 if pow2 else 0)
    return y, q, scales, sum_out, rstd


@functools.lru_cache(maxsize=256)
def moe_decode_rms_norm_backward_workspace(M, H):
    """Bytes of device workspace moe_decode_rms_norm_backward needs."""
    n = ctypes.c_size_t()
    rc = lib().moe_decode_rms_norm_backward_workspace(M, H, ctypes.byref(n))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_rms_norm_backward_workspace")
    return n.value


def moe_decode_rms_norm_backward(dy, r, weight, rstd, dx, dweight, dsum=None, workspace=None, stream=None):
    """dx [M,H] (the gradient of x and of the residual) and dweight fp32 [H] of moe_decode_rms_norm from dy [M,H], r (its
    sum_out, or x where it had no residual) and rstd; dsum [M,H]: the gradient that reaches sum_out from elsewhere, which
    may be dx (see include/moe_decode.h).  With no rows nothing is written, dweight neither.

    Without a workspace one is taken from torch's allocator for the call (which then runs on the current stream)."""
    L = _load()
    d = _gpu(dy, "dy")
    M, H = dy.shape
    t = dy.dtype
    dt = _dtype_code(dy, "dy", (MOE_F32, MOE_BF16, MOE_F16))
    gp, gl = _mat(dy, "dy", d, t, M, H)
    rp, rl = _mat(r, "r", d, t, M, H)
    sp, sl = (None, 0) if dsum is None else _mat(dsum, "dsum", d, t, M, H)
    xp, xl = _mat(dx, "dx", d, t, M, H)
    ws, n, keep = _workspace(workspace, moe_decode_rms_norm_backward_workspace(M, H) if M else 0, d, stream,
                             "moe_decode_rms_norm_backward")
    _call("moe_decode_rms_norm_backward", L.moe_decode_rms_norm_backward, d, stream, gp, gl, rp, rl, dt,
          _flat(weight, "weight", d, (H,), weight.dtype), dt if weight.dtype is t else _dtype_code(weight, "weight", (MOE_F32, dt)),
          _flat(rstd, "rstd", d, (M,), _f32), sp, sl, xp, xl, _flat(dweight, "dweight", d, (H,), _f32), ws, n, M, H)
    return dx, dweight


@functools.lru_cache(maxsize=256)
def moe_decode_adapters_workspace(M, K, N, R, L):
    """Bytes of device workspace moe_decode_adapters needs."""
    n = ctypes.c_size_t()
    rc = lib().moe_decode_adapters_workspace(M, K, N, R, L, ctypes.byref(n))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_adapters_workspace")
    return n.value


def moe_decode_adapters(x, row_adapters, a, b, scaling, y, base=None, workspace=None, stream=None):
    """y [M,N] = base + scaling[l] * (x a[l]^T) b[l]^T for each row's adapter l = row_adapters[m] (int32; outside [0,L):
    none), x [M,K], a [L,R,K], b [L,N,R] (bf16 or fp16), scaling fp32 [L]; base [M,N] or None (0), which may be y (see
    include/moe_decode.h).

    Without a workspace one is taken from torch's allocator for the call (which then runs on the current stream)."""
    lb = _load()
    d = _gpu(x, "x")
    M, K = x.shape
    L, R, _ = a.shape
    N = b.shape[1]
    t = x.dtype
    dt = _dtype_code(x, "x", (MOE_BF16, MOE_F16))
    xp, xl = _mat(x, "x", d, t, M, K)
    bp, bl = (None, 0) if base is None else _mat(base, "base", d, t, M, N)
    yp, yl = _mat(y, "y", d, t, M, N)
    ws, n, keep = _workspace(workspace, moe_decode_adapters_workspace(M, K, N, R, L), d, stream, "moe_decode_adapters")
    for m, name in ((a, "a"), (b, "b")):
        if m.dtype is not t and _codes.get(m.dtype) != dt:
            raise ValueError(f"{name} must have the type of x")
    _call("moe_decode_adapters", lb.moe_decode_adapters, d, stream, xp, xl, dt, _flat(row_adapters, "row_adapters", d, M, _i32),
          _flat(a, "a", d, (L, R, K), a.dtype), _flat(b, "b", d, (L, N, R), b.dtype), _flat(scaling, "scaling", d, (L,), _f32),
          bp, bl, yp, yl, ws, n, M, K, N, R, L)
    return y


def moe_decode_copy_peak(src, dst, stream=None):
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() < n:
        raise ValueError("dst smaller than src")
    rc = lib().moe_decode_copy_peak(_dev(src, "src"), _dev(dst, "dst"), n, _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_copy_peak")


def moe_decode_read_peak(src, sink, stream=None):
    n = src.numel() * src.element_size()
    if sink.numel() * sink.element_size() < 4:
        raise ValueError("sink needs 4 bytes")
    rc = lib().moe_decode_read_peak(_dev(src, "src"), n, _dev(sink, "sink"), _stream(stream))
    if rc:
        raise MoeDecodeError(rc, "moe_decode_read_peak")
