"""ctypes binding of libqpl.so: argument marshalling only.

Every call forwards raw device pointers, sizes and the current HIP stream to the
C ABI declared in include/qpl.h; all arithmetic runs in the library's gfx950
kernels.  torch is used for device memory and streams only.  There is no CPU
fallback: a missing library or a non-OK status raises.
"""
import ctypes
import os
import struct

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqpl.so")

QPL_FP8R = 0
QPL_NVFP4 = 1
QPL_INT4 = 2
QPL_INT8 = 3
QPL_FP8B = 4

EXPORTS = ("quant_act_fp8_row", "quant_act_nvfp4", "qlinear_fp8r", "qlinear_nvfp4", "dequant_weight",
           "quant_weight_awq", "qlinear_awq_w4a16", "quant_act_int4", "qlinear_int4", "qlinear_fp8r_ex",
           "qlinear_nvfp4_ex", "qlinear_int4_ex", "qlinear_mlp_nvfp4", "qlinear_mlp_nvfp4_workspace_bytes",
           "qlinear_workspace_bytes", "qpl_amax_bf16", "qpl_nvfp4_global_scale", "qpl_status_str",
           "qpl_timing_enable", "qpl_timing_select", "qpl_timing_collect", "qpl_timing_collect_n", "qlinear_fp8r_noalloc",
           "quant_act_int8", "qlinear_int8", "qlinear_int8_ex", "expert_plan", "expert_plan_workspace_bytes",
           "qlinear_grouped_int8",
           "qlinear_grouped_int8_workspace_bytes", "expert_combine", "qlinear_moe_int8",
           "qlinear_moe_int8_workspace_bytes", "quant_act_fp8b", "quant_weight_fp8b", "transpose_fp8b", "qlinear_fp8b",
           "qlinear_fp8b_ex", "qlinear_gated_fp8b", "qlinear_gated_fp8b_workspace_bytes",
           "qlinear_gated_fp8b_backward", "qlinear_gated_fp8b_backward_workspace_bytes", "qlinear_weight_grad",
           "qk_norm_rope", "qk_norm_rope_backward", "qk_norm_rope_backward_workspace_bytes", "qpl_rope_frequencies")

# qpl_kernel order of include/qpl.h
KERNELS = ("quant_fp8_row", "quant_nvfp4", "quant_nvfp4_linear", "gemm_fp8r", "gemm_nvfp4", "gemm_nvfp4_lowrank",
           "lowrank_prep", "dequant", "amax", "nvfp4_prep", "quant_nvfp4_lowrank", "quant_w4g", "gemv_w4a16",
           "quant_int4", "int4_expand", "gemm_int4", "quant_int4_lowrank", "gemm_epilogue", "quant_int8", "gemm_int8",
           "gemm_int8_grouped", "expert_plan", "expert_combine", "quant_fp8b", "gemm_fp8b", "gated_fp8b",
           "gated_backward", "transpose_fp8b", "weight_grad", "qk_norm_rope")

QPL_ACT_NONE = 0
QPL_ACT_GELU_TANH = 1
QPL_ACT_SILU = 2
_ACTS = {None: QPL_ACT_NONE, "none": QPL_ACT_NONE, "gelu_tanh": QPL_ACT_GELU_TANH}

_GATED_ACTS = {"silu": QPL_ACT_SILU, "gelu_tanh": QPL_ACT_GELU_TANH}

_P, _I64, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float


class Epilogue(ctypes.Structure):
    """qpl_epilogue of include/qpl.h."""
    _fields_ = [("act", ctypes.c_int), ("q", _P), ("k", _P), ("v", _P), ("heads", _I64), ("head_dim", _I64),
                ("tokens", _I64), ("token_offset", _I64)]


class Nvfp4Layer(ctypes.Structure):
    """qpl_nvfp4_layer of include/qpl.h."""
    _fields_ = [("weight", _P), ("weight_scale", _P), ("weight_scale_2", _F), ("input_scale", _F),
                ("smooth", _P), ("lora_down", _P), ("lora_up", _P), ("R", _I64)]


class Fp8bWeight(ctypes.Structure):
    """qpl_fp8b_weight of include/qpl.h."""
    _fields_ = [("weight", _P), ("weight_scale", _P)]


class Heads(ctypes.Structure):
    """qpl_heads of include/qpl.h."""
    _fields_ = [("x", _P), ("y", _P), ("heads", _I64), ("x_head_stride", _I64), ("x_token_stride", _I64),
                ("y_head_stride", _I64), ("y_token_stride", _I64), ("weight", _P), ("dx", _P),
                ("dx_head_stride", _I64), ("dx_token_stride", _I64), ("dweight", _P)]


class Rope(ctypes.Structure):
    """qpl_rope of include/qpl.h."""
    _fields_ = [("positions", _P), ("inv_freq", _P), ("rotary_dim", _I64), ("axes", _I64), ("sections", _I64 * 4),
                ("interleaved", ctypes.c_int), ("scale", _F)]


class RopeScaling(ctypes.Structure):
    """qpl_rope_scaling of include/qpl.h."""
    _fields_ = [("kind", ctypes.c_int), ("factor", ctypes.c_double), ("trained_tokens", ctypes.c_double),
                ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double)]


_lib = None


class QPLError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def load():
    """Load libqpl.so (once) and declare the signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m precision_quantized_linear_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sig = {
        "quant_act_fp8_row": [P, I64, I64, P, P, P],
        "quant_act_nvfp4": [P, I64, I64, F, P, P, P, P],
        "qlinear_fp8r": [P, I64, I64, I64, P, P, P, P, SZ, P],
        "qlinear_nvfp4": [P, I64, I64, I64, P, P, F, F, P, P, P, I64, P, P, SZ, P],
        "dequant_weight": [ctypes.c_int, P, P, F, I64, I64, P, P],
        "quant_weight_awq": [P, I64, I64, I64, P, P, P, P],
        "qlinear_awq_w4a16": [P, I64, I64, I64, P, P, P, I64, P, P],
        "quant_act_int4": [P, I64, I64, P, P, P, P],
        "qlinear_int4": [P, I64, I64, I64, P, P, P, P, P, I64, P, P, SZ, P],
        "qpl_amax_bf16": [P, I64, P, P],
        "qlinear_fp8r_ex": [P, I64, I64, I64, P, P, P, P, P, SZ, P],
        "qlinear_nvfp4_ex": [P, I64, I64, I64, P, P, F, F, P, P, P, I64, P, P, P, SZ, P],
        "qlinear_int4_ex": [P, I64, I64, I64, P, P, P, P, P, I64, P, P, P, SZ, P],
        "qlinear_mlp_nvfp4": [P, I64, I64, I64, I64, P, P, P, P, SZ, P],
        "qlinear_fp8r_noalloc": [P, I64, I64, I64, P, P, P, P],
        "quant_act_int8": [P, I64, I64, P, P, P, P],
        "qlinear_int8": [P, I64, I64, I64, P, P, P, P, P, SZ, P],
        "qlinear_int8_ex": [P, I64, I64, I64, P, P, P, P, P, P, SZ, P],
        "expert_plan": [P, I64, I64, I64, P, P, P, P, SZ, P],
        "qlinear_grouped_int8": [P, I64, I64, I64, I64, P, P, P, I64, P, ctypes.c_int, P, P, SZ, P],
        "expert_combine": [P, I64, I64, P, P, I64, I64, P, P],
        "qlinear_moe_int8": [P, I64, I64, I64, I64, I64, I64, P, P, P, P, P, P, P, P, SZ, P],
        "quant_act_fp8b": [P, I64, I64, P, P, P],
        "quant_weight_fp8b": [P, I64, I64, P, P, P],
        "transpose_fp8b": [P, P, I64, I64, P, P, P],
        "qlinear_fp8b": [P, I64, I64, I64, P, P, P, P, SZ, P],
        "qlinear_fp8b_ex": [P, I64, I64, I64, P, P, P, P, P, SZ, P],
        "qlinear_gated_fp8b": [P, I64, I64, I64, P, P, ctypes.c_int, P, P, P, P, SZ, P],
        "qlinear_gated_fp8b_backward": [P, P, P, I64, I64, I64, P, P, ctypes.c_int, P, P, P, P, SZ, P],
        "qlinear_weight_grad": [P, P, I64, I64, I64, P, P],
        "qk_norm_rope": [P, P, I64, I64, ctypes.c_int, F, P, P],
        "qk_norm_rope_backward": [P, P, I64, I64, ctypes.c_int, F, P, P, SZ, P],
        "qpl_rope_frequencies": [I64, ctypes.c_double, P, P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.qlinear_workspace_bytes.argtypes = [ctypes.c_int, I64, I64, I64, I64]
    lib.qlinear_workspace_bytes.restype = SZ
    lib.qlinear_mlp_nvfp4_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I64]
    lib.qlinear_mlp_nvfp4_workspace_bytes.restype = SZ
    lib.expert_plan_workspace_bytes.argtypes = [I64, I64, I64]
    lib.expert_plan_workspace_bytes.restype = SZ
    lib.qlinear_grouped_int8_workspace_bytes.argtypes = [I64, I64, I64, I64]
    lib.qlinear_grouped_int8_workspace_bytes.restype = SZ
    lib.qlinear_moe_int8_workspace_bytes.argtypes = [I64, I64, I64, I64, I64, I64]
    lib.qlinear_moe_int8_workspace_bytes.restype = SZ
    lib.qlinear_gated_fp8b_workspace_bytes.argtypes = [I64, I64, I64]
    lib.qlinear_gated_fp8b_workspace_bytes.restype = SZ
    lib.qlinear_gated_fp8b_backward_workspace_bytes.argtypes = [I64, I64, I64]
    lib.qlinear_gated_fp8b_backward_workspace_bytes.restype = SZ
    lib.qk_norm_rope_backward_workspace_bytes.argtypes = [I64, I64]
    lib.qk_norm_rope_backward_workspace_bytes.restype = SZ
    lib.qpl_nvfp4_global_scale.argtypes = [F]
    lib.qpl_nvfp4_global_scale.restype = F
    lib.qpl_status_str.argtypes = [ctypes.c_int]
    lib.qpl_status_str.restype = ctypes.c_char_p
    lib.qpl_timing_enable.argtypes = [ctypes.c_int]
    lib.qpl_timing_enable.restype = None
    lib.qpl_timing_select.argtypes = [ctypes.c_uint32]
    lib.qpl_timing_select.restype = None
    lib.qpl_timing_collect.argtypes = [P, P]
    lib.qpl_timing_collect.restype = ctypes.c_int
    lib.qpl_timing_collect_n.argtypes = [P, P, ctypes.c_int]
    lib.qpl_timing_collect_n.restype = ctypes.c_int
    _lib = lib
    return lib


def _check(fn, status):
    if status != 0:
        raise QPLError(fn, status, load().qpl_status_str(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _expect(t, dtype, shape, name):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on a GPU, got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} device={t.device}")


def _bits(t):
    """bf16 tensor -> same storage viewed as int16 (the C ABI takes the bit patterns)."""
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def quant_act_fp8_row(x, x_q=None, x_scale=None, stream=None):
    """bf16 [M,K] -> (E4M3 codes uint8 [M,K], fp32 row scales [M])."""
    M, K = x.shape
    _expect(x, torch.bfloat16, (M, K), "x")
    x_q = torch.empty((M, K), dtype=torch.uint8, device=x.device) if x_q is None else x_q
    x_scale = torch.empty((M,), dtype=torch.float32, device=x.device) if x_scale is None else x_scale
    _check("quant_act_fp8_row", load().quant_act_fp8_row(_ptr(x), M, K, _ptr(x_q), _ptr(x_scale), _stream(stream)))
    return x_q, x_scale


def quant_act_nvfp4(x, input_scale, smooth=None, x_q=None, x_block_scale=None, stream=None):
    """bf16 [M,K] -> (packed E2M1 uint8 [M,K/2], E4M3 block scales uint8 [M,K/16]);
    with smooth (float32 [K]) the quantized activation is bf16(x / smooth)."""
    M, K = x.shape
    _expect(x, torch.bfloat16, (M, K), "x")
    if smooth is not None:
        _expect(smooth, torch.float32, (K,), "smooth")
    x_q = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device) if x_q is None else x_q
    x_block_scale = (torch.empty((M, K // 16), dtype=torch.uint8, device=x.device)
                     if x_block_scale is None else x_block_scale)
    _check("quant_act_nvfp4", load().quant_act_nvfp4(_ptr(x), M, K, float(input_scale), _ptr(smooth), _ptr(x_q),
                                                      _ptr(x_block_scale), _stream(stream)))
    return x_q, x_block_scale


def qlinear_workspace_bytes(scheme, M, K, N, R=0):
    return int(load().qlinear_workspace_bytes(scheme, M, K, N, R))


def _workspace(scheme, M, K, N, R, ws, device):
    need = qlinear_workspace_bytes(scheme, M, K, N, R)
    if ws is None:
        ws = torch.empty((max(need, 1),), dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def _epilogue(act, qkv, M, N, y, device):
    """(Epilogue or None, y, result): act names the activation ("gelu_tanh"); qkv is
    (q, k, v, token_offset) with q, k, v bf16 [heads, tokens, head_dim]."""
    if act not in _ACTS:
        raise ValueError(f"act: expected one of {sorted(k for k in _ACTS if k)}, got {act!r}")
    if act is None and qkv is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=device) if y is None else y
        return None, y, y
    e = Epilogue()
    e.act = _ACTS[act]
    if qkv is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=device) if y is None else y
        return e, y, y
    q, k, v, off = qkv
    heads, tokens, head_dim = q.shape
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        _expect(t, torch.bfloat16, (heads, tokens, head_dim), name)
    e.q, e.k, e.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    e.heads, e.head_dim, e.tokens, e.token_offset = heads, head_dim, tokens, int(off)
    return e, None, (q, k, v)


def _ref(e):
    return None if e is None else ctypes.byref(e)


def qlinear_fp8r(x, weight, weight_scale, y=None, workspace=None, stream=None, act=None, qkv=None):
    """y[M,N] bf16 = fp8r linear of bf16 x [M,K] with E4M3 weight [N,K] and fp32 weight_scale [N].
    act="gelu_tanh" applies GELU before the rounding; qkv=(q, k, v, token_offset) writes the
    three column parts to q, k, v [heads, tokens, head_dim] instead (and returns them)."""
    M, K = x.shape
    N = weight.shape[0]
    _expect(x, torch.bfloat16, (M, K), "x")
    _expect(weight, torch.uint8, (N, K), "weight")
    _expect(weight_scale, torch.float32, (N,), "weight_scale")
    e, y, out = _epilogue(act, qkv, M, N, y, x.device)
    ws, nbytes = _workspace(QPL_FP8R, M, K, N, 0, workspace, x.device)
    if e is None:
        _check("qlinear_fp8r", load().qlinear_fp8r(_ptr(x), M, K, N, _ptr(weight), _ptr(weight_scale), _ptr(y),
                                                   _ptr(ws), nbytes, _stream(stream)))
    else:
        _check("qlinear_fp8r_ex", load().qlinear_fp8r_ex(_ptr(x), M, K, N, _ptr(weight), _ptr(weight_scale),
                                                         _ref(e), _ptr(y), _ptr(ws), nbytes, _stream(stream)))
    return out


def qlinear_fp8r_noalloc(x, weight, weight_scale, y, stream=None):
    """qlinear_fp8r into a caller-provided y [M,N] bf16 with the library's static
    device scratch as workspace: the call itself allocates nothing."""
    M, K = x.shape
    N = weight.shape[0]
    _expect(x, torch.bfloat16, (M, K), "x")
    _expect(weight, torch.uint8, (N, K), "weight")
    _expect(weight_scale, torch.float32, (N,), "weight_scale")
    _expect(y, torch.bfloat16, (M, N), "y")
    _check("qlinear_fp8r_noalloc", load().qlinear_fp8r_noalloc(_ptr(x), M, K, N, _ptr(weight), _ptr(weight_scale),
                                                               _ptr(y), _stream(stream)))
    return y


def qlinear_nvfp4(x, weight, weight_scale, weight_scale_2, input_scale, lora_down=None, lora_up=None, y=None,
                  workspace=None, stream=None, smooth=None, act=None, qkv=None):
    """y[M,N] bf16 = nvfp4 linear (+ (x L1) L2 when lora_down [K,R] / lora_up [R,N] are given);
    with smooth (float32 [K]) both terms take the smoothed activation bf16(x / smooth).
    act and qkv as in qlinear_fp8r."""
    M, K = x.shape
    N = weight.shape[0]
    _expect(x, torch.bfloat16, (M, K), "x")
    if smooth is not None:
        _expect(smooth, torch.float32, (K,), "smooth")
    _expect(weight, torch.uint8, (N, K // 2), "weight")
    _expect(weight_scale, torch.uint8, (N, K // 16), "weight_scale")
    R = 0
    if lora_down is not None:
        R = lora_down.shape[1]
        _expect(lora_down, torch.bfloat16, (K, R), "lora_down")
        _expect(lora_up, torch.bfloat16, (R, N), "lora_up")
    e, y, out = _epilogue(act, qkv, M, N, y, x.device)
    ws, nbytes = _workspace(QPL_NVFP4, M, K, N, R, workspace, x.device)
    args = (_ptr(x), M, K, N, _ptr(weight), _ptr(weight_scale), float(weight_scale_2), float(input_scale),
            _ptr(smooth), _ptr(lora_down), _ptr(lora_up), R)
    if e is None:
        _check("qlinear_nvfp4", load().qlinear_nvfp4(*args, _ptr(y), _ptr(ws), nbytes, _stream(stream)))
    else:
        _check("qlinear_nvfp4_ex", load().qlinear_nvfp4_ex(*args, _ref(e), _ptr(y), _ptr(ws), nbytes,
                                                           _stream(stream)))
    return out


def quant_act_int4(x, smooth=None, x_q=None, x_scale=None, stream=None):
    """bf16 [M,K] (K % 64 == 0) -> (packed INT4 codes uint8 [M,K/2], fp32 group scales [M,K/64])."""
    M, K = x.shape
    _expect(x, torch.bfloat16, (M, K), "x")
    if smooth is not None:
        _expect(smooth, torch.float32, (K,), "smooth")
    x_q = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device) if x_q is None else x_q
    x_scale = torch.empty((M, K // 64), dtype=torch.float32, device=x.device) if x_scale is None else x_scale
    _check("quant_act_int4", load().quant_act_int4(_ptr(x), M, K, _ptr(smooth), _ptr(x_q), _ptr(x_scale),
                                                    _stream(stream)))
    return x_q, x_scale


def qlinear_int4(x, weight, weight_scale, lora_down=None, lora_up=None, y=None, workspace=None, stream=None,
                 smooth=None, act=None, qkv=None):
    """y[M,N] bf16 = INT4 W4A4 linear (+ (x L1) L2), the INT4 variant of svdq_w4a4; act and
    qkv as in qlinear_fp8r."""
    M, K = x.shape
    N = weight.shape[0]
    _expect(x, torch.bfloat16, (M, K), "x")
    _expect(weight, torch.uint8, (N, K // 2), "weight")
    _expect(weight_scale, torch.float32, (N, K // 64), "weight_scale")
    if smooth is not None:
        _expect(smooth, torch.float32, (K,), "smooth")
    R = 0
    if lora_down is not None:
        R = lora_down.shape[1]
        _expect(lora_down, torch.bfloat16, (K, R), "lora_down")
        _expect(lora_up, torch.bfloat16, (R, N), "lora_up")
    e, y, out = _epilogue(act, qkv, M, N, y, x.device)
    ws, nbytes = _workspace(QPL_INT4, M, K, N, R, workspace, x.device)
    args = (_ptr(x), M, K, N, _ptr(weight), _ptr(weight_scale), _ptr(smooth), _ptr(lora_down), _ptr(lora_up), R)
    if e is None:
        _check("qlinear_int4", load().qlinear_int4(*args, _ptr(y), _ptr(ws), nbytes, _stream(stream)))
    else:
        _check("qlinear_int4_ex", load().qlinear_int4_ex(*args, _ref(e), _ptr(y), _ptr(ws), nbytes,
                                                         _stream(stream)))
    return out


def qlinear_mlp_nvfp4_workspace_bytes(M, K, H, N, R1=0, R2=0):
    return int(load().qlinear_mlp_nvfp4_workspace_bytes(M, K, H, N, R1, R2))


def _layer(d, rows, cols, name):
    """Nvfp4Layer from a dict with weight [rows, cols/2], weight_scale [rows, cols/16],
    weight_scale_2, input_scale and optional smooth [cols], lora_down [cols, R], lora_up [R, rows]."""
    _expect(d["weight"], torch.uint8, (rows, cols // 2), name + ".weight")
    _expect(d["weight_scale"], torch.uint8, (rows, cols // 16), name + ".weight_scale")
    L = Nvfp4Layer()
    L.weight, L.weight_scale = d["weight"].data_ptr(), d["weight_scale"].data_ptr()
    L.weight_scale_2, L.input_scale = float(d["weight_scale_2"]), float(d["input_scale"])
    if d.get("smooth") is not None:
        _expect(d["smooth"], torch.float32, (cols,), name + ".smooth")
        L.smooth = d["smooth"].data_ptr()
    if d.get("lora_down") is not None:
        R = d["lora_down"].shape[1]
        _expect(d["lora_down"], torch.bfloat16, (cols, R), name + ".lora_down")
        _expect(d["lora_up"], torch.bfloat16, (R, rows), name + ".lora_up")
        L.lora_down, L.lora_up, L.R = d["lora_down"].data_ptr(), d["lora_up"].data_ptr(), R
    return L


def qlinear_mlp_nvfp4(x, fc1, fc2, y=None, workspace=None, stream=None):
    """y [M,N] bf16 = fc2(bf16(gelu(fc1(x)))) for nvfp4 layers fc1 [H,K] and fc2 [N,H]
    given as dicts (see _layer); GELU runs in fc1's epilogue.  After the call the first
    2 M H bytes of the workspace hold fc2's expanded operand, and h follows fc2's part."""
    M, K = x.shape
    _expect(x, torch.bfloat16, (M, K), "x")
    H = fc1["weight"].shape[0]
    N = fc2["weight"].shape[0]
    l1, l2 = _layer(fc1, H, K, "fc1"), _layer(fc2, N, H, "fc2")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    need = qlinear_mlp_nvfp4_workspace_bytes(M, K, H, N, l1.R, l2.R)
    ws = torch.empty((max(need, 1),), dtype=torch.uint8, device=x.device) if workspace is None else workspace
    _check("qlinear_mlp_nvfp4", load().qlinear_mlp_nvfp4(_ptr(x), M, K, H, N, ctypes.byref(l1), ctypes.byref(l2),
                                                         _ptr(y), _ptr(ws), ws.numel() * ws.element_size(),
                                                         _stream(stream)))
    return y


def _addr(t, dtype, shape, dev, name):
    """Address of t, checked: contiguous, of this type and shape, on GPU dev (None: 0)."""
    if t is None:
        return 0
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on the current GPU ({dev}), got "
                         f"{t.dtype} {tuple(t.shape)} contiguous={t.is_contiguous()} device={t.device}")
    return t.data_ptr()


def _current(t, dims, name):
    """The current GPU, which has to be t's: a call runs on it and reads all its tensors there."""
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got {tuple(t.shape)}")
    dev = t.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError(f"{name}: expected a tensor on the current GPU, got {t.device}")
    return dev


def _dims(t, n, name):
    if t.dim() != n:
        raise ValueError(f"{name}: expected {n} dimensions, got {tuple(t.shape)}")
    return t.shape


def _queue(stream, dev):
    """The hipStream_t of a call on GPU dev."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device_index != dev:
        raise ValueError(f"stream: expected a stream of the current GPU ({dev}), got one of {stream.device_index}")
    return stream.cuda_stream


def _new(shape, dtype, like, stream):
    """A tensor on like's GPU that belongs to the stream the call runs on."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _scratch(ws, need, like, dev, stream):
    """(workspace, its address, its bytes): the caller's, or a new one if any is needed (need is 0 too
    for sizes that the call refuses)."""
    if ws is None:
        if need == 0:
            return None, 0, 0
        ws = _new((need,), torch.uint8, like, stream)
        return ws, ws.data_ptr(), need
    if not ws.is_contiguous() or ws.get_device() != dev:
        raise ValueError(f"workspace: expected a contiguous tensor on the current GPU ({dev}), got {ws.device}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _act_code(act):
    if act not in _ACTS:
        raise ValueError(f"act: expected one of {sorted(k for k in _ACTS if k)}, got {act!r}")
    return _ACTS[act]


def quant_act_int8(x, smooth=None, x_q=None, x_scale=None, stream=None):
    """bf16 [M,K] -> (int8 codes [M,K], fp32 row scales [M]); with smooth (float32 [K]) the
    quantized activation is bf16(x / smooth).  The same call quantizes a weight [N,K]."""
    dev = _current(x, 2, "x")
    M, K = x.shape
    x_q = _new((M, K), torch.int8, x, stream) if x_q is None else x_q
    x_scale = _new((M,), torch.float32, x, stream) if x_scale is None else x_scale
    _check("quant_act_int8", load().quant_act_int8(
        _addr(x, torch.bfloat16, (M, K), dev, "x"), M, K, _addr(smooth, torch.float32, (K,), dev, "smooth"),
        _addr(x_q, torch.int8, (M, K), dev, "x_q"), _addr(x_scale, torch.float32, (M,), dev, "x_scale"),
        _queue(stream, dev)))
    return x_q, x_scale


def qlinear_int8(x, weight, weight_scale, y=None, workspace=None, stream=None, smooth=None, act=None, qkv=None):
    """y[M,N] bf16 = 8-bit integer linear of bf16 x [M,K] with int8 weight [N,K] and fp32
    weight_scale [N]; smooth, act and qkv as in qlinear_int4."""
    N = _dims(weight, 2, "weight")[0]
    dev = _current(x, 2, "x")
    M, K = x.shape
    args = (_addr(x, torch.bfloat16, (M, K), dev, "x"), M, K, N, _addr(weight, torch.int8, (N, K), dev, "weight"),
            _addr(weight_scale, torch.float32, (N,), dev, "weight_scale"),
            _addr(smooth, torch.float32, (K,), dev, "smooth"))
    act_code = _act_code(act)
    ya = 0
    if qkv is None:
        y = _new((M, N), torch.bfloat16, x, stream) if y is None else y
        ya = _addr(y, torch.bfloat16, (M, N), dev, "y")
    else:
        for t, name in zip(qkv[:3], ("q", "k", "v")):
            _addr(t, torch.bfloat16, _dims(qkv[0], 3, "q"), dev, name)
    ws, wa, nbytes = _scratch(workspace, qlinear_workspace_bytes(QPL_INT8, M, K, N), x, dev, stream)
    if act_code == QPL_ACT_NONE and qkv is None:
        _check("qlinear_int8", load().qlinear_int8(*args, ya, wa, nbytes, _queue(stream, dev)))
        return y
    e, _, out = _epilogue(act, qkv, M, N, y, x.device)
    _check("qlinear_int8_ex", load().qlinear_int8_ex(*args, _ref(e), ya, wa, nbytes, _queue(stream, dev)))
    return out


def expert_plan_workspace_bytes(T, topk, num_experts):
    return int(load().expert_plan_workspace_bytes(T, topk, num_experts))


def expert_plan(expert_ids, num_experts, row_index=None, slot=None, offsets=None, workspace=None, stream=None):
    """Router choices int32 [T, topk] sorted by expert -> (row_index int32 [T topk]: the token of
    each place; slot int32 [T, topk]: the place of each choice; offsets int32 [num_experts + 1]:
    the experts' first places).  An id outside [0, num_experts) gets slot -1; row_index is -1
    behind the last place."""
    dev = _current(expert_ids, 2, "expert_ids")
    T, topk = expert_ids.shape
    E = int(num_experts)
    if E < 1:
        raise ValueError(f"num_experts: expected at least 1, got {E}")
    row_index = _new((T * topk,), torch.int32, expert_ids, stream) if row_index is None else row_index
    slot = _new((T, topk), torch.int32, expert_ids, stream) if slot is None else slot
    offsets = _new((E + 1,), torch.int32, expert_ids, stream) if offsets is None else offsets
    ws, wa, nbytes = _scratch(workspace, expert_plan_workspace_bytes(T, topk, E), expert_ids, dev, stream)
    _check("expert_plan", load().expert_plan(
        _addr(expert_ids, torch.int32, (T, topk), dev, "expert_ids"), T, topk, E,
        _addr(row_index, torch.int32, (T * topk,), dev, "row_index"), _addr(slot, torch.int32, (T, topk), dev, "slot"),
        _addr(offsets, torch.int32, (E + 1,), dev, "offsets"), wa, nbytes, _queue(stream, dev)))
    return row_index, slot, offsets


def qlinear_grouped_int8_workspace_bytes(R, K, N, E):
    return int(load().qlinear_grouped_int8_workspace_bytes(R, K, N, E))


def qlinear_grouped_int8(x, weight, weight_scale, offsets, row_index=None, y=None, workspace=None, stream=None,
                         act=None):
    """y[R,N] bf16: rows offsets[e] .. offsets[e+1] - 1 are the 8-bit integer linear of
    x[row_index[i]] (bf16 [M,K]; x[i] without row_index, R = M) with expert e's int8 weight
    [E,N,K] and fp32 weight_scale [E,N].  offsets int32 [E + 1] and row_index int32 [R] stay on
    the GPU.  Rows of y in no expert's range are not written (a new y holds anything there)."""
    E, N, _ = _dims(weight, 3, "weight")
    dev = _current(x, 2, "x")
    M, K = x.shape
    R = M if row_index is None else _dims(row_index, 1, "row_index")[0]
    act_code = _act_code(act)
    y = _new((R, N), torch.bfloat16, x, stream) if y is None else y
    ws, wa, nbytes = _scratch(workspace, qlinear_grouped_int8_workspace_bytes(R, K, N, E), x, dev, stream)
    _check("qlinear_grouped_int8", load().qlinear_grouped_int8(
        _addr(x, torch.bfloat16, (M, K), dev, "x"), M, K, N, E, _addr(weight, torch.int8, (E, N, K), dev, "weight"),
        _addr(weight_scale, torch.float32, (E, N), dev, "weight_scale"),
        _addr(row_index, torch.int32, (R,), dev, "row_index"), R,
        _addr(offsets, torch.int32, (E + 1,), dev, "offsets"), act_code, _addr(y, torch.bfloat16, (R, N), dev, "y"),
        wa, nbytes, _queue(stream, dev)))
    return y


def expert_combine(y, slot, weights, out=None, stream=None):
    """out[t] bf16 [T,N] = sum_j weights[t,j] y[slot[t,j]] of bf16 y [R,N], int32 slot [T,topk] and
    fp32 weights [T,topk]; a slot outside [0, R) adds nothing."""
    T, topk = _dims(slot, 2, "slot")
    dev = _current(y, 2, "y")
    R, N = y.shape
    out = _new((T, N), torch.bfloat16, y, stream) if out is None else out
    _check("expert_combine", load().expert_combine(
        _addr(y, torch.bfloat16, (R, N), dev, "y"), R, N, _addr(slot, torch.int32, (T, topk), dev, "slot"),
        _addr(weights, torch.float32, (T, topk), dev, "weights"), T, topk,
        _addr(out, torch.bfloat16, (T, N), dev, "out"), _queue(stream, dev)))
    return out


def qlinear_moe_int8_workspace_bytes(T, topk, K, H, N, E):
    return int(load().qlinear_moe_int8_workspace_bytes(T, topk, K, H, N, E))


def qlinear_moe_int8(x, expert_ids, expert_weights, fc1, fc2, y=None, workspace=None, stream=None):
    """y [T,N] bf16 = sum_j expert_weights[t,j] fc2_e(bf16(gelu(fc1_e(x[t])))) over e = expert_ids[t,j]
    (int32 [T,topk]; an id outside the experts adds nothing); fc1 and fc2 are dicts with weight
    int8 [E,H,K] / [E,N,H] and weight_scale float32 [E,H] / [E,N]."""
    topk = _dims(expert_ids, 2, "expert_ids")[1]
    E, H, _ = _dims(fc1["weight"], 3, "fc1.weight")
    N = _dims(fc2["weight"], 3, "fc2.weight")[1]
    dev = _current(x, 2, "x")
    T, K = x.shape
    y = _new((T, N), torch.bfloat16, x, stream) if y is None else y
    ws, wa, nbytes = _scratch(workspace, qlinear_moe_int8_workspace_bytes(T, topk, K, H, N, E), x, dev, stream)
    _check("qlinear_moe_int8", load().qlinear_moe_int8(
        _addr(x, torch.bfloat16, (T, K), dev, "x"), T, K, H, N, E, topk,
        _addr(expert_ids, torch.int32, (T, topk), dev, "expert_ids"),
        _addr(expert_weights, torch.float32, (T, topk), dev, "expert_weights"),
        _addr(fc1["weight"], torch.int8, (E, H, K), dev, "fc1.weight"),
        _addr(fc1["weight_scale"], torch.float32, (E, H), dev, "fc1.weight_scale"),
        _addr(fc2["weight"], torch.int8, (E, N, H), dev, "fc2.weight"),
        _addr(fc2["weight_scale"], torch.float32, (E, N), dev, "fc2.weight_scale"),
        _addr(y, torch.bfloat16, (T, N), dev, "y"), wa, nbytes, _queue(stream, dev)))
    return y


# qpl_heads, qpl_rope and qpl_fp8b_weight as bytes (the layouts of Heads, Rope and Fp8bWeight): packing them takes a tenth of the
# time of building ctypes objects, which counts in calls that take a few microseconds.
_PACK_HEADS = struct.Struct("@PPqqqqqPPqqP").pack
_PACK_ROPE = struct.Struct("@PPqqqqqqif").pack
_PACK_WEIGHT = struct.Struct("@PP").pack


def _blocks(n):
    return (n + 127) // 128


def quant_act_fp8b(x, x_q=None, x_scale=None, stream=None):
    """bf16 [M,K] -> (E4M3 codes uint8 [M,K], fp32 scales [M, ceil(K/128)]), a scale for each 128 channels of a row."""
    dev = _current(x, 2, "x")
    M, K = x.shape
    x_q = _new((M, K), torch.uint8, x, stream) if x_q is None else x_q
    x_scale = _new((M, _blocks(K)), torch.float32, x, stream) if x_scale is None else x_scale
    _check("quant_act_fp8b", load().quant_act_fp8b(
        _addr(x, torch.bfloat16, (M, K), dev, "x"), M, K, _addr(x_q, torch.uint8, (M, K), dev, "x_q"),
        _addr(x_scale, torch.float32, (M, _blocks(K)), dev, "x_scale"), _queue(stream, dev)))
    return x_q, x_scale


def quant_weight_fp8b(w, w_q=None, w_scale=None, stream=None):
    """bf16 weight [N,K] -> (E4M3 codes uint8 [N,K], fp32 scales [ceil(N/128), ceil(K/128)])."""
    dev = _current(w, 2, "w")
    N, K = w.shape
    w_q = _new((N, K), torch.uint8, w, stream) if w_q is None else w_q
    w_scale = _new((_blocks(N), _blocks(K)), torch.float32, w, stream) if w_scale is None else w_scale
    _check("quant_weight_fp8b", load().quant_weight_fp8b(
        _addr(w, torch.bfloat16, (N, K), dev, "w"), N, K, _addr(w_q, torch.uint8, (N, K), dev, "w_q"),
        _addr(w_scale, torch.float32, (_blocks(N), _blocks(K)), dev, "w_scale"), _queue(stream, dev)))
    return w_q, w_scale


def transpose_fp8b(weight, weight_scale, weight_t=None, weight_t_scale=None, stream=None):
    """A quantized weight [N,K] turned over -> (uint8 [K,N], fp32 [ceil(K/128), ceil(N/128)]); N % 16 == 0.  The
    gradient of a linear's input is the linear of dy with it."""
    dev = _current(weight, 2, "weight")
    N, K = weight.shape
    weight_t = _new((K, N), torch.uint8, weight, stream) if weight_t is None else weight_t
    if weight_t_scale is None:
        weight_t_scale = _new((_blocks(K), _blocks(N)), torch.float32, weight, stream)
    _check("transpose_fp8b", load().transpose_fp8b(
        _addr(weight, torch.uint8, (N, K), dev, "weight"),
        _addr(weight_scale, torch.float32, (_blocks(N), _blocks(K)), dev, "weight_scale"), N, K,
        _addr(weight_t, torch.uint8, (K, N), dev, "weight_t"),
        _addr(weight_t_scale, torch.float32, (_blocks(K), _blocks(N)), dev, "weight_t_scale"), _queue(stream, dev)))
    return weight_t, weight_t_scale


def qlinear_fp8b(x, weight, weight_scale, y=None, workspace=None, stream=None, act=None, qkv=None):
    """y[M,N] bf16 = block-scaled fp8 linear of bf16 x [M,K] with E4M3 weight uint8 [N,K] and fp32 weight_scale
    [ceil(N/128), ceil(K/128)]; act and qkv as in qlinear_fp8r."""
    N = _dims(weight, 2, "weight")[0]
    dev = _current(x, 2, "x")
    M, K = x.shape
    args = (_addr(x, torch.bfloat16, (M, K), dev, "x"), M, K, N, _addr(weight, torch.uint8, (N, K), dev, "weight"),
            _addr(weight_scale, torch.float32, (_blocks(N), _blocks(K)), dev, "weight_scale"))
    act_code = _act_code(act)
    ya = 0
    if qkv is None:
        y = _new((M, N), torch.bfloat16, x, stream) if y is None else y
        ya = _addr(y, torch.bfloat16, (M, N), dev, "y")
    else:
        for t, name in zip(qkv[:3], ("q", "k", "v")):
            _addr(t, torch.bfloat16, _dims(qkv[0], 3, "q"), dev, name)
    ws, wa, nbytes = _scratch(workspace, qlinear_workspace_bytes(QPL_FP8B, M, K, N), x, dev, stream)
    if act_code == QPL_ACT_NONE and qkv is None:
        _check("qlinear_fp8b", load().qlinear_fp8b(*args, ya, wa, nbytes, _queue(stream, dev)))
        return y
    e, _, out = _epilogue(act, qkv, M, N, y, x.device)
    _check("qlinear_fp8b_ex", load().qlinear_fp8b_ex(*args, _ref(e), ya, wa, nbytes, _queue(stream, dev)))
    return out


def _gated_act(act):
    if act not in _GATED_ACTS:
        raise ValueError(f"act: expected one of {sorted(_GATED_ACTS)}, got {act!r}")
    return _GATED_ACTS[act]


def _fp8b_weight(layer, N, K, dev, name):
    """qpl_fp8b_weight, as bytes, of a dict with weight uint8 [N,K] and weight_scale float32 [ceil(N/128),
    ceil(K/128)]."""
    return _PACK_WEIGHT(_addr(layer["weight"], torch.uint8, (N, K), dev, name + ".weight"),
                        _addr(layer["weight_scale"], torch.float32, (_blocks(N), _blocks(K)), dev,
                              name + ".weight_scale"))


def qlinear_gated_fp8b_workspace_bytes(M, K, H):
    return int(load().qlinear_gated_fp8b_workspace_bytes(M, K, H))


def qlinear_gated_fp8b(x, gate, up, act="silu", h=None, save=False, workspace=None, stream=None):
    """h [M,H] bf16 = act(x Wg^T) * (x Wu^T) for block-scaled fp8 weights gate and up, dicts with weight uint8 [H,K]
    and weight_scale float32 [ceil(H/128), ceil(K/128)]; act "silu" or "gelu_tanh".  With save (True, or a pair of
    bf16 [M,H] tensors to write) the result is (h, g, u) with both projections, which the backward pass needs."""
    H = _dims(gate["weight"], 2, "gate.weight")[0]
    dev = _current(x, 2, "x")
    M, K = x.shape
    code = _gated_act(act)
    wg, wu = _fp8b_weight(gate, H, K, dev, "gate"), _fp8b_weight(up, H, K, dev, "up")
    h = _new((M, H), torch.bfloat16, x, stream) if h is None else h
    if save is True:
        save = (_new((M, H), torch.bfloat16, x, stream), _new((M, H), torch.bfloat16, x, stream))
    g, u = save if save else (None, None)
    ws, wa, nbytes = _scratch(workspace, qlinear_gated_fp8b_workspace_bytes(M, K, H), x, dev, stream)
    _check("qlinear_gated_fp8b", load().qlinear_gated_fp8b(
        _addr(x, torch.bfloat16, (M, K), dev, "x"), M, K, H, wg, wu, code,
        _addr(h, torch.bfloat16, (M, H), dev, "h"), _addr(g, torch.bfloat16, (M, H), dev, "g"),
        _addr(u, torch.bfloat16, (M, H), dev, "u"), wa, nbytes, _queue(stream, dev)))
    return (h, g, u) if save else h


def qlinear_gated_fp8b_backward_workspace_bytes(M, K, H):
    return int(load().qlinear_gated_fp8b_backward_workspace_bytes(M, K, H))


def qlinear_gated_fp8b_backward(dh, g, u, gate_t, up_t, act="silu", dx=None, dg=None, du=None, workspace=None,
                                stream=None):
    """(dx [M,K], dg [M,H], du [M,H]), all bf16, from dh and the saved g, u (bf16 [M,H]): the gradients of both
    projections, and of x through the weights turned over (dicts with what transpose_fp8b returns: weight uint8
    [K,H], weight_scale float32 [ceil(K/128), ceil(H/128)]).  The weights' gradients are
    qlinear_weight_grad(dg, x) and qlinear_weight_grad(du, x)."""
    K = _dims(gate_t["weight"], 2, "gate_t.weight")[0]
    dev = _current(dh, 2, "dh")
    M, H = dh.shape
    code = _gated_act(act)
    wg, wu = _fp8b_weight(gate_t, K, H, dev, "gate_t"), _fp8b_weight(up_t, K, H, dev, "up_t")
    dx = _new((M, K), torch.bfloat16, dh, stream) if dx is None else dx
    dg = _new((M, H), torch.bfloat16, dh, stream) if dg is None else dg
    du = _new((M, H), torch.bfloat16, dh, stream) if du is None else du
    ws, wa, nbytes = _scratch(workspace, qlinear_gated_fp8b_backward_workspace_bytes(M, K, H), dh, dev, stream)
    _check("qlinear_gated_fp8b_backward", load().qlinear_gated_fp8b_backward(
        _addr(dh, torch.bfloat16, (M, H), dev, "dh"), _addr(g, torch.bfloat16, (M, H), dev, "g"),
        _addr(u, torch.bfloat16, (M, H), dev, "u"), M, K, H, wg, wu, code,
        _addr(dx, torch.bfloat16, (M, K), dev, "dx"), _addr(dg, torch.bfloat16, (M, H), dev, "dg"),
        _addr(du, torch.bfloat16, (M, H), dev, "du"), wa, nbytes, _queue(stream, dev)))
    return dx, dg, du


def qlinear_weight_grad(dy, x, dw=None, stream=None):
    """dw [N,K] float32 = dy^T x of bf16 dy [M,N] and x [M,K]: the gradient of a linear's weight."""
    N = _dims(dy, 2, "dy")[1]
    dev = _current(x, 2, "x")
    M, K = x.shape
    dw = _new((N, K), torch.float32, x, stream) if dw is None else dw
    _check("qlinear_weight_grad", load().qlinear_weight_grad(
        _addr(dy, torch.bfloat16, (M, N), dev, "dy"), _addr(x, torch.bfloat16, (M, K), dev, "x"), M, N, K,
        _addr(dw, torch.float32, (N, K), dev, "dw"), _queue(stream, dev)))
    return dw


def _head_view(t, heads, tokens, dim, dev, name):
    """(address, head stride, token stride) of bf16 heads [heads, tokens, head_dim] whose channels are contiguous."""
    hs, ts, cs = t.stride()
    if t.dtype != torch.bfloat16 or t.shape != (heads, tokens, dim) or t.get_device() != dev or (cs != 1 and dim > 1):
        raise ValueError(f"{name}: expected torch.bfloat16 {(heads, tokens, dim)} with contiguous channels on the current "
                         f"GPU ({dev}), got {t.dtype} {tuple(t.shape)} strides={t.stride()} device={t.device}")
    # the stride of a single head or token is never used
    return t.data_ptr(), hs if heads > 1 else 0, ts if tokens > 1 else 0


def _new_heads(like, stream):
    """New heads in the order of `like`'s (token-major heads stay token-major)."""
    heads, tokens, dim = like.shape
    hs, ts, _ = like.stride()
    if tokens > 1 and heads > 1 and hs < ts:
        if stream is None:
            return like.new_empty_strided((heads, tokens, dim), (dim, heads * dim, 1))
        with torch.cuda.stream(stream):
            return like.new_empty_strided((heads, tokens, dim), (dim, heads * dim, 1))
    return _new((heads, tokens, dim), torch.bfloat16, like, stream)


def _rope(positions, inv_freq, tokens, interleaved, sections, scale, dev):
    """qpl_rope as bytes, or None for the norm alone."""
    if inv_freq is None:
        return None
    n = _dims(inv_freq, 1, "inv_freq")[0]
    if positions is None:
        raise ValueError("positions: needed with inv_freq")
    axes = 1 if sections is None else len(sections)
    if sections is not None and not 1 <= axes <= 4:
        raise ValueError(f"sections: expected one to four numbers of pairs, got {axes}")
    if sections is not None and axes == 1 and sections[0] != n:
        raise ValueError(f"sections: expected {n} pairs in all, got {tuple(sections)}")
    if axes > 1 and positions.dim() != 2:
        raise ValueError(f"positions: expected [tokens, {axes}] for {axes} sections, got {tuple(positions.shape)}")
    shape = (tokens, axes) if positions.dim() == 2 else (tokens,)
    parts = (n, 0, 0, 0) if sections is None else (tuple(int(v) for v in sections) + (0, 0, 0))[:4]
    return _PACK_ROPE(_addr(positions, torch.int32, shape, dev, "positions"),
                      _addr(inv_freq, torch.float32, (n,), dev, "inv_freq"), 2 * n, axes, *parts,
                      1 if interleaved else 0, scale)


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, norm=True, interleaved=False,
                 sections=None, scale=1.0, q_out=None, k_out=None, stream=None):
    """(q, k) normed per head and rotated by their positions, in one pass.  q and k: bf16 [heads, tokens, head_dim],
    channels contiguous, any strides of heads and tokens in multiples of 8 (token-major callers pass a transposed
    view); k may be None.  n = x * weight / sqrt(mean(x^2) + eps) over each head (norm False: as it is), then the
    first 2 len(inv_freq) channels turned by position * inv_freq[i], as pairs (i, i + half) or, interleaved,
    (2 i, 2 i + 1), times scale.  positions int32 [tokens], or [tokens, len(sections)] with sections pairs for each
    axis; inv_freq float32 (rope_frequencies), or None for the norm alone.  q_out and k_out may be q and k."""
    dev = _current(q, 3, "q")
    _, tokens, dim = q.shape
    r = _rope(positions, inv_freq, tokens, interleaved, sections, scale, dev)

    def side(t, w, o, name):
        heads = _dims(t, 3, name)[0]
        xa, xh, xt = _head_view(t, heads, tokens, dim, dev, name)
        if o is None:
            o = _new_heads(t, stream)
        ya, yh, yt = _head_view(o, heads, tokens, dim, dev, name + "_out")
        return o, _PACK_HEADS(xa, ya, heads, xh, xt, yh, yt, _addr(w, torch.bfloat16, (dim,), dev, name + "_weight"),
                              0, 0, 0, 0)

    q_out, qs = side(q, q_weight, q_out, "q")
    k_out, ks = (None, None) if k is None else side(k, k_weight, k_out, "k")
    _check("qk_norm_rope", load().qk_norm_rope(qs, ks, tokens, dim, 1 if norm else 0, eps, r, _queue(stream, dev)))
    return q_out, k_out


def qk_norm_rope_backward_workspace_bytes(tokens, head_dim):
    return int(load().qk_norm_rope_backward_workspace_bytes(tokens, head_dim))


def qk_norm_rope_backward(dq, dk, q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, norm=True,
                          interleaved=False, sections=None, scale=1.0, dq_out=None, dk_out=None, workspace=None,
                          stream=None):
    """Gradients (of q, of k, of q_weight, of k_weight) from those of qk_norm_rope's outputs and its inputs; the
    weights' in float32 [head_dim], None where there is no weight.  dq_out and dk_out may be dq and dk (or q and k)."""
    dev = _current(q, 3, "q")
    _, tokens, dim = q.shape
    r = _rope(positions, inv_freq, tokens, interleaved, sections, scale, dev)

    def side(d, t, w, o, name):
        heads = _dims(t, 3, name)[0]
        xa, xh, xt = _head_view(t, heads, tokens, dim, dev, name)
        da, dh, dt = _head_view(d, heads, tokens, dim, dev, "d" + name)
        if o is None:
            o = _new_heads(d, stream)
        oa, oh, ot = _head_view(o, heads, tokens, dim, dev, "d" + name + "_out")
        gw = None if w is None else _new((dim,), torch.float32, t, stream)
        return o, gw, _PACK_HEADS(xa, da, heads, xh, xt, dh, dt, _addr(w, torch.bfloat16, (dim,), dev, name + "_weight"),
                                  oa, oh, ot, 0 if gw is None else gw.data_ptr())

    dq_out, gq, qs = side(dq, q, q_weight, dq_out, "q")
    dk_out, gk, ks = (None, None, None) if k is None else side(dk, k, k_weight, dk_out, "k")
    need = 0 if gq is None and gk is None else qk_norm_rope_backward_workspace_bytes(tokens, dim)
    ws, wa, nbytes = _scratch(workspace, need, q, dev, stream)
    _check("qk_norm_rope_backward", load().qk_norm_rope_backward(qs, ks, tokens, dim, 1 if norm else 0, eps, r, wa,
                                                                 nbytes, _queue(stream, dev)))
    return dq_out, dk_out, gq, gk


_ROPE_KINDS = {"linear": 1, "ntk": 2, "yarn": 3}


def rope_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, trained_tokens=0, low_turns=1.0,
                     high_turns=32.0, device=None):
    """(inv_freq float32 [rotary_dim / 2], scale) for qk_norm_rope: base^(-2 i / rotary_dim), scaled for longer
    contexts by scaling "linear" (divided by factor), "ntk" (a larger base) or "yarn" (channels that turn at most
    low_turns times over trained_tokens are divided by factor, those that turn at least high_turns times are kept,
    in between mixed linearly in the number of turns, not in the channel's index, and scale = 0.1 ln(factor) + 1).
    Without device on the host."""
    if scaling is not None and scaling not in _ROPE_KINDS:
        raise ValueError(f"scaling: expected one of {sorted(_ROPE_KINDS)}, got {scaling!r}")
    s = None
    if scaling is not None:
        s = RopeScaling(_ROPE_KINDS[scaling], factor, trained_tokens, low_turns, high_turns)
    out = torch.empty((max(rotary_dim // 2, 1),), dtype=torch.float32, device="cpu")
    scale = ctypes.c_float()
    _check("qpl_rope_frequencies", load().qpl_rope_frequencies(rotary_dim, base, _ref(s), _ptr(out),
                                                               ctypes.byref(scale)))
    return (out if device is None else out.to(device)), scale.value


def quant_weight_awq(w, group=64, w_q=None, w_scale=None, w_zero=None, stream=None):
    """bf16 weight [N,K] -> (codes uint8 [N,K/2], scales bf16 [N,K/group], zero points uint8 [N,K/group])."""
    N, K = w.shape
    _expect(w, torch.bfloat16, (N, K), "w")
    G = K // group
    w_q = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device) if w_q is None else w_q
    w_scale = torch.empty((N, G), dtype=torch.bfloat16, device=w.device) if w_scale is None else w_scale
    w_zero = torch.empty((N, G), dtype=torch.uint8, device=w.device) if w_zero is None else w_zero
    _check("quant_weight_awq", load().quant_weight_awq(_ptr(w), N, K, group, _ptr(w_q), _ptr(w_scale), _ptr(w_zero),
                                                        _stream(stream)))
    return w_q, w_scale, w_zero


def qlinear_awq_w4a16(x, weight, weight_scale, weight_zero, group=64, y=None, stream=None):
    """y[M,N] bf16 = x [M,K] (bf16) times the group-wise 4-bit weight, dequantized as (q - z) s."""
    M, K = x.shape
    N = weight.shape[0]
    _expect(x, torch.bfloat16, (M, K), "x")
    _expect(weight, torch.uint8, (N, K // 2), "weight")
    _expect(weight_scale, torch.bfloat16, (N, K // group), "weight_scale")
    _expect(weight_zero, torch.uint8, (N, K // group), "weight_zero")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device) if y is None else y
    _check("qlinear_awq_w4a16", load().qlinear_awq_w4a16(_ptr(x), M, K, N, _ptr(weight), _ptr(weight_scale),
                                                          _ptr(weight_zero), group, _ptr(y), _stream(stream)))
    return y


def dequant_weight(scheme, weight, weight_scale, weight_scale_2=1.0, K=None, out=None, stream=None):
    """Dequantize an fp8r or nvfp4 weight to bf16 [N,K]."""
    N = weight.shape[0]
    if K is None:
        K = weight.shape[1] * (2 if scheme == QPL_NVFP4 else 1)
    out = torch.empty((N, K), dtype=torch.bfloat16, device=weight.device) if out is None else out
    _check("dequant_weight", load().dequant_weight(scheme, _ptr(weight), _ptr(weight_scale), float(weight_scale_2),
                                                   N, K, _ptr(out), _stream(stream)))
    return out


def amax_bf16(x, amax=None, stream=None):
    """Running max |x| into a device float32 [1] (initialised to 0 when not given)."""
    amax = torch.zeros((1,), dtype=torch.float32, device=x.device) if amax is None else amax
    _check("qpl_amax_bf16", load().qpl_amax_bf16(_ptr(x), x.numel(), _ptr(amax), _stream(stream)))
    return amax


def nvfp4_global_scale(amax):
    """amax / (448 * 6) in fp32 (host)."""
    return float(load().qpl_nvfp4_global_scale(float(amax)))


def timing_enable(on=True):
    """Bracket every library kernel launch with HIP events (profiling aid)."""
    load().qpl_timing_enable(1 if on else 0)


def timing_select(kinds):
    """Time only the named kernel kinds (names from KERNELS); an empty list turns timing off."""
    mask = 0
    for k in kinds:
        mask |= 1 << KERNELS.index(k)
    load().qpl_timing_select(mask)


def timing_collect():
    """Wait for the recorded events; return {kernel: (launches, total_ms)} and clear."""
    n = len(KERNELS)
    launches = (ctypes.c_int64 * n)()
    total = (ctypes.c_double * n)()
    _check("qpl_timing_collect_n", load().qpl_timing_collect_n(ctypes.cast(launches, ctypes.c_void_p),
                                                               ctypes.cast(total, ctypes.c_void_p), n))
    return {k: (int(launches[i]), float(total[i])) for i, k in enumerate(KERNELS)}
