"""Thin ctypes binding of libmoe_mi355x.so (include/moe.h).

Argument marshalling only: torch tensors become device pointers, the current torch stream
becomes the hipStream_t, and non-zero status codes become ``MoEError``.  Every computation runs
in the library's HIP kernels; if the library is missing, the first call raises.
The functions keep the C names: ``moe_route``, ``moe_permute``, ``moe_grouped_ffn``,
``moe_combine``, ``moe_forward``, ``moe_backward``, ``moe_decode``, ``moe_quantize_fp8``,
``moe_grouped_ffn_fp8``, ``moe_quantize_mx``, ``moe_grouped_ffn_mx``, ``moe_router_loss``,
``moe_router_loss_backward``, ``moe_backward_aux``, ``moe_dropout``, ``moe_combine_dropout``,
``moe_linear``, ``moe_linear_backward``, ``moe_norm``, ``moe_norm_backward``, ``moe_grad_norm``,
``moe_grad_clip``, ``moe_quantize_w4``, ``moe_dequantize_w4``, ``moe_linear_w4``, ``moe_decode_w4`` (plus
sizing helpers).
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

MOE_F32, MOE_BF16 = 0, 1
ROUND_NONE, ROUND_NEAREST, ROUND_UP, ROUND_DOWN, ROUND_STOCHASTIC = 0, 1, 2, 3, 4
OP_ROUTE, OP_PERMUTE, OP_FFN, OP_COMBINE, OP_FORWARD, OP_BACKWARD, OP_DECODE, OP_FFN_FP8, OP_FFN_MX = range(9)
FP8_E4M3, FP8_E5M2 = 0, 1
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}
LINEAR_FORWARD, LINEAR_BACKWARD = 0, 1
W4_WAYS = ["streamed", "tiled", "expanded"]
W4_FORMATS = {"int4": 0, "fp4": 1}
NORM_KINDS = {"layer": 0, "rms": 1}
LINEAR_OUT, LINEAR_DX, LINEAR_DW = 0, 1, 2
STATUS = {0: "MOE_OK", -1: "MOE_EINVAL", -2: "MOE_ENOTSUP", -3: "MOE_EWORKSPACE", -4: "MOE_EHIP"}

EXPORTS = ["moe_max_rows", "moe_workspace_bytes", "moe_route", "moe_permute", "moe_grouped_ffn",
           "moe_combine", "moe_forward", "moe_backward", "moe_decode", "moe_decode_status",
           "moe_route_noalloc", "moe_route_noalloc_max_bytes", "moe_mx_scale_bytes", "moe_quantize_mx",
           "moe_grouped_ffn_mx",
           "moe_decode_set_spin_limit", "moe_quantize_fp8",
           "moe_grouped_ffn_fp8", "moe_status_string", "moe_last_error",
           "moe_backward_aux", "moe_router_loss", "moe_router_loss_backward",
           "moe_router_loss_workspace_bytes", "moe_dropout", "moe_combine_dropout", "moe_linear",
           "moe_linear_backward", "moe_linear_workspace_bytes", "moe_linear_plan",
           "moe_norm", "moe_norm_workspace_bytes", "moe_norm_backward", "moe_grad_table_bytes", "moe_grad_table",
           "moe_grad_workspace_bytes", "moe_grad_norm",
           "moe_grad_clip", "moe_w4_scale_bytes", "moe_quantize_w4", "moe_dequantize_w4", "moe_linear_w4_workspace_bytes",
           "moe_linear_w4_plan", "moe_linear_w4_cut", "moe_linear_w4", "moe_decode_w4",
           "moe_version", "moe_timing_enable", "moe_timing_read"]
STAGES = ["router_gemm", "route", "tiles", "up_gemm", "down_gemm", "permute", "combine", "dact_gemm",
          "dw_down_gemm", "dw_gu_gemm", "dx_gemm", "router_bwd", "dwr_gemm", "decode", "fp8_quant",
          "fp8_up_gemm", "fp8_down_gemm", "router_loss", "dropout", "linear", "linear_bwd", "norm",
          "grad", "w4", "linear_w4"]


class MoEError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (STATUS.get(status, status), message))
        self.status = status


class Dims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("n", ctypes.c_int64),
                ("E", ctypes.c_int32), ("K", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("round_mode", ctypes.c_int32), ("tile_m", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("round_rand", ctypes.c_void_p)]


class LinearDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("ldx", ctypes.c_int64),
                ("ldr", ctypes.c_int64), ("ldy", ctypes.c_int64), ("dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("flags", ctypes.c_int32)]


class NormDims(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int64) for k in ("rows", "cols", "ldx", "ldr", "lds", "ldy")] + [
        (k, ctypes.c_int32) for k in ("dtype", "wtype", "kind", "flags")] + [("eps", ctypes.c_float)]


class GradStruct(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("n", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class GradListStruct(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("count", ctypes.c_int32), ("chunks", ctypes.c_int32)]


class W4Struct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("format", ctypes.c_int32), ("group", ctypes.c_int32)]


PLAN_FIELDS = ["topk_idx", "topk_w", "counts", "expert_off", "row_token", "row_w", "tok_off",
               "tok_row", "meta"]


class PlanStruct(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in PLAN_FIELDS]


_lib = None


def lib():
    """The loaded library (loaded once; raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("%s is missing: build it with `python -m mixture_experts_layer_lds_amd.build`"
                               % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, st = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        pd = ctypes.POINTER(Dims)
        pp = ctypes.POINTER(PlanStruct)
        L.moe_max_rows.argtypes, L.moe_max_rows.restype = [pd], ctypes.c_int64
        L.moe_workspace_bytes.argtypes, L.moe_workspace_bytes.restype = [pd, ctypes.c_int], sz
        L.moe_route.argtypes = [pd, vp, vp, vp, vp, pp, vp, sz, vp]
        L.moe_route_noalloc.argtypes = [pd, vp, vp, vp, vp, pp, vp]
        L.moe_route_noalloc_max_bytes.argtypes, L.moe_route_noalloc_max_bytes.restype = [], sz
        L.moe_permute.argtypes = [pd, pp, vp, vp, vp]
        L.moe_grouped_ffn.argtypes = [pd, pp, vp, ctypes.c_int, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_combine.argtypes = [pd, pp, vp, ctypes.c_int, vp, vp]
        L.moe_forward.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, pp, vp, vp, vp, sz, vp]
        L.moe_backward.argtypes = [pd, vp, vp, vp, vp, vp, vp, pp, vp, vp, vp, vp, vp, vp, vp, vp,
                                   vp, sz, vp]
        L.moe_decode.argtypes = [pd, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_decode_status.argtypes, L.moe_decode_status.restype = [vp], st
        L.moe_decode_set_spin_limit.argtypes = [ctypes.c_longlong]
        L.moe_decode_set_spin_limit.restype = ctypes.c_longlong
        L.moe_quantize_fp8.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, vp, vp, vp, vp]
        L.moe_grouped_ffn_fp8.argtypes = [pd, pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_mx_scale_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64]
        L.moe_mx_scale_bytes.restype = ctypes.c_int64
        L.moe_quantize_mx.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp]
        L.moe_grouped_ffn_mx.argtypes = [pd, pp, ctypes.c_int, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                         sz, vp]
        i32, i64, pl = ctypes.c_int32, ctypes.c_int64, ctypes.POINTER(LinearDims)
        L.moe_backward_aux.argtypes = [pd, vp, vp, vp, vp, vp, vp, pp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_router_loss_workspace_bytes.argtypes, L.moe_router_loss_workspace_bytes.restype = [pd, i32], sz
        L.moe_router_loss.argtypes = [pd, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_router_loss_backward.argtypes = [pd, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp]
        L.moe_dropout.argtypes = [i64, i64, ctypes.c_int, vp, i64, vp, i64, ctypes.c_double, vp, vp, i64, vp]
        L.moe_combine_dropout.argtypes = [pd, pp, vp, ctypes.c_int, vp, ctypes.c_double, vp, vp, vp]
        L.moe_linear_workspace_bytes.argtypes, L.moe_linear_workspace_bytes.restype = [pl, ctypes.c_int], sz
        L.moe_linear_plan.argtypes = [pl, ctypes.c_int, ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.moe_linear_plan.restype = ctypes.c_int
        L.moe_linear.argtypes = [pl, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_linear_backward.argtypes = [pl, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        pn, pg = ctypes.POINTER(NormDims), ctypes.POINTER(GradStruct)
        L.moe_norm.argtypes = [pn, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.moe_norm_workspace_bytes.argtypes, L.moe_norm_workspace_bytes.restype = [pn], sz
        L.moe_norm_backward.argtypes = [pn, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        po = ctypes.POINTER(GradListStruct)
        L.moe_grad_table_bytes.argtypes, L.moe_grad_table_bytes.restype = [pg, i32], sz
        L.moe_grad_table.argtypes = [pg, i32, vp, sz, po]
        L.moe_grad_workspace_bytes.argtypes, L.moe_grad_workspace_bytes.restype = [], sz
        L.moe_grad_norm.argtypes = [po, vp, vp, sz, vp]
        L.moe_grad_clip.argtypes = [po, ctypes.c_double, vp, vp, vp, sz, vp]
        pw, ci, pi = ctypes.POINTER(W4Struct), ctypes.c_int, ctypes.POINTER(i32)
        L.moe_w4_scale_bytes.argtypes, L.moe_w4_scale_bytes.restype = [i64, i64, i32, i32], i64
        L.moe_quantize_w4.argtypes = [i64, i64, ci, vp, pw, vp]
        L.moe_dequantize_w4.argtypes = [i64, i64, ci, pw, vp, vp]
        L.moe_linear_w4_workspace_bytes.argtypes, L.moe_linear_w4_workspace_bytes.restype = [pl], sz
        L.moe_linear_w4_plan.argtypes, L.moe_linear_w4_plan.restype = [pl], ci
        L.moe_linear_w4_cut.argtypes, L.moe_linear_w4_cut.restype = [pl, pi, pi, pi], ci
        L.moe_linear_w4.argtypes = [pl, vp, pw, vp, vp, vp, vp, sz, vp]
        L.moe_decode_w4.argtypes = [pd, vp, vp, vp, pw, pw, pw, vp, vp, vp, vp, vp, sz, vp]
        for f in ("moe_norm", "moe_norm_backward", "moe_grad_table", "moe_grad_norm", "moe_grad_clip", "moe_quantize_w4", "moe_dequantize_w4",
                  "moe_linear_w4", "moe_decode_w4"):
            getattr(L, f).restype = st
        for f in ("moe_backward_aux", "moe_router_loss", "moe_router_loss_backward", "moe_dropout",
                  "moe_combine_dropout", "moe_linear", "moe_linear_backward"):
            getattr(L, f).restype = st
        for f in ("moe_route", "moe_route_noalloc", "moe_permute", "moe_grouped_ffn", "moe_combine", "moe_forward",
                  "moe_backward", "moe_decode", "moe_quantize_fp8", "moe_grouped_ffn_fp8", "moe_quantize_mx",
                  "moe_grouped_ffn_mx"):
            getattr(L, f).restype = st
        L.moe_status_string.argtypes, L.moe_status_string.restype = [ctypes.c_int], ctypes.c_char_p
        L.moe_last_error.argtypes, L.moe_last_error.restype = [], ctypes.c_char_p
        L.moe_version.argtypes, L.moe_version.restype = [], ctypes.c_char_p
        L.moe_timing_enable.argtypes, L.moe_timing_enable.restype = [ctypes.c_int], ctypes.c_int
        L.moe_timing_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_float), ctypes.c_int]
        L.moe_timing_read.restype = ctypes.c_int
        _lib = L
    return _lib


def make_dims(T, d, n, E, K, dtype="bf16", round_mode=ROUND_NONE, tile_m=128, round_rand=None):
    """Layer shape; ``round_rand`` is the [E] int32/uint32 device tensor of random words that
    stochastic token rounding reads (the caller keeps it alive while the dims are used)."""
    dt = {"bf16": MOE_BF16, "f32": MOE_F32, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[dtype]
    return Dims(int(T), int(d), int(n), int(E), int(K), dt, int(round_mode), int(tile_m), 0,
                _p(round_rand))


def torch_dtype(dims):
    return torch.bfloat16 if dims.dtype == MOE_BF16 else torch.float32


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


# the current stream's handle without building a torch stream object (2.8 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None):
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return (stream if stream is not None else torch.cuda.current_stream()).cuda_stream


def _stream_on(dev, stream):
    """As _stream, where the current device is known."""
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def _gp(t, dev):
    """Address of a tensor that GPU ``dev`` can read (None and addresses pass)."""
    if t is None or t.__class__ is int:
        return t
    if t.get_device() != dev:
        raise MoEError(-1, "a tensor is on %s: it must be on the current GPU, cuda:%d" % (t.device, dev))
    return t.data_ptr()


def _on_gpu(*tensors):
    dev = torch.cuda.current_device()
    for t in tensors:
        _gp(t, dev)


_TYPES = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


# The tensors that a call takes (None and addresses pass): what is as expected leaves by the first return, for 0.15 us of a
# call's 6 each.
def _gv(t, dev, dtype, n, name):
    """Address of a contiguous tensor of at least n elements of dtype that GPU ``dev`` can read."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is dtype and t.get_device() == dev and t.numel() >= n and t.is_contiguous():
        return t.data_ptr()
    _check_type(t, dtype, name)
    if t.numel() < n or not t.is_contiguous():
        raise MoEError(-1, "%s has %d elements (contiguous: %s), %d contiguous ones expected" % (name, t.numel(), t.is_contiguous(), n))
    return _gp(t, dev)


def _gm(t, dev, dtype, rows, cols, ld, name):
    """Address of a tensor of ``rows`` rows of cols elements of dtype, ld elements apart (0: cols), as _gv."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is dtype and t.get_device() == dev and t.numel() == rows * cols and (not ld or ld == cols) and t.is_contiguous():
        return t.data_ptr()
    _check_type(t, dtype, name)
    _check_rows(t, rows, cols, ld or cols, name)
    return _gp(t, dev)


def _check_type(t, dtype, name):
    if t.dtype is not dtype:
        raise MoEError(-1, "%s is %s, %s expected" % (name, t.dtype, dtype))


def _check_rows(t, rows, cols, ld, name):
    size, step, dim = t.shape, t.stride(), t.dim()
    if rows <= 0 or dim == 2 and step == (ld, 1) and size[0] >= rows and size[1] >= cols:
        return
    if dim and cols > 1 and size[-1] > 1 and step[-1] != 1:
        raise MoEError(-1, "%s: neighbours in a row lie %d elements apart" % (name, step[-1]))
    if dim > 1 and rows > 1 and size[-2] > 1 and step[-2] != ld and size[-1] > 1:
        raise MoEError(-1, "%s: its rows lie %d elements apart, by the dims %d" % (name, step[-2], ld))
    if dim > 2 and not t.is_contiguous() and any(step[i] != step[i + 1] * size[i + 1] for i in range(dim - 2) if size[i] > 1):
        raise MoEError(-1, "%s: its rows do not lie at one distance" % name)
    # (a view of the first columns of longer rows ends before the last row's stride does)
    room = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if t.numel() < rows * cols or room < (rows - 1) * ld + cols:
        raise MoEError(-1, "%s has %d elements, %d rows of %d (%d apart) expected" % (name, t.numel(), rows, cols, ld))


def _gw(ws, dev, ws_bytes):
    """Address of a workspace tensor of at least ws_bytes bytes, as _gv."""
    if ws is None or ws.__class__ is int:
        return ws
    if ws.numel() * ws.element_size() < ws_bytes or not ws.is_contiguous():
        raise MoEError(-1, "the workspace has %d bytes, not ws_bytes=%d" % (ws.numel() * ws.element_size(), ws_bytes))
    return _gp(ws, dev)


def _check(status):
    if status != 0:
        raise MoEError(status, lib().moe_last_error().decode())


def moe_max_rows(dims):
    r = lib().moe_max_rows(ctypes.byref(dims))
    if r == 0:
        raise MoEError(-1, lib().moe_last_error().decode())
    return r


def moe_workspace_bytes(dims, op):
    return lib().moe_workspace_bytes(ctypes.byref(dims), op)


class Plan:
    """Caller-owned routing plan: the device arrays of ``moe_plan`` with their ctypes view."""

    def __init__(self, dims, device="cuda"):
        T, E, K = dims.T, dims.E, dims.K
        R = moe_max_rows(dims)
        i32, f32 = torch.int32, torch.float32
        self.R_max = R
        self.topk_idx = torch.empty(T * K, dtype=i32, device=device)
        self.topk_w = torch.empty(T * K, dtype=f32, device=device)
        self.counts = torch.empty(E, dtype=i32, device=device)
        self.expert_off = torch.empty(E + 1, dtype=i32, device=device)
        self.row_token = torch.empty(R, dtype=i32, device=device)
        self.row_w = torch.empty(R, dtype=f32, device=device)
        self.tok_off = torch.empty(T + 1, dtype=i32, device=device)
        self.tok_row = torch.empty(R, dtype=i32, device=device)
        self.meta = torch.zeros(16, dtype=i32, device=device)
        self.struct = PlanStruct(*[getattr(self, f).data_ptr() for f in PLAN_FIELDS])

    def ref(self):
        return ctypes.byref(self.struct)

    def to_host(self):
        """numpy copies of the plan arrays, trimmed to the actual row count R."""
        R = int(self.meta[0].item())
        out = {f: getattr(self, f).cpu().numpy() for f in PLAN_FIELDS}
        for f in ("row_token", "row_w", "tok_row"):
            out[f] = out[f][:R]
        out["R"] = R
        return out


def workspace(dims, op, device="cuda"):
    nbytes = moe_workspace_bytes(dims, op)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), nbytes


def moe_route(dims, X, W_r, bias, logits, plan, ws, ws_bytes, stream=None):
    _check(lib().moe_route(ctypes.byref(dims), _p(X), _p(W_r), _p(bias), _p(logits), plan.ref(),
                           _p(ws), ws_bytes, _stream(stream)))


def moe_route_noalloc(dims, X, W_r, bias, logits, plan, stream=None):
    """moe_route with the library's static routing buffer as workspace (no allocation)."""
    _check(lib().moe_route_noalloc(ctypes.byref(dims), _p(X), _p(W_r), _p(bias), _p(logits), plan.ref(),
                                   _stream(stream)))


def moe_route_noalloc_max_bytes():
    return lib().moe_route_noalloc_max_bytes()


def moe_permute(dims, plan, X, X_perm, stream=None):
    _check(lib().moe_permute(ctypes.byref(dims), plan.ref(), _p(X), _p(X_perm), _stream(stream)))


def moe_grouped_ffn(dims, plan, A_in, gathered, W_gate, W_up, W_down, H_cache, Y_perm, ws, ws_bytes,
                    stream=None):
    _check(lib().moe_grouped_ffn(ctypes.byref(dims), plan.ref(), _p(A_in), int(bool(gathered)),
                                 _p(W_gate), _p(W_up), _p(W_down), _p(H_cache), _p(Y_perm), _p(ws),
                                 ws_bytes, _stream(stream)))


def moe_combine(dims, plan, Y_perm, weighted, out, stream=None):
    _check(lib().moe_combine(ctypes.byref(dims), plan.ref(), _p(Y_perm), int(bool(weighted)), _p(out),
                             _stream(stream)))


def moe_forward(dims, X, W_r, bias, W_gate, W_up, W_down, logits, plan, H_cache, out, ws, ws_bytes,
                stream=None):
    _check(lib().moe_forward(ctypes.byref(dims), _p(X), _p(W_r), _p(bias), _p(W_gate), _p(W_up),
                             _p(W_down), _p(logits), plan.ref(), _p(H_cache), _p(out), _p(ws), ws_bytes,
                             _stream(stream)))


def moe_decode(dims, X, W_r, bias, W_gate, W_up, W_down, logits, topk_idx, topk_w, out, ws, ws_bytes,
               stream=None):
    _check(lib().moe_decode(ctypes.byref(dims), _p(X), _p(W_r), _p(bias), _p(W_gate), _p(W_up),
                            _p(W_down), _p(logits), _p(topk_idx), _p(topk_w), _p(out), _p(ws), ws_bytes,
                            _stream(stream)))


def moe_decode_status(stream=None):
    """Raises MoEError(MOE_EHIP) if a moe_decode kernel on the current device gave up at a grid
    barrier since the last check (waits for the stream first); clears the device's status word."""
    _check(lib().moe_decode_status(_stream(stream)))


def moe_decode_set_spin_limit(limit):
    """Polls before a moe_decode grid barrier gives up (later launches); returns the previous limit."""
    prev = lib().moe_decode_set_spin_limit(int(limit))
    if prev < 0:
        raise MoEError(-1, lib().moe_last_error().decode())
    return prev


def moe_quantize_fp8(src, codes, scales, stream=None):
    """Per-row E4M3 codes and power-of-two scales of a 2-D bf16 / fp32 tensor (rows x K)."""
    rows, K = src.shape[0], src.shape[-1]
    dtype = MOE_BF16 if src.dtype == torch.bfloat16 else MOE_F32
    _check(lib().moe_quantize_fp8(rows, K, dtype, _p(src), _p(codes), _p(scales), _stream(stream)))


def moe_grouped_ffn_fp8(dims, plan, Xq, sx, Wg_q, sg, Wu_q, su, Wd_q, sd, act, act_q, sact, Y_perm, ws,
                        ws_bytes, stream=None):
    _check(lib().moe_grouped_ffn_fp8(ctypes.byref(dims), plan.ref(), _p(Xq), _p(sx), _p(Wg_q), _p(sg),
                                     _p(Wu_q), _p(su), _p(Wd_q), _p(sd), _p(act), _p(act_q), _p(sact),
                                     _p(Y_perm), _p(ws), ws_bytes, _stream(stream)))


def moe_mx_scale_bytes(rows, K):
    return lib().moe_mx_scale_bytes(int(rows), int(K))


def moe_quantize_mx(src, fmt, codes, scales, stream=None):
    """Block-scaled FP8 codes and E8M0 scale bytes of a 2-D bf16 / fp32 tensor (rows x K)."""
    rows, K = src.shape[0], src.shape[-1]
    dtype = MOE_BF16 if src.dtype == torch.bfloat16 else MOE_F32
    _check(lib().moe_quantize_mx(rows, K, dtype, int(fmt), _p(src), _p(codes), _p(scales), _stream(stream)))


def moe_grouped_ffn_mx(dims, plan, fmt, Xq, sx, Wg_q, sg, Wu_q, su, Wd_q, sd, act, act_q, sact, Y_perm, ws, ws_bytes,
                       stream=None):
    _check(lib().moe_grouped_ffn_mx(ctypes.byref(dims), plan.ref(), int(fmt), _p(Xq), _p(sx), _p(Wg_q), _p(sg),
                                    _p(Wu_q), _p(su), _p(Wd_q), _p(sd), _p(act), _p(act_q), _p(sact), _p(Y_perm),
                                    _p(ws), ws_bytes, _stream(stream)))


def moe_backward(dims, dY, X, W_r, W_gate, W_up, W_down, plan, H_cache, dX, dW_gate, dW_up, dW_down,
                 dS, dLogits, dW_r, ws, ws_bytes, stream=None):
    _check(lib().moe_backward(ctypes.byref(dims), _p(dY), _p(X), _p(W_r), _p(W_gate), _p(W_up),
                              _p(W_down), plan.ref(), _p(H_cache), _p(dX), _p(dW_gate), _p(dW_up),
                              _p(dW_down), _p(dS), _p(dLogits), _p(dW_r), _p(ws), ws_bytes,
                              _stream(stream)))


def moe_backward_aux(dims, dY, X, W_r, W_gate, W_up, W_down, plan, H_cache, dLogits_aux, dX, dW_gate, dW_up, dW_down,
                     dS, dLogits, dW_r, ws, ws_bytes, stream=None):
    """moe_backward with further gradients of the router logits ([T, E] fp32, or None)."""
    _check(lib().moe_backward_aux(ctypes.byref(dims), _p(dY), _p(X), _p(W_r), _p(W_gate), _p(W_up), _p(W_down),
                                  plan.ref(), _p(H_cache), _p(dLogits_aux), _p(dX), _p(dW_gate), _p(dW_up),
                                  _p(dW_down), _p(dS), _p(dLogits), _p(dW_r), _p(ws), ws_bytes, _stream(stream)))


def router_loss_workspace(dims, n_seq, device="cuda"):
    nbytes = lib().moe_router_loss_workspace_bytes(ctypes.byref(dims), int(n_seq))
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), nbytes


def moe_router_loss(dims, logits, topk_idx, n_seq, seq_off, token_mask, seq_tokens, seq_counts, prob_sum, lse, loss,
                    ws, ws_bytes, stream=None):
    """Balance loss and z-loss of a batch of router logits, with the per-sequence expert counts."""
    _check(lib().moe_router_loss(ctypes.byref(dims), _p(logits), _p(topk_idx), int(n_seq), _p(seq_off),
                                 _p(token_mask), _p(seq_tokens), _p(seq_counts), _p(prob_sum), _p(lse), _p(loss),
                                 _p(ws), ws_bytes, _stream(stream)))


def moe_router_loss_backward(dims, dloss, logits, n_seq, seq_off, token_mask, seq_tokens, seq_counts, lse, dLogits,
                             stream=None):
    """Gradient of the two router losses (weights dloss, fp32 [2] on the device) for the logits."""
    _check(lib().moe_router_loss_backward(ctypes.byref(dims), _p(dloss), _p(logits), int(n_seq), _p(seq_off),
                                          _p(token_mask), _p(seq_tokens), _p(seq_counts), _p(lse), _p(dLogits),
                                          _stream(stream)))


def _row_stride(t, rows, cols, name):
    """Row stride of a rows x cols tensor whose rows are contiguous."""
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise MoEError(-1, "%s must have contiguous rows" % name)
    return ld if rows > 1 else cols


def _rng_ptr(rng, dev):
    """Address of the generator's two words, which the kernels read on GPU ``dev`` (None: not known)."""
    if isinstance(rng, int):
        return rng
    dtype = rng.dtype
    if rng.numel() < 2 or (dtype is not torch.int64 and dtype is not torch.uint64) or not rng.is_contiguous():
        raise MoEError(-1, "rng must hold two consecutive 64-bit words")
    on = rng.get_device()  # -1: not a GPU's memory
    if on < 0 or (dev is not None and on != dev):
        raise MoEError(-1, "rng is on %s: it must be on the GPU that holds the tensors" % rng.device)
    return rng.data_ptr()


def moe_dropout(x, residual, p, rng, out, stream=None):
    """out = residual + dropout(x) of 2-D bf16 / fp32 tensors (residual may be None; rows may be
    strided); rng is a device tensor of two 64-bit words, {seed, offset}.  Without a residual this is
    also the gradient of dropout."""
    dtype, shape = x.dtype, x.shape
    if dtype is torch.bfloat16:
        code = MOE_BF16
    elif dtype is torch.float32:
        code = MOE_F32
    else:
        raise MoEError(-2, "dtype %s not supported" % dtype)
    if len(shape) != 2:
        raise MoEError(-1, "x must have two dimensions")
    if out.shape != shape or out.dtype is not dtype:
        raise MoEError(-1, "out must be %s of %s" % (tuple(shape), dtype))
    rows, cols = shape
    res, ldr = None, 0
    if residual is not None:
        if residual.shape != shape or residual.dtype is not dtype:
            raise MoEError(-1, "residual must be %s of %s" % (tuple(shape), dtype))
        res, ldr = residual.data_ptr(), _row_stride(residual, rows, cols, "residual")
    ldx, ldo, dev = _row_stride(x, rows, cols, "x"), _row_stride(out, rows, cols, "out"), x.get_device()
    words = _rng_ptr(rng, dev)
    if out.get_device() != dev or (residual is not None and residual.get_device() != dev):
        raise MoEError(-1, "x, residual and out must be on one GPU")
    status = lib().moe_dropout(rows, cols, code, x.data_ptr(), ldx, res, ldr, p, words, out.data_ptr(), ldo, _stream(stream))
    if status:
        _check(status)


def moe_combine_dropout(dims, plan, Y_perm, weighted, residual, p, rng, out, stream=None):
    """moe_combine with dropout and the residual sum (None: no residual) in its epilogue."""
    words = _rng_ptr(rng, out.get_device() if isinstance(out, torch.Tensor) else None)
    _check(lib().moe_combine_dropout(ctypes.byref(dims), plan.ref(), _p(Y_perm), int(bool(weighted)), _p(residual),
                                     float(p), words, _p(out), _stream(stream)))


def make_linear_dims(M, N, K, dtype="bf16", act="none", ldx=0, ldr=0, ldy=0):
    """Shape of a dense projection: M rows, N outputs, K inputs; row strides of X / dX, residual and
    out / dY in elements (0 = dense)."""
    dt = {"bf16": MOE_BF16, "f32": MOE_F32, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}[dtype]
    return LinearDims(int(M), int(N), int(K), int(ldx), int(ldr), int(ldy), dt, ACTS[act], 0)


def moe_linear_workspace_bytes(dims, op):
    return lib().moe_linear_workspace_bytes(ctypes.byref(dims), op)


def linear_workspace(dims, op, device="cuda"):
    nbytes = moe_linear_workspace_bytes(dims, op)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), nbytes


def moe_linear_plan(dims, product):
    """(tile edge, slices of the reduction, whether dX and dW share a launch) of one product."""
    slices, paired = ctypes.c_int32(), ctypes.c_int32()
    tile = lib().moe_linear_plan(ctypes.byref(dims), product, ctypes.byref(slices), ctypes.byref(paired))
    if tile < 0:
        _check(tile)
    return tile, slices.value, bool(paired.value)


def moe_linear(dims, X, W, bias, residual, Z, out, ws, ws_bytes, stream=None):
    """out = residual + act(X W^T + bias); bias, residual and Z (the saved pre-activation) may be None."""
    _check(lib().moe_linear(ctypes.byref(dims), _p(X), _p(W), _p(bias), _p(residual), _p(Z), _p(out), _p(ws),
                            ws_bytes, _stream(stream)))


def moe_linear_backward(dims, dY, X, W, Z, dX, dW, dbias, ws, ws_bytes, stream=None):
    """Gradients of moe_linear from dY and the saved pre-activation; dX, dW and dbias may be None."""
    _check(lib().moe_linear_backward(ctypes.byref(dims), _p(dY), _p(X), _p(W), _p(Z), _p(dX), _p(dW), _p(dbias),
                                     _p(ws), ws_bytes, _stream(stream)))


def make_norm_dims(rows, cols, dtype="bf16", kind="layer", eps=1e-5, wtype="f32", ldx=0, ldr=0, lds=0, ldy=0):
    """Shape of a layer / RMS norm; wtype: type of weight and bias; row strides in elements of x / dx, residual /
    dsum, sum and y / dy (0 = dense)."""
    types = {"bf16": MOE_BF16, "f32": MOE_F32, torch.bfloat16: MOE_BF16, torch.float32: MOE_F32}
    return NormDims(int(rows), int(cols), int(ldx), int(ldr), int(lds), int(ldy), types[dtype], types[wtype],
                    NORM_KINDS[kind], 0, float(eps))


def norm_workspace(dims, device="cuda"):
    nbytes = lib().moe_norm_workspace_bytes(ctypes.byref(dims))
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), nbytes


def moe_norm(dims, x, residual, weight, bias, sum, y, mean, rstd, stream=None):
    """sum = x + residual, y = norm(sum) weight + bias, with the rows' mean and 1 / deviation; residual, weight,
    bias, sum, mean and rstd may be None."""
    d, t, w, n, c = torch.cuda.current_device(), _TYPES.get(dims.dtype), _TYPES.get(dims.wtype), dims.rows, dims.cols
    status = lib().moe_norm(ctypes.byref(dims), _gm(x, d, t, n, c, dims.ldx, "x"), _gm(residual, d, t, n, c, dims.ldr, "residual"),
                            _gv(weight, d, w, c, "weight"), _gv(bias, d, w, c, "bias"), _gm(sum, d, t, n, c, dims.lds, "sum"),
                            _gm(y, d, t, n, c, dims.ldy, "y"), _gv(mean, d, torch.float32, n, "mean"),
                            _gv(rstd, d, torch.float32, n, "rstd"), _stream_on(d, stream))
    if status:
        _check(status)


def moe_norm_backward(dims, dy, s, weight, mean, rstd, dsum, dx, dweight, dbias, ws, ws_bytes, stream=None):
    """Gradients of moe_norm from dy and the normalised sum s (x without a residual); dsum: the gradient that
    reaches s directly, or None; dx, dweight and dbias may be None."""
    d, t, w, n, c = torch.cuda.current_device(), _TYPES.get(dims.dtype), _TYPES.get(dims.wtype), dims.rows, dims.cols
    f = torch.float32
    _check(lib().moe_norm_backward(ctypes.byref(dims), _gm(dy, d, t, n, c, dims.ldy, "dy"), _gm(s, d, t, n, c, dims.lds, "s"),
                                   _gv(weight, d, w, c, "weight"), _gv(mean, d, f, n, "mean"), _gv(rstd, d, f, n, "rstd"),
                                   _gm(dsum, d, t, n, c, dims.ldr, "dsum"), _gm(dx, d, t, n, c, dims.ldx, "dx"),
                                   _gv(dweight, d, f, c, "dweight"), _gv(dbias, d, f, c, "dbias"), _gw(ws, d, ws_bytes), ws_bytes,
                                   _stream_on(d, stream)))


class Gradients:
    """A list of gradient tensors (contiguous, bf16 or fp32, on one GPU) and where moe_grad_clip writes the
    scaled ones: ``dst``, tensors of the same sizes and types, or in place without it.  Holds the tensors and
    the device table that the kernels read; made once for tensors that stay where they are, and kept until the calls
    on it have run (a captured graph: as long as it is replayed)."""

    def __init__(self, src, dst=None):
        self.src = list(src)
        self.dst = self.src if dst is None else list(dst)
        if len(self.src) != len(self.dst):
            raise MoEError(-1, "%d gradients but %d destinations" % (len(self.src), len(self.dst)))
        self.count = len(self.src)
        self.array = (GradStruct * max(self.count, 1))()
        for i, (s, d) in enumerate(zip(self.src, self.dst)):
            if s.dtype not in (torch.bfloat16, torch.float32):
                raise MoEError(-2, "gradient %d: dtype %s not supported" % (i, s.dtype))
            if d.dtype != s.dtype or d.numel() != s.numel():
                raise MoEError(-1, "gradient %d: its destination must be %d elements of %s" % (i, s.numel(), s.dtype))
            if not (s.is_contiguous() and d.is_contiguous()):
                raise MoEError(-1, "gradient %d must be contiguous" % i)
            if s.device != self.src[0].device or d.device != s.device:
                raise MoEError(-1, "gradient %d is on another device" % i)
            self.array[i] = GradStruct(s.data_ptr(), d.data_ptr(), s.numel(),
                                       MOE_BF16 if s.dtype is torch.bfloat16 else MOE_F32, 0)
        nbytes = lib().moe_grad_table_bytes(self.array, self.count)
        if nbytes == 0:
            raise MoEError(-1, lib().moe_last_error().decode())
        host = torch.empty(nbytes + 16, dtype=torch.uint8)
        host = host[-host.data_ptr() % 16:][:nbytes]
        self.struct = GradListStruct()
        _check(lib().moe_grad_table(self.array, self.count, host.data_ptr(), nbytes, ctypes.byref(self.struct)))
        self.table = host.to(self.src[0].device) if self.count else host
        self.struct.table = self.table.data_ptr()
        self._ref = ctypes.byref(self.struct)


def grad_workspace(grads, device="cuda"):
    nbytes = lib().moe_grad_workspace_bytes()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def moe_grad_norm(grads, norm, ws, ws_bytes, stream=None):
    """The global norm (fp32 [1]) of a list of gradients."""
    d = torch.cuda.current_device()
    _gp(grads.table if grads.count else None, d)
    _check(lib().moe_grad_norm(grads._ref, _gv(norm, d, torch.float32, 1, "norm"), _gw(ws, d, ws_bytes), ws_bytes, _stream_on(d, stream)))


def moe_grad_clip(grads, max_norm, norm_in, norm, ws, ws_bytes, stream=None):
    """Gradients scaled down to a global norm of max_norm.  norm_in (fp32 [1]): the norm to use; None: it is
    computed and written to norm."""
    d = torch.cuda.current_device()
    _gp(grads.table if grads.count else None, d)
    _check(lib().moe_grad_clip(grads._ref, max_norm, _gv(norm_in, d, torch.float32, 1, "norm_in"),
                               _gv(norm, d, torch.float32, 1, "norm"), _gw(ws, d, ws_bytes), ws_bytes, _stream_on(d, stream)))


class W4:
    """4-bit weights: codes uint8 [..., K / 2] (the even element in the low half) and their group scales, "int4"
    (bf16 [K / group, rows]) or "fp4" (bytes [ceil(K / 128), rows, 4]; group 32).  The leading dimensions of codes
    make up the rows."""

    def __init__(self, codes, scales, format="int4", group=128):
        self.codes, self.scales, self.format, self.group = codes, scales, format, int(group)
        self.K = 2 * codes.shape[-1]
        self.rows = codes.numel() // max(codes.shape[-1], 1)
        if codes.dtype is not torch.uint8 or not codes.is_contiguous():
            raise MoEError(-1, "codes must be contiguous bytes")
        if scales.dtype is not (torch.bfloat16 if format == "int4" else torch.uint8) or not scales.is_contiguous():
            raise MoEError(-1, "scales must be contiguous %s" % ("bf16" if format == "int4" else "bytes"))
        need = lib().moe_w4_scale_bytes(self.rows, self.K, W4_FORMATS[format], self.group)
        if need == 0 and self.rows > 0:
            raise MoEError(-2, lib().moe_last_error().decode())
        if scales.numel() * scales.element_size() != need:
            raise MoEError(-1, "scales hold %d bytes, %d x %d weights need %d" % (scales.numel() * scales.element_size(),
                                                                                  self.rows, self.K, need))
        if scales.device != codes.device:
            raise MoEError(-1, "codes are on %s but scales on %s" % (codes.device, scales.device))
        self.struct = W4Struct(codes.data_ptr(), scales.data_ptr(), W4_FORMATS[format], self.group)
        self._ref = ctypes.byref(self.struct)


def make_w4(rows, K, format="int4", group=128, device="cuda"):
    """Room for rows x K 4-bit weights, for moe_quantize_w4 to fill."""
    codes = torch.empty(rows, K // 2, dtype=torch.uint8, device=device)
    if format == "int4":
        return W4(codes, torch.empty(K // group, rows, dtype=torch.bfloat16, device=device), format, group)
    return W4(codes, torch.full((-(-K // 128), rows, 4), 127, dtype=torch.uint8, device=device), format, group)


def _w4_matrix(t, w4, name):
    if t.dtype not in (torch.bfloat16, torch.float32) or not t.is_contiguous() or t.numel() != w4.rows * w4.K:
        raise MoEError(-1, "%s must be %d x %d contiguous bf16 or fp32" % (name, w4.rows, w4.K))
    return MOE_BF16 if t.dtype is torch.bfloat16 else MOE_F32


def moe_quantize_w4(src, w4, stream=None):
    """4-bit codes and scales of a bf16 / fp32 tensor of w4's size."""
    dtype = _w4_matrix(src, w4, "src")
    _on_gpu(src, w4.codes)
    _check(lib().moe_quantize_w4(w4.rows, w4.K, dtype, _p(src), w4._ref, _stream(stream)))


def moe_dequantize_w4(w4, out, stream=None):
    """The values of 4-bit weights as bf16 or fp32."""
    dtype = _w4_matrix(out, w4, "out")
    _on_gpu(out, w4.codes)
    _check(lib().moe_dequantize_w4(w4.rows, w4.K, dtype, w4._ref, _p(out), _stream(stream)))


def linear_w4_workspace(dims, device="cuda"):
    nbytes = lib().moe_linear_w4_workspace_bytes(ctypes.byref(dims))
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device), nbytes


def moe_linear_w4_plan(dims):
    """How a product on 4-bit weights goes: "streamed", "tiled" or "expanded"."""
    way = lib().moe_linear_w4_plan(ctypes.byref(dims))
    if way < 0:
        _check(way)
    return W4_WAYS[way]


def moe_linear_w4_cut(dims):
    """(way, row tiles, token groups, slices) of a product on 4-bit weights."""
    n = [ctypes.c_int32() for _ in range(3)]
    way = lib().moe_linear_w4_cut(ctypes.byref(dims), *[ctypes.byref(v) for v in n])
    if way < 0:
        _check(way)
    return (W4_WAYS[way],) + tuple(v.value for v in n)


def _w4_rows(w4, rows, K, name):
    if w4.rows != rows or w4.K != K:
        raise MoEError(-1, "%s holds %d x %d weights, %d x %d expected" % (name, w4.rows, w4.K, rows, K))


def moe_linear_w4(dims, X, W, bias, residual, out, ws, ws_bytes, stream=None):
    """out = residual + act(X W^T + bias) with 4-bit weights W (a W4); bias and residual may be None."""
    _w4_rows(W, 2 * dims.N if dims.act == ACTS["swiglu"] else dims.N, dims.K, "W")
    d, t, m, n = torch.cuda.current_device(), torch.bfloat16, dims.M, dims.N
    _gp(W.codes, d)
    status = lib().moe_linear_w4(ctypes.byref(dims), _gm(X, d, t, m, dims.K, dims.ldx, "X"), W._ref,
                                 _gv(bias, d, torch.float32, W.rows, "bias"), _gm(residual, d, t, m, n, dims.ldr, "residual"),
                                 _gm(out, d, t, m, n, dims.ldy, "out"), _gw(ws, d, ws_bytes), ws_bytes, _stream_on(d, stream))
    if status:
        _check(status)


def moe_decode_w4(dims, X, W_r, bias, W_gate, W_up, W_down, logits, topk_idx, topk_w, out, ws, ws_bytes, stream=None):
    """moe_decode with 4-bit expert weights (W4 of E n, E n and E d rows)."""
    _w4_rows(W_gate, dims.E * dims.n, dims.d, "W_gate")
    _w4_rows(W_up, dims.E * dims.n, dims.d, "W_up")
    _w4_rows(W_down, dims.E * dims.d, dims.n, "W_down")
    d, T, E, K, w, b, f = torch.cuda.current_device(), dims.T, dims.E, dims.K, dims.d, torch.bfloat16, torch.float32
    for part in (W_gate, W_up, W_down):
        _gp(part.codes, d)
    _check(lib().moe_decode_w4(ctypes.byref(dims), _gv(X, d, b, T * w, "X"), _gv(W_r, d, b, E * w, "W_r"), _gv(bias, d, f, E, "bias"),
                               W_gate._ref, W_up._ref, W_down._ref, _gv(logits, d, f, T * E, "logits"),
                               _gv(topk_idx, d, torch.int32, T * K, "topk_idx"), _gv(topk_w, d, f, T * K, "topk_w"),
                               _gv(out, d, b, T * w, "out"), _gw(ws, d, ws_bytes), ws_bytes, _stream_on(d, stream)))


def moe_timing_enable(on):
    _check(lib().moe_timing_enable(int(bool(on))))


def moe_timing_read(stage, max_n=4096):
    """Per-launch durations (ms) recorded for a stage (name or index) since timing was enabled."""
    idx = STAGES.index(stage) if isinstance(stage, str) else int(stage)
    buf = (ctypes.c_float * max_n)()
    n = lib().moe_timing_read(idx, buf, max_n)
    if n < 0:
        _check(n)
    return list(buf[:n])
