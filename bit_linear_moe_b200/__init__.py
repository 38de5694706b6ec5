"""Python binding of libnvfp4, the NVFP4 linear layer for B200 (sm_100a).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  The functions carry the names of the C entry points declared in
``include/nvfp4.h`` and take torch CUDA tensors for device memory; outputs and
workspaces not passed in are allocated with torch (the library itself never
allocates).  Every call is enqueued on the current torch stream.

There is no fallback: if ``libnvfp4.so`` has not been built, importing the
library raises ``ImportError``; a non-zero status raises :class:`NVFP4Error`.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

# status codes, enumerations (values of include/nvfp4.h)
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_DTYPE, ERR_WORKSPACE, ERR_ARCH, ERR_LAUNCH, ERR_LAYOUT, ERR_MODE, \
    ERR_DEVICE_TIMEOUT, ERR_PAGE = range(12)
DTYPE_F32, DTYPE_BF16 = 0, 1
SF_ROWMAJOR, SF_TILED = 0, 1
MODE_AUTO, MODE_W4A16, MODE_W4A4 = 0, 1, 2
EPI_NONE, EPI_SWIGLU, EPI_COMBINE = 0, 1, 2


KV_BF16, KV_E4M3, KV_NVFP4 = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_SCALE_NONE, ROPE_SCALE_LINEAR, ROPE_SCALE_NTK, ROPE_SCALE_YARN = 0, 1, 2, 3
CHAIN_SRC_X, CHAIN_SRC_OP = 0, 1
CHAIN_XFORM_NONE, CHAIN_XFORM_RMS, CHAIN_XFORM_SILU_MUL = 0, 1, 2


class ChainOp(ctypes.Structure):
    """``nvfp4_chain_op`` of include/nvfp4.h."""
    _fields_ = [("w_codes", ctypes.c_void_p), ("w_scales", ctypes.c_void_p), ("w_gs", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("src", ctypes.c_int32), ("src_op", ctypes.c_int32),
                ("x", ctypes.c_void_p), ("x_ld", ctypes.c_int64), ("xform", ctypes.c_int32),
                ("y_xform", ctypes.c_int32), ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class KvCacheDesc(ctypes.Structure):
    """``nvfp4_kv_cache`` of include/nvfp4.h."""
    _fields_ = [("data", ctypes.c_void_p), ("k_gs", ctypes.c_void_p), ("v_gs", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32)]


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call} failed: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libnvfp4 (raises ImportError when it is not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m bit_linear_moe_b200.build` "
                              "(there is no fallback implementation)")
        L = ctypes.CDLL(LIB_PATH)
        p, i64, i32, sz, i = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int
        f32, f64 = ctypes.c_float, ctypes.c_double
        sig = {
            "nvfp4_status_string": (ctypes.c_char_p, [i]),
            "nvfp4_version": (i, []),
            "nvfp4_scales_bytes": (sz, [i64, i64, i]),
            "nvfp4_read_device_status": (i, [p, p]),
            "nvfp4_debug_wait_timeout": (i, [i64, p]),
            "nvfp4_quantize_workspace": (sz, [i64, i64]),
            "nvfp4_quantize": (i, [p, i, i64, i64, p, i, p, p, p, p, sz, p]),
            "nvfp4_linear_workspace": (sz, [i64, i64, i64, i]),
            "nvfp4_linear": (i, [p, i, i64, i64, p, p, i, p, i64, p, i, i, p, sz, p]),
            "nvfp4_linear_w4a4q": (i, [p, p, p, i64, i64, p, p, p, i64, p, i, p]),
            "nvfp4_rms_norm": (i, [p, i, i64, i64, i64, p, p]),
            "nvfp4_chain_workspace": (sz, [p, i32, i64]),
            "nvfp4_calibrate_workspace": (sz, [i64, i64, i64]),
            "nvfp4_calibrate": (i, [p, i64, i64, p, i, i64, i, p, p, p, p, p, p, p, sz, p]),
            "nvfp4_chain": (i, [p, i32, i64, p, sz, p]),
            "nvfp4_silu_mul": (i, [p, i, i64, i64, p, p]),
            "nvfp4_rms_norm_quant_workspace": (sz, [i64]),
            "nvfp4_rms_norm_quant": (i, [p, i, i64, i64, i64, i, p, p, p, p, sz, p]),
            "nvfp4_rope_freqs": (i, [i32, f64, i, f64, f64, f64, f64, p, p]),
            "nvfp4_rope": (i, [p, i, i64, i32, i32, i64, p, p, i32, i, f64, i, p, i, i64, p]),
            "nvfp4_kv_cache_bytes": (sz, [i64, i32, i32, i32, i]),
            "nvfp4_kv_write": (i, [p, p, p, i, i64, i64, i64, p, p]),
            "nvfp4_kv_read": (i, [p, p, i64, p, p, i, p]),
            "nvfp4_rope_kv_write": (i, [p, p, p, p, i, i64, i32, i64, i64, i64, p, p, p, i32, i, f64, p, p]),
            "nvfp4_attn_decode_workspace": (sz, [p, i64, i32, i64]),
            "nvfp4_attn_decode": (i, [p, i64, i32, i64, p, p, i64, i64, p, f32, i32, p, i, p, p, sz, p]),
            "moe_route_topk_workspace": (sz, [i64, i32, i32]),
            "moe_route_topk": (i, [p, p, p, i64, i64, i32, i32, p, p, p, p, p, p, p, p, sz, p]),
            "moe_route_topk_noalloc": (i, [p, p, p, i64, i64, i32, i32, p, p, p, p, p, p, p, p]),
            "moe_grouped_linear_workspace": (sz, [i64, i64, i64, i32, i32, i, i]),
            "nvfp4_linear_w4a4_ws_layout": (i, [i64, i64, p]),
            "moe_layer_decode_workspace": (sz, [i64, i64, i64, i32, i32]),
            "moe_layer_decode": (i, [p, p, p, i64, i64, i32, i32, p, p, p, i64, p, p, p, p, p, p, p, p, i, p, sz,
                                     p]),
            "moe_grouped_linear_w4a4_ws_layout": (i, [i64, i64, i64, i32, i32, i, p]),
            "moe_grouped_linear": (i, [p, i, i64, i, p, p, i32, i64, p, p, i, p, i64, i, p, p, i32, p, i, i,
                                       p, sz, p]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().nvfp4_status_string(int(status)).decode()


def _check(status: int, call: str):
    if status != OK:
        raise NVFP4Error(status, call)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _workspace(nbytes: int, device, ws=None):
    if nbytes == 0:
        return None, 0
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.numel() * ws.element_size()


def nvfp4_scales_bytes(rows: int, cols: int, sf_layout: int) -> int:
    return int(lib().nvfp4_scales_bytes(rows, cols, sf_layout))


def nvfp4_quantize(x: torch.Tensor, gs_in: torch.Tensor | None = None, sf_layout: int = SF_ROWMAJOR,
                   codes=None, scales=None, gs_out=None, ws=None):
    """Quantize ``x [rows, cols]`` (fp32 or bf16) to ``(codes, scales, gs)`` on the device."""
    rows, cols = x.shape
    dev = x.device
    if codes is None:
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(nvfp4_scales_bytes(rows, cols, sf_layout), dtype=torch.uint8, device=dev)
    if gs_out is None:
        gs_out = torch.empty(1, dtype=torch.float32, device=dev)
    ws, wsb = _workspace(int(lib().nvfp4_quantize_workspace(rows, cols)), dev, ws)
    _check(lib().nvfp4_quantize(_ptr(x), _dtype_code(x), rows, cols, _ptr(gs_in), sf_layout, _ptr(codes),
                                _ptr(scales), _ptr(gs_out), _ptr(ws), wsb, _stream()), "nvfp4_quantize")
    return codes, scales, gs_out


def nvfp4_calibrate(w: torch.Tensor, x_calib: torch.Tensor, sf_layout: int = SF_ROWMAJOR, ws=None):
    """Activation-calibrated quantization of ``w [N, K]`` (fp32) from ``x_calib
    [S, K]`` (bf16).  Returns ``(codes, scales, gs, col_scale, err[9], alpha_idx)``:
    the quantized ``w * col_scale``; use it on activations divided by ``col_scale``."""
    N, K = w.shape
    S = x_calib.shape[0]
    dev = w.device
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty(nvfp4_scales_bytes(N, K, sf_layout), dtype=torch.uint8, device=dev)
    gs = torch.empty(1, dtype=torch.float32, device=dev)
    col = torch.empty(K, dtype=torch.float32, device=dev)
    err = torch.empty(9, dtype=torch.float32, device=dev)
    aidx = torch.empty(1, dtype=torch.int32, device=dev)
    ws, wsb = _workspace(int(lib().nvfp4_calibrate_workspace(N, K, S)), dev, ws)
    _check(lib().nvfp4_calibrate(_ptr(w), N, K, _ptr(x_calib), _dtype_code(x_calib), S, sf_layout, _ptr(codes),
                                 _ptr(scales), _ptr(gs), _ptr(col), _ptr(err), _ptr(aidx), _ptr(ws), wsb,
                                 _stream()), "nvfp4_calibrate")
    return codes, scales, gs, col, err, aidx


def nvfp4_rms_norm(x: torch.Tensor, cols: int | None = None, y=None):
    """``bf16(v / sqrt(mean(v^2)))`` for the first ``cols`` columns of each row v of
    ``x [rows, ld]`` (fp32 or bf16, rows contiguous); returns ``y [rows, cols]`` bf16."""
    rows, ld = x.shape
    if x.stride(1) != 1 or x.stride(0) != ld:
        raise ValueError("x must be a contiguous [rows, ld] tensor")
    cols = ld if cols is None else int(cols)
    if y is None:
        y = torch.empty((rows, cols), dtype=torch.bfloat16, device=x.device)
    _check(lib().nvfp4_rms_norm(_ptr(x), _dtype_code(x), rows, cols, ld, _ptr(y), _stream()), "nvfp4_rms_norm")
    return y


def nvfp4_rms_norm_quant(x: torch.Tensor, cols: int | None = None, sf_layout: int = SF_TILED, ws=None):
    """NVFP4 ``(codes, scales, gs)`` of ``nvfp4_rms_norm(x, cols)``, without the bf16 rows."""
    rows, ld = x.shape
    if x.stride(1) != 1 or x.stride(0) != ld:
        raise ValueError("x must be a contiguous [rows, ld] tensor")
    cols = ld if cols is None else int(cols)
    dev = x.device
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty(nvfp4_scales_bytes(rows, cols, sf_layout), dtype=torch.uint8, device=dev)
    gs = torch.empty(1, dtype=torch.float32, device=dev)
    ws, wsb = _workspace(int(lib().nvfp4_rms_norm_quant_workspace(rows)), dev, ws)
    _check(lib().nvfp4_rms_norm_quant(_ptr(x), _dtype_code(x), rows, cols, ld, sf_layout, _ptr(codes), _ptr(scales),
                                      _ptr(gs), _ptr(ws), wsb, _stream()), "nvfp4_rms_norm_quant")
    return codes, scales, gs


def nvfp4_silu_mul(g: torch.Tensor, h=None):
    """``bf16(silu(g[:, :n]) * g[:, n:])`` for ``g [rows, 2n]`` (fp32 or bf16, contiguous)."""
    rows, w = g.shape
    if not g.is_contiguous() or w % 2:
        raise ValueError("g must be a contiguous [rows, 2n] tensor")
    half = w // 2
    if h is None:
        h = torch.empty((rows, half), dtype=torch.bfloat16, device=g.device)
    _check(lib().nvfp4_silu_mul(_ptr(g), _dtype_code(g), rows, half, _ptr(h), _stream()), "nvfp4_silu_mul")
    return h


def nvfp4_linear(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, w_gs: torch.Tensor,
                 w_sf_layout: int = SF_ROWMAJOR, y=None, y_dtype=torch.float32, mode: int = MODE_AUTO, ws=None):
    """``y = x @ W^T`` with W NVFP4 ``(w_codes [N, K/2], w_scales, w_gs)``; x bf16 [M, K]."""
    M, K = x.shape
    N = w_codes.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=x.device)
    ws, wsb = _workspace(int(lib().nvfp4_linear_workspace(M, K, N, mode)), x.device, ws)
    _check(lib().nvfp4_linear(_ptr(x), _dtype_code(x), M, K, _ptr(w_codes), _ptr(w_scales), w_sf_layout,
                              _ptr(w_gs), N, _ptr(y), _dtype_code(y), mode, _ptr(ws), wsb, _stream()),
           "nvfp4_linear")
    return y


def nvfp4_linear_w4a4q(x_codes: torch.Tensor, x_scales: torch.Tensor, x_gs: torch.Tensor, w_codes: torch.Tensor,
                       w_scales: torch.Tensor, w_gs: torch.Tensor, y=None, y_dtype=torch.bfloat16):
    """W4A4 with pre-quantized activations (codes [M, K/2], TILED scales, device gs)."""
    M, K = x_codes.shape[0], x_codes.shape[1] * 2
    N = w_codes.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=x_codes.device)
    _check(lib().nvfp4_linear_w4a4q(_ptr(x_codes), _ptr(x_scales), _ptr(x_gs), M, K, _ptr(w_codes), _ptr(w_scales),
                                    _ptr(w_gs), N, _ptr(y), _dtype_code(y), _stream()), "nvfp4_linear_w4a4q")
    return y


def chain_ops(specs) -> "ctypes.Array":
    """Build the ``nvfp4_chain_op`` array from dicts with keys ``w`` = (codes,
    TILED scales, gs), ``src`` (a bf16 tensor [M, K] or the index of an earlier
    op), ``K`` (when ``src`` is an op index: the columns the transform reads),
    ``xform``, ``y`` (tensor or None) and ``y_xform``."""
    arr = (ChainOp * len(specs))()
    for i, sp in enumerate(specs):
        c, sc, g = sp["w"]
        o = arr[i]
        o.w_codes, o.w_scales, o.w_gs = c.data_ptr(), sc.data_ptr(), g.data_ptr()
        o.N, o.K = c.shape[0], c.shape[1] * 2
        src = sp["src"]
        if hasattr(src, "data_ptr"):
            o.src, o.src_op, o.x, o.x_ld = CHAIN_SRC_X, -1, src.data_ptr(), src.stride(0)
        else:
            o.src, o.src_op, o.x, o.x_ld = CHAIN_SRC_OP, int(src), None, 0
        o.xform = int(sp.get("xform", CHAIN_XFORM_NONE))
        y = sp.get("y")
        o.y = None if y is None else y.data_ptr()
        o.y_dtype = DTYPE_F32 if y is None else _dtype_code(y)
        o.y_xform = int(sp.get("y_xform", CHAIN_XFORM_NONE))
    return arr


def nvfp4_chain(specs, M: int, ws=None, ops=None):
    """Run a list of W4A16 decode linears in one persistent launch per 12 ops
    (see ``nvfp4_chain`` in include/nvfp4.h).  Outputs go to the ``y`` tensors
    of the specs.  ``ops`` may pass a prebuilt :func:`chain_ops` array."""
    if ops is None:
        ops = chain_ops(specs)
    n = len(ops)
    dev = torch.device("cuda", torch.cuda.current_device())
    optr = ctypes.cast(ops, ctypes.c_void_p)
    ws, wsb = _workspace(int(lib().nvfp4_chain_workspace(optr, n, M)), dev, ws)
    _check(lib().nvfp4_chain(optr, n, M, _ptr(ws), wsb, _stream()), "nvfp4_chain")
    return ws


def moe_route_topk(h: torch.Tensor, w_router: torch.Tensor, k: int, logit_bias=None, want_logits: bool = False,
                   out=None, ws=None):
    """Router, top-k and permutation.  Returns a dict of device tensors:
    ``logits`` (if wanted), ``topk_idx``, ``topk_w``, ``expert_offsets``, ``perm_tok``, ``perm_slot``, ``row_of``."""
    T, H = h.shape
    E = w_router.shape[0]
    dev = h.device
    o = dict(out or {})
    if want_logits and "logits" not in o:
        o["logits"] = torch.empty((T, E), dtype=torch.float32, device=dev)
    o.setdefault("topk_idx", torch.empty((T, k), dtype=torch.int32, device=dev))
    o.setdefault("topk_w", torch.empty((T, k), dtype=torch.float32, device=dev))
    o.setdefault("expert_offsets", torch.empty(E + 1, dtype=torch.int32, device=dev))
    o.setdefault("perm_tok", torch.empty(T * k, dtype=torch.int32, device=dev))
    o.setdefault("perm_slot", torch.empty(T * k, dtype=torch.int32, device=dev))
    o.setdefault("row_of", torch.empty((T, k), dtype=torch.int32, device=dev))
    ws, wsb = _workspace(int(lib().moe_route_topk_workspace(T, E, k)), dev, ws)
    _check(lib().moe_route_topk(_ptr(h), _ptr(w_router), _ptr(logit_bias), T, H, E, k, _ptr(o.get("logits")),
                                _ptr(o["topk_idx"]), _ptr(o["topk_w"]), _ptr(o["expert_offsets"]),
                                _ptr(o["perm_tok"]), _ptr(o["perm_slot"]), _ptr(o["row_of"]), _ptr(ws), wsb,
                                _stream()), "moe_route_topk")
    return o


def moe_route_topk_noalloc(h: torch.Tensor, w_router: torch.Tensor, k: int, logit_bias=None,
                           want_logits: bool = False, out=None):
    """``moe_route_topk`` without a workspace: for callers that cannot allocate
    device memory while routing.  The library's built-in 1 MiB scratch is used
    instead (shared by every call; overlapping calls race)."""
    T, H = h.shape
    E = w_router.shape[0]
    dev = h.device
    o = dict(out or {})
    if want_logits and "logits" not in o:
        o["logits"] = torch.empty((T, E), dtype=torch.float32, device=dev)
    o.setdefault("topk_idx", torch.empty((T, k), dtype=torch.int32, device=dev))
    o.setdefault("topk_w", torch.empty((T, k), dtype=torch.float32, device=dev))
    o.setdefault("expert_offsets", torch.empty(E + 1, dtype=torch.int32, device=dev))
    o.setdefault("perm_tok", torch.empty(T * k, dtype=torch.int32, device=dev))
    o.setdefault("perm_slot", torch.empty(T * k, dtype=torch.int32, device=dev))
    o.setdefault("row_of", torch.empty((T, k), dtype=torch.int32, device=dev))
    _check(lib().moe_route_topk_noalloc(_ptr(h), _ptr(w_router), _ptr(logit_bias), T, H, E, k,
                                        _ptr(o.get("logits")), _ptr(o["topk_idx"]), _ptr(o["topk_w"]),
                                        _ptr(o["expert_offsets"]), _ptr(o["perm_tok"]), _ptr(o["perm_slot"]),
                                        _ptr(o["row_of"]), _stream()), "moe_route_topk_noalloc")
    return o


def moe_grouped_linear(x: torch.Tensor, expert_offsets: torch.Tensor, w_codes: torch.Tensor,
                       w_scales: torch.Tensor, w_gs: torch.Tensor, R: int, perm_tok=None, gather: bool = True,
                       w_sf_layout: int = SF_ROWMAJOR, epilogue: int = EPI_NONE, topk_w=None, row_of=None,
                       k: int = 0, y=None, y_dtype=torch.float32, mode: int = MODE_AUTO, ws=None):
    """Expert linears over permuted rows; see ``moe_grouped_linear`` in ``include/nvfp4.h``."""
    K = x.shape[1]
    E, N = w_codes.shape[0], w_codes.shape[1]
    if y is None:
        if epilogue == EPI_SWIGLU:
            shape = (R, N // 2)
        elif epilogue == EPI_COMBINE:
            shape = (R // k, N)
        else:
            shape = (R, N)
        y = torch.empty(shape, dtype=y_dtype, device=x.device)
    ws, wsb = _workspace(int(lib().moe_grouped_linear_workspace(R, K, N, E, k, epilogue, mode)), x.device, ws)
    _check(lib().moe_grouped_linear(_ptr(x), _dtype_code(x), K, int(gather), _ptr(expert_offsets),
                                    _ptr(perm_tok), E, R, _ptr(w_codes), _ptr(w_scales), w_sf_layout, _ptr(w_gs),
                                    N, epilogue, _ptr(topk_w), _ptr(row_of), k, _ptr(y), _dtype_code(y), mode,
                                    _ptr(ws), wsb, _stream()), "moe_grouped_linear")
    return y


def moe_layer_decode(h: torch.Tensor, w_router: torch.Tensor, k: int, gate_up, down, logit_bias=None,
                     y=None, y_dtype=torch.float32, want_logits: bool = False, want_routing: bool = False,
                     want_a: bool = False, ws=None):
    """One expert layer for a decode batch (T <= 32): ``gate_up`` and ``down`` are
    the stacked ``(codes, TILED scales, gs)`` of the experts.  Returns ``y``, or
    ``(y, extras)`` with the requested ``logits``, ``topk_idx``/``topk_w`` and ``a``."""
    T, H = h.shape
    E = w_router.shape[0]
    I = gate_up[0].shape[1] // 2
    dev = h.device
    if y is None:
        y = torch.empty((T, H), dtype=y_dtype, device=dev)
    ex = {}
    if want_logits:
        ex["logits"] = torch.empty((T, E), dtype=torch.float32, device=dev)
    if want_routing:
        ex["topk_idx"] = torch.empty((T, k), dtype=torch.int32, device=dev)
        ex["topk_w"] = torch.empty((T, k), dtype=torch.float32, device=dev)
    if want_a:
        ex["a"] = torch.empty((T * k, I), dtype=torch.bfloat16, device=dev)
    ws, wsb = _workspace(int(lib().moe_layer_decode_workspace(T, H, I, E, k)), dev, ws)
    _check(lib().moe_layer_decode(_ptr(h), _ptr(w_router), _ptr(logit_bias), T, H, E, k, _ptr(gate_up[0]),
                                  _ptr(gate_up[1]), _ptr(gate_up[2]), I, _ptr(down[0]), _ptr(down[1]),
                                  _ptr(down[2]), _ptr(ex.get("logits")), _ptr(ex.get("topk_idx")),
                                  _ptr(ex.get("topk_w")), _ptr(ex.get("a")), _ptr(y), _dtype_code(y), _ptr(ws),
                                  wsb, _stream()), "moe_layer_decode")
    return (y, ex) if ex else y

# ---- rotary positions, the paged key-value cache, attention of one new token -------


# These calls are made once per layer and step, so their enqueue time counts: the current
# stream's handle and device come from the functions under the public ones (3 us for the
# Stream object that torch.cuda.current_stream builds, 0.1 us here), and sizes are passed
# to torch.empty one by one (a tuple costs it 0.7 us more).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(dev: torch.device, name: str, args: tuple):
    """Call a C entry point on ``dev``'s current stream (made the current device for
    the call when it is not)."""
    index = dev.index
    if index != _current_device():
        with torch.cuda.device(dev):
            return _launch(dev, name, args)
    status = getattr(_lib or lib(), name)(*args, _raw_stream(index))
    if status != OK:
        raise NVFP4Error(status, name)


def _heads_view(t: torch.Tensor, dev, what: str, T=None, heads=None, head_dim=None) -> int:
    """Row stride (elements) of a ``[rows, heads, head_dim]`` view on ``dev`` whose heads
    are packed, as a slice of fused QKV rows is."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{what} must be a [rows, heads, head_dim] view with packed heads")
    n, h, d = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and h > 1):
        raise ValueError(f"{what} must be a [rows, heads, head_dim] view with packed heads")
    if T is not None and (n != T or h != heads or d != head_dim):
        raise ValueError(f"{what} must have shape {(T, heads, head_dim)}, not {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{what} must be on {dev}, not {t.device}")
    return s0 if n > 1 else h * d


def _vector(t: torch.Tensor, dtype, n: int | None, dev, what: str) -> int:
    """Address of a contiguous tensor of ``n`` elements of ``dtype`` on ``dev``."""
    if t.dtype != dtype or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{what} must be a contiguous {dtype} tensor" + (f" of {n} elements" if n is not None else ""))
    if t.device != dev:
        raise ValueError(f"{what} must be on {dev}, not {t.device}")
    return t.data_ptr()


def _cuda(t: torch.Tensor, what: str) -> torch.device:
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    return t.device


class KVCache:
    """A paged key-value cache: the device memory ``data`` (uint8, contiguous, a whole
    number of pages) with its shape, format and the fp32 global scales of the keys
    and values (one-element tensors; not used by ``KV_BF16``).

    The calls use the tensors given here, which the object keeps alive: its attributes
    cannot be set again.  New values are copied into the tensors (``cache.k_gs.copy_``);
    other tensors make another ``KVCache``."""

    _FIXED = frozenset(("data", "k_gs", "v_gs", "num_pages", "page_size", "heads", "head_dim", "format", "device",
                        "_desc", "_ref"))

    def __setattr__(self, name, value):
        if name in self._FIXED and name in self.__dict__:
            raise AttributeError(f"{name} of a KVCache cannot be set: its calls use what it was made with")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._FIXED:
            raise AttributeError(f"{name} of a KVCache cannot be deleted: its calls use what it was made with")
        object.__delattr__(self, name)

    def __init__(self, data: torch.Tensor, page_size: int, heads: int, head_dim: int, format: int, k_gs=None,
                 v_gs=None):
        page = nvfp4_kv_cache_bytes(1, page_size, heads, head_dim, format)
        if page == 0:
            raise ValueError("page_size, heads, head_dim or format out of range")
        dev = _cuda(data, "data")
        if data.dtype != torch.uint8 or not data.is_contiguous() or data.numel() == 0 or data.numel() % page:
            raise ValueError(f"data must be a contiguous uint8 tensor of whole pages ({page} bytes each)")
        if format == KV_BF16:
            k_gs = v_gs = None
        elif k_gs is None or v_gs is None:
            raise ValueError("this format needs k_gs and v_gs")
        self.data, self.k_gs, self.v_gs = data, k_gs, v_gs
        self.num_pages, self.page_size, self.heads = data.numel() // page, int(page_size), int(heads)
        self.head_dim, self.format, self.device = int(head_dim), int(format), dev
        self._desc = KvCacheDesc(data.data_ptr(), None if k_gs is None else _vector(k_gs, torch.float32, 1, dev, "k_gs"),
                                 None if v_gs is None else _vector(v_gs, torch.float32, 1, dev, "v_gs"),
                                 self.num_pages, self.page_size, self.heads, self.head_dim, self.format)
        self._ref = ctypes.byref(self._desc)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, heads: int, head_dim: int, format: int, k_gs=None, v_gs=None,
              device="cuda"):
        n = nvfp4_kv_cache_bytes(num_pages, page_size, heads, head_dim, format)
        if n == 0:
            raise ValueError("num_pages, page_size, heads, head_dim or format out of range")
        return cls(torch.empty(n, dtype=torch.uint8, device=device), page_size, heads, head_dim, format, k_gs, v_gs)


def nvfp4_kv_cache_bytes(num_pages: int, page_size: int, heads: int, head_dim: int, format: int) -> int:
    return int(lib().nvfp4_kv_cache_bytes(num_pages, page_size, heads, head_dim, format))


def nvfp4_rope_freqs(rot_dim: int, theta: float = 10000.0, scaling: int = ROPE_SCALE_NONE, factor: float = 1.0,
                     original_len: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """Rotary frequencies in turns per token (fp64, on the CPU) and the magnitude of
    cos and sin: ``(freqs [rot_dim / 2], mscale)``."""
    if rot_dim < 2:
        raise NVFP4Error(ERR_SHAPE, "nvfp4_rope_freqs")
    f = torch.empty(int(rot_dim) // 2, dtype=torch.float64)
    m = ctypes.c_double(0.0)
    _check(lib().nvfp4_rope_freqs(rot_dim, theta, scaling, factor, original_len, beta_fast, beta_slow, f.data_ptr(),
                                  ctypes.byref(m)), "nvfp4_rope_freqs")
    return f, m.value


def nvfp4_rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, layout: int = ROPE_HALF,
               mscale: float = 1.0, inverse: bool = False, y=None, y_dtype=torch.bfloat16):
    """Rotary positions of ``x [T, heads, head_dim]`` (fp32 or bf16; a view of wider rows
    is read in place).  ``positions [T]`` int64, ``freqs`` from :func:`nvfp4_rope_freqs`
    on x's device.  ``y=x`` rotates in place.  Like the other calls it records nothing for
    autograd; ``inverse=True`` on a gradient of ``y`` is the gradient of ``x``."""
    dev = _cuda(x, "x")
    x_ld = _heads_view(x, dev, "x")
    T, heads, D = x.shape
    if y is None:
        y = torch.empty(T, heads, D, dtype=y_dtype, device=dev)
        y_ld = heads * D
    else:
        y_ld = _heads_view(y, dev, "y", T, heads, D)
    _launch(dev, "nvfp4_rope", (x.data_ptr(), _dtype_code(x), T, heads, D, x_ld,
            _vector(positions, torch.int64, T, dev, "positions"), _vector(freqs, torch.float64, None, dev, "freqs"),
            2 * freqs.numel(), layout, mscale, int(inverse), y.data_ptr(), _dtype_code(y), y_ld))
    return y


def nvfp4_kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor):
    """Write token t's keys and values (``[T, heads, head_dim]`` views, fp32 or bf16) to
    slot ``slots[t]`` (int64; page * page_size + offset; negative: skipped)."""
    dev = cache.device
    T, heads, D = k.shape[0], cache.heads, cache.head_dim
    k_ld, v_ld = _heads_view(k, dev, "k", T, heads, D), _heads_view(v, dev, "v", T, heads, D)
    if k.dtype != v.dtype:
        raise TypeError("k and v must have one dtype")
    _launch(dev, "nvfp4_kv_write", (cache._ref, k.data_ptr(), v.data_ptr(), _dtype_code(k), T, k_ld, v_ld,
            _vector(slots, torch.int64, T, dev, "slots")))


def nvfp4_kv_read(cache: KVCache, slots: torch.Tensor, k_out=None, v_out=None, y_dtype=torch.bfloat16):
    """The dequantized keys and values of ``slots [T]``: two ``[T, heads, head_dim]``
    tensors (bf16 or fp32); zeros for negative slots."""
    dev = cache.device
    T, heads, D = slots.numel(), cache.heads, cache.head_dim
    if k_out is None and v_out is None:
        k_out = torch.empty(T, heads, D, dtype=y_dtype, device=dev)
        v_out = torch.empty_like(k_out)
        k_ptr, v_ptr = k_out.data_ptr(), v_out.data_ptr()
    else:
        k_out = torch.empty(T, heads, D, dtype=v_out.dtype, device=dev) if k_out is None else k_out
        v_out = torch.empty(T, heads, D, dtype=k_out.dtype, device=dev) if v_out is None else v_out
        if k_out.dtype != v_out.dtype:
            raise TypeError("k_out and v_out must have one dtype")
        k_ptr = _vector(k_out, k_out.dtype, T * heads * D, dev, "k_out")
        v_ptr = _vector(v_out, v_out.dtype, T * heads * D, dev, "v_out")
    _launch(dev, "nvfp4_kv_read", (cache._ref, _vector(slots, torch.int64, T, dev, "slots"), T, k_ptr, v_ptr,
            _dtype_code(k_out)))
    return k_out, v_out


def nvfp4_rope_kv_write(cache: KVCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                        slots: torch.Tensor, freqs: torch.Tensor, layout: int = ROPE_HALF, mscale: float = 1.0,
                        q_out=None):
    """Rotate queries and keys and write the rotated keys and the values to the cache in
    one pass over the QKV rows; returns the rotated queries ``[T, q_heads, head_dim]``
    (bf16).  Same bits as :func:`nvfp4_rope` and :func:`nvfp4_kv_write`."""
    dev = cache.device
    T, q_heads, heads, D = q.shape[0], q.shape[1], cache.heads, cache.head_dim
    q_ld = _heads_view(q, dev, "q", T, q_heads, D)
    k_ld, v_ld = _heads_view(k, dev, "k", T, heads, D), _heads_view(v, dev, "v", T, heads, D)
    if q.dtype != k.dtype or k.dtype != v.dtype:
        raise TypeError("q, k and v must have one dtype")
    if q_out is None:
        q_out = torch.empty(T, q_heads, D, dtype=torch.bfloat16, device=dev)
    _launch(dev, "nvfp4_rope_kv_write", (cache._ref, q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(q), T,
            q_heads, q_ld, k_ld, v_ld, _vector(positions, torch.int64, T, dev, "positions"),
            _vector(slots, torch.int64, T, dev, "slots"), _vector(freqs, torch.float64, None, dev, "freqs"),
            2 * freqs.numel(), layout, mscale,
            _vector(q_out, torch.bfloat16, T * q_heads * D, dev, "q_out")))
    return q_out


def nvfp4_attn_decode_workspace(cache: KVCache, B: int, q_heads: int, max_pages: int) -> int:
    return int(lib().nvfp4_attn_decode_workspace(cache._ref, B, q_heads, max_pages))


def nvfp4_attn_decode(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor, scale=None,
                      window: int = 0, y=None, y_dtype=torch.bfloat16, want_lse: bool = False, ws=None):
    """Attention of one new token per sequence: ``q [B, q_heads, head_dim]`` (bf16 view)
    over the paged cache.  ``page_table [B, max_pages]`` and ``seq_lens [B]`` int32;
    ``scale`` defaults to ``head_dim ** -0.5``.  Returns ``y [B, q_heads, head_dim]``,
    or ``(y, lse [B, q_heads])``.  Short batches are faster with a narrow table (a slice
    ``table[:, :n]`` is taken in place): the work is split by its width."""
    dev = cache.device
    B, q_heads, D = q.shape[0], q.shape[1], cache.head_dim
    q_ld = _heads_view(q, dev, "q", B, q_heads, D)
    if q.dtype != torch.bfloat16:
        raise TypeError(f"q must be bfloat16, not {q.dtype}")
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != B or \
            page_table.stride(1) != 1 or page_table.device != dev:
        raise ValueError(f"page_table must be an int32 [{B}, max_pages] tensor on {dev} with contiguous rows")
    max_pages = page_table.shape[1]
    table_ld = page_table.stride(0) if B > 1 else max_pages
    if y is None:
        y = torch.empty(B, q_heads, D, dtype=y_dtype, device=dev)
        y_ptr = y.data_ptr()
    else:
        y_ptr = _vector(y, y.dtype, B * q_heads * D, dev, "y")
    lse = torch.empty((B, q_heads), dtype=torch.float32, device=dev) if want_lse else None
    if ws is None:
        ws = torch.empty(nvfp4_attn_decode_workspace(cache, B, q_heads, max_pages), dtype=torch.uint8, device=dev)
    elif ws.device != dev or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous tensor on {dev}")
    _launch(dev, "nvfp4_attn_decode", (q.data_ptr(), B, q_heads, q_ld, cache._ref, page_table.data_ptr(), max_pages,
            table_ld, _vector(seq_lens, torch.int32, B, dev, "seq_lens"), D ** -0.5 if scale is None else scale, window,
            y_ptr, _dtype_code(y), None if lse is None else lse.data_ptr(), ws.data_ptr(),
            ws.numel() * ws.element_size()))
    return y if lse is None else (y, lse)


def nvfp4_linear_w4a4_ws_layout(M: int, K: int) -> dict:
    """Byte offsets, inside a W4A4 ``nvfp4_linear`` workspace, of the quantized
    activations the call leaves there: ``gs_x``, ``codes``, ``scales``."""
    out = (ctypes.c_int64 * 3)()
    _check(lib().nvfp4_linear_w4a4_ws_layout(M, K, out), "nvfp4_linear_w4a4_ws_layout")
    return dict(zip(("gs_x", "codes", "scales"), (int(v) for v in out)))


def moe_grouped_linear_w4a4_ws_layout(R: int, K: int, N: int, E: int, k: int, epilogue: int) -> dict:
    """Byte offsets, inside a W4A4 ``moe_grouped_linear`` workspace, of the padded
    permuted activations the call leaves there (see include/nvfp4.h)."""
    out = (ctypes.c_int64 * 6)()
    _check(lib().moe_grouped_linear_w4a4_ws_layout(R, K, N, E, k, epilogue, out),
           "moe_grouped_linear_w4a4_ws_layout")
    return dict(zip(("gs_x", "pad_off", "src_rows", "codes", "scales", "rows_pad"), (int(v) for v in out)))


def nvfp4_debug_wait_timeout(limit_cycles: int):
    """Launch the library's wait-timeout probe (a bounded wait that runs out)."""
    _check(lib().nvfp4_debug_wait_timeout(int(limit_cycles), _stream()), "nvfp4_debug_wait_timeout")


def nvfp4_read_device_status() -> int:
    st = ctypes.c_int(0)
    _check(lib().nvfp4_read_device_status(_stream(), ctypes.byref(st)), "nvfp4_read_device_status")
    return st.value
