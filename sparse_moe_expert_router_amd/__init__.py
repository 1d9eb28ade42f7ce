"""Python binding of libmoe.so, the gfx950 HIP library for one sparse MoE FFN layer forward.

Argument marshalling only: every step of the layer runs in the library's HIP kernels.  Tensors
are torch tensors on the GPU (torch supplies device memory and the current stream).  There is no
fallback: if libmoe.so is missing, or a call returns an error status, this module raises.

The C ABI is declared and documented in include/moe.h; names here match it.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# MOE_SANITIZE=1 loads the build whose host code carries AddressSanitizer / UBSan checks
LIB_PATH = os.path.join(_PKG, "libmoe_san.so" if os.environ.get("MOE_SANITIZE") == "1" else "libmoe.so")

X_F32, X_BF16, X_MX4, X_F64 = 0, 1, 2, 3
W_Q8_0, W_I8_ROW, W_E2M1_G16, W_Q8_0_TILED, W_I8_ROW_TILED = 0, 1, 2, 3, 4
W_FP8_ROW, W_FP8_ROW_TILED = 5, 6
W_MX4 = 8
ACT_SWIGLU, ACT_RELU2, ACT_NONE = 0, 1, 2
F_ZERO_SKIP, F_PREFILL_I8, F_PREFILL_FP8, F_PREFILL_MX4 = 1, 4, 8, 16
OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP, ESCRATCH = 0, -1, -2, -3, -4, -5
STATIC_WORKSPACE_BYTES = 64 << 20       # MOE_STATIC_WORKSPACE_BYTES: the buffer of layer_forward_static

EXPORTED = ("moe_workspace_bytes", "moe_route_workspace_bytes", "moe_route", "moe_permute",
            "moe_layer_forward", "moe_layer_forward_static", "moe_experts_forward", "moe_quantize_rows_i8", "moe_quantize_rows_fp8",
            "moe_repack_experts", "moe_read_intermediates", "moe_quantize_rows_mx4", "moe_matmul_mx4",
            "moe_balance_workspace_bytes", "moe_balance_loss", "moe_balance_loss_backward",
            "moe_status_str", "moe_abi_version", "moe_profile_enable", "moe_profile_collect",
            "moe_profile_reset", "moe_profile_kinds", "moe_profile_get")


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn} failed: {msg} ({status})")
        self.status = status


class Experts(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("E", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("gate_up", ctypes.c_void_p),
                ("gate_up_scales", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("down_scales", ctypes.c_void_p), ("n_shared", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python sparse_moe_expert_router_amd/build.py` (hipcc, gfx950)")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
        pex = ctypes.POINTER(Experts)
        L.moe_workspace_bytes.argtypes = [i32, i32, pex, i32, u32]
        L.moe_workspace_bytes.restype = sz
        L.moe_route_workspace_bytes.argtypes = [i32, i32]
        L.moe_route_workspace_bytes.restype = sz
        L.moe_route.argtypes = [vp, i32, i32, i32, vp, vp, i32, i32, vp, vp, vp, sz, vp]
        L.moe_route.restype = i32
        L.moe_permute.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, vp]
        L.moe_permute.restype = i32
        L.moe_layer_forward.argtypes = [vp, i32, i32, vp, vp, pex, i32, i32, u32, vp, vp, vp, vp,
                                        sz, vp]
        L.moe_layer_forward.restype = i32
        L.moe_layer_forward_static.argtypes = [vp, i32, i32, vp, vp, pex, i32, i32, u32, vp, vp, vp, vp]
        L.moe_layer_forward_static.restype = i32
        L.moe_experts_forward.argtypes = [vp, i32, i32, vp, vp, pex, i32, i32, u32, vp, vp, sz, vp]
        L.moe_experts_forward.restype = i32
        L.moe_repack_experts.argtypes = [pex, i32, pex, vp]
        L.moe_repack_experts.restype = i32
        L.moe_quantize_rows_i8.argtypes = [vp, i32, i32, i32, vp, vp, vp]
        L.moe_quantize_rows_i8.restype = i32
        L.moe_quantize_rows_fp8.argtypes = [vp, i32, i32, i32, vp, vp, vp]
        L.moe_quantize_rows_fp8.restype = i32
        L.moe_quantize_rows_mx4.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp]
        L.moe_quantize_rows_mx4.restype = i32
        L.moe_matmul_mx4.argtypes = [vp, vp, i32, i32, i32, vp, i32, i32, vp, vp, i32, i32, vp, i32, vp, vp, i32, vp]
        L.moe_matmul_mx4.restype = i32
        L.moe_balance_workspace_bytes.argtypes = [i32, i32]
        L.moe_balance_workspace_bytes.restype = sz
        L.moe_balance_loss.argtypes = [vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, sz, vp]
        L.moe_balance_loss.restype = i32
        L.moe_balance_loss_backward.argtypes = [vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, i32, vp]
        L.moe_balance_loss_backward.restype = i32
        L.moe_read_intermediates.argtypes = [i32, i32, pex, i32, u32, i32, vp, sz, vp, vp, vp, vp]
        L.moe_read_intermediates.restype = i32
        L.moe_status_str.argtypes = [i32]
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_abi_version.restype = i32
        L.moe_profile_enable.argtypes = [i32]
        L.moe_profile_enable.restype = i32
        L.moe_profile_collect.restype = i32
        L.moe_profile_reset.restype = None
        L.moe_profile_kinds.restype = i32
        L.moe_profile_get.argtypes = [i32, ctypes.POINTER(ctypes.c_char_p),
                                      ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_double)]
        L.moe_profile_get.restype = i32
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != OK:
        raise MoeError(fn, status, lib().moe_status_str(status).decode())


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _xtype(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return X_BF16
    if x.dtype == torch.float32:
        return X_F32
    raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")


def experts_struct(ex: dict) -> Experts:
    """The C struct for an experts dict (fmt, E, d_model, d_ff, four device tensors, n_shared)."""
    return Experts(int(ex["fmt"]), int(ex["E"]), int(ex["d_model"]), int(ex["d_ff"]),
                   ex["gate_up"].data_ptr(), ex["gate_up_scales"].data_ptr(),
                   ex["down"].data_ptr(), ex["down_scales"].data_ptr(), int(ex.get("n_shared", 0)))


def workspace_bytes(T: int, k: int, experts: dict, act: int, flags: int = 0) -> int:
    s = Experts(int(experts["fmt"]), int(experts["E"]), int(experts["d_model"]),
                int(experts["d_ff"]), None, None, None, None, int(experts.get("n_shared", 0)))
    return int(lib().moe_workspace_bytes(T, k, ctypes.byref(s), act, flags))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def route(x, w_router, bias, k: int, ws=None):
    """moe_route: (topk_idx int32 [T,k], topk_w fp32 [T,k])."""
    T, d = x.shape
    E = w_router.shape[0]
    need = int(lib().moe_route_workspace_bytes(T, E))
    ws = alloc_workspace(need, x.device) if ws is None else ws
    idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
    w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    _check("moe_route", lib().moe_route(_p(x), _xtype(x), T, d, _p(w_router), _p(bias), E, k,
                                        _p(idx), _p(w), _p(ws), ws.numel(), _stream()))
    return idx, w


def permute(topk_idx, E: int):
    """moe_permute: (counts [E], offsets [E+1], perm [P], inv [P]), all int32."""
    T, k = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty(T * k, dtype=torch.int32, device=dev)
    _check("moe_permute", lib().moe_permute(_p(topk_idx), T, k, E, _p(counts), _p(offsets),
                                            _p(perm), _p(inv), _stream()))
    return counts, offsets, perm, inv


def layer_forward(x, w_router, bias, experts: dict, k: int, act: int, flags: int = 0, out=None,
                  ws=None, want_routing: bool = False):
    """moe_layer_forward: out fp32 [T, d_model] (and the routing if want_routing)."""
    T = x.shape[0]
    s = experts_struct(experts)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(T, k, experts, act, flags), x.device)
    out = torch.empty((T, int(experts["d_model"])), dtype=torch.float32, device=x.device) \
        if out is None else out
    idx = w = None
    if want_routing:
        idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
        w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    _check("moe_layer_forward",
           lib().moe_layer_forward(_p(x), _xtype(x), T, _p(w_router), _p(bias), ctypes.byref(s), k,
                                   act, flags, _p(out), _p(idx), _p(w), _p(ws), ws.numel(),
                                   _stream()))
    return (out, idx, w) if want_routing else out


def layer_forward_static(x, w_router, bias, experts: dict, k: int, act: int, flags: int = 0, out=None,
                         want_routing: bool = False):
    """moe_layer_forward_static: moe_layer_forward on the library's static device buffer (no
    workspace argument; the library allocates nothing).  Calls on one GPU must not overlap."""
    T = x.shape[0]
    s = experts_struct(experts)
    out = torch.empty((T, int(experts["d_model"])), dtype=torch.float32, device=x.device) \
        if out is None else out
    idx = w = None
    if want_routing:
        idx = torch.empty((T, k), dtype=torch.int32, device=x.device)
        w = torch.empty((T, k), dtype=torch.float32, device=x.device)
    _check("moe_layer_forward_static",
           lib().moe_layer_forward_static(_p(x), _xtype(x), T, _p(w_router), _p(bias), ctypes.byref(s), k,
                                          act, flags, _p(out), _p(idx), _p(w), _stream()))
    return (out, idx, w) if want_routing else out


def experts_forward(x, topk_idx, topk_w, experts: dict, act: int, flags: int = 0, out=None,
                    ws=None):
    """moe_experts_forward: out fp32 [T, d_model] for a given routing."""
    T, k = topk_idx.shape
    s = experts_struct(experts)
    if ws is None:
        ws = alloc_workspace(workspace_bytes(T, k, experts, act, flags), x.device)
    out = torch.empty((T, int(experts["d_model"])), dtype=torch.float32, device=x.device) \
        if out is None else out
    _check("moe_experts_forward",
           lib().moe_experts_forward(_p(x), _xtype(x), T, _p(topk_idx), _p(topk_w),
                                     ctypes.byref(s), k, act, flags, _p(out), _p(ws), ws.numel(),
                                     _stream()))
    return out


def repack_experts(experts: dict, act: int) -> dict:
    """moe_repack_experts: a tiled copy (new device tensors) of plain Q8_0 / I8_ROW / FP8_ROW experts."""
    fmt = int(experts["fmt"])
    tiled = {W_Q8_0: W_Q8_0_TILED, W_I8_ROW: W_I8_ROW_TILED, W_FP8_ROW: W_FP8_ROW_TILED}[fmt]
    out = dict(experts)
    out["fmt"] = tiled
    for key in ("gate_up", "gate_up_scales", "down", "down_scales"):
        out[key] = torch.empty_like(experts[key])
    src, dst = experts_struct(experts), experts_struct(out)
    _check("moe_repack_experts", lib().moe_repack_experts(ctypes.byref(src), act, ctypes.byref(dst),
                                                          _stream()))
    return out


def quantize_rows_i8(v):
    """moe_quantize_rows_i8: (q int8 [rows, cols], scale fp32 [rows])."""
    rows, cols = v.shape
    q = torch.empty((rows, cols), dtype=torch.int8, device=v.device)
    scale = torch.empty(rows, dtype=torch.float32, device=v.device)
    _check("moe_quantize_rows_i8", lib().moe_quantize_rows_i8(_p(v), _xtype(v), rows, cols, _p(q),
                                                              _p(scale), _stream()))
    return q, scale


def quantize_rows_fp8(v):
    """moe_quantize_rows_fp8: (q uint8 E4M3 codes [rows, cols], scale fp32 [rows])."""
    rows, cols = v.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=v.device)
    scale = torch.empty(rows, dtype=torch.float32, device=v.device)
    _check("moe_quantize_rows_fp8", lib().moe_quantize_rows_fp8(_p(v), _xtype(v), rows, cols, _p(q),
                                                                _p(scale), _stream()))
    return q, scale


# ---- MX4 operators and the router's training losses.  These check their tensors here (type, shape,
# device, contiguity) and run on the current stream of the tensors' device.

_XTYPES = {torch.float32: X_F32, torch.bfloat16: X_BF16, torch.float64: X_F64}


def _need(name, t, dtypes, shape, dev):
    """Raises unless t is a contiguous tensor on GPU `dev` (an index) of one of `dtypes` and of `shape` (None: any)."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and (shape is None or t.shape == shape)
            and dev >= 0 and t.get_device() == dev and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")
    if dev < 0 or t.get_device() != dev:
        where = f"on GPU {dev}, where the call runs" if dev >= 0 else "on a GPU"
        raise ValueError(f"{name} must be {where}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _rows_of(name, t, dtypes):
    """As _need, for the 2-d tensor that decides the call's GPU, whose index it returns."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got {tuple(t.shape)}")
    dev = t.get_device()
    _need(name, t, dtypes, None, dev)
    return dev


def _run(fn, dev, *args):
    """Calls the library on GPU `dev`'s current stream, with `dev` the current device."""
    call = getattr(_lib or lib(), fn)
    if dev == torch.cuda.current_device():
        status = call(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = call(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status != OK:
        _check(fn, status)


_FLOATS = (torch.float32, torch.bfloat16)
_LOGITS = (torch.float32, torch.bfloat16, torch.float64)
_U8, _I32, _F32 = (torch.uint8,), (torch.int32,), (torch.float32,)
_MASK = (torch.bool, torch.uint8)


def quantize_rows_mx4(v, want_values: bool = False):
    """moe_quantize_rows_mx4: (q uint8 [rows, cols/2], scale uint8 [rows, cols/32]) of v [rows, cols]
    (float32 or bfloat16); with want_values also the values they stand for, in v's type."""
    dev = _rows_of("v", v, _FLOATS)
    rows, cols = v.shape
    q = v.new_empty((rows, cols // 2), dtype=torch.uint8)
    scale = v.new_empty((rows, cols // 32), dtype=torch.uint8)
    values = torch.empty_like(v) if want_values else None
    _run("moe_quantize_rows_mx4", dev, v.data_ptr(), _XTYPES[v.dtype], rows, cols, q.data_ptr(), scale.data_ptr(),
         values.data_ptr() if want_values else None)
    return (q, scale, values) if want_values else (q, scale)


def matmul_mx4(x, w, w_scales, x_scales=None, offsets=None, perm=None, k: int = 1, act: int = ACT_NONE,
               out_dtype=torch.bfloat16, out=None):
    """moe_matmul_mx4: out[r] = act(W[g] x[perm[r] // k]) for the rows r of group g.

    x [x_rows, K] float32 or bfloat16, or uint8 MX4 codes [x_rows, K/2] with x_scales; w uint8
    [E, N, K/2] and w_scales uint8 [E, N, K/32] ([N, ..] for one group); offsets int32 [E+1] (None:
    one group); perm int32 [rows] (None: row r reads x[r]).  out [rows, N] ([rows, N/2] with
    ACT_SWIGLU) of out_dtype; rows outside every group are left as they were (unset in a new
    tensor).  out_dtype uint8 (x in MX4 only) gives MX4 rows: a (codes, scales) pair."""
    dev = _rows_of("x", x, (torch.float32, torch.bfloat16, torch.uint8))
    mx = x.dtype == torch.uint8
    x_rows, K = x.shape
    if mx:
        K *= 2
        _need("x_scales", x_scales, _U8, (x_rows, K // 32), dev)
    elif x_scales is not None:
        raise ValueError("x_scales goes with x as MX4 codes only")
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError("w must be [E, N, K/2] or [N, K/2]")
    if w.dim() == 3:
        E, N, _ = w.shape
        _need("w", w, _U8, (E, N, K // 2), dev)
        _need("w_scales", w_scales, _U8, (E, N, K // 32), dev)
    else:
        E, N = 1, w.shape[0]
        _need("w", w, _U8, (N, K // 2), dev)
        _need("w_scales", w_scales, _U8, (N, K // 32), dev)
    if offsets is not None:
        _need("offsets", offsets, _I32, (E + 1,), dev)
    elif E != 1:
        raise ValueError("several groups need offsets")
    if perm is not None:
        _need("perm", perm, _I32, None, dev)
        if perm.dim() != 1:
            raise ValueError("perm must have one dimension")
    rows = x_rows if perm is None else perm.shape[0]
    cols = N // 2 if act == ACT_SWIGLU else N
    scales = None
    if out_dtype == torch.uint8:
        if out is None:
            out = (x.new_empty((rows, cols // 2), dtype=torch.uint8), x.new_empty((rows, cols // 32), dtype=torch.uint8))
        codes, scales = out
        _need("out[0]", codes, _U8, (rows, cols // 2), dev)
        _need("out[1]", scales, _U8, (rows, cols // 32), dev)
        otype, ptr, sptr = X_MX4, codes.data_ptr(), scales.data_ptr()
    else:
        if out_dtype not in _FLOATS:
            raise TypeError(f"out_dtype must be float32, bfloat16 or uint8, got {out_dtype}")
        if out is None:
            out = x.new_empty((rows, cols), dtype=out_dtype)
        else:
            _need("out", out, (out_dtype,), (rows, cols), dev)
        otype, ptr, sptr = _XTYPES[out_dtype], out.data_ptr(), None
    _run("moe_matmul_mx4", dev, x.data_ptr(), x_scales.data_ptr() if mx else None, X_MX4 if mx else _XTYPES[x.dtype],
         x_rows, K, None if perm is None else perm.data_ptr(), k, rows, w.data_ptr(), w_scales.data_ptr(), E, N,
         None if offsets is None else offsets.data_ptr(), act, ptr, sptr, otype)
    return out


def _batch(logits, topk_idx, mask):
    dev = _rows_of("logits", logits, _LOGITS)
    T, E = logits.shape
    _need("topk_idx", topk_idx, _I32, None, dev)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError(f"topk_idx must have the shape ({T}, k), got {tuple(topk_idx.shape)}")
    if mask is not None:
        _need("mask", mask, _MASK, (T,), dev)
    return dev, T, E, topk_idx.shape[1]


def balance_loss(logits, topk_idx, mask=None, ws=None):
    """moe_balance_loss: (loss fp32 [2] = balance loss and z loss, counts int32 [E], mean_prob fp32
    [E]) of router logits [T, E] (float32, bfloat16 or float64) and the selected ids [T, k]; mask
    [T] (bool or uint8): False for padding."""
    dev, T, E, k = _batch(logits, topk_idx, mask)
    if ws is not None:
        _need("ws", ws, _U8, None, dev)
        ws_ptr, ws_bytes, own = ws.data_ptr(), ws.numel(), 0
    else:
        ws_bytes = (_lib or lib()).moe_balance_workspace_bytes(T, E)
        own = ws_bytes if ws_bytes <= 4096 else 0    # a small workspace lies behind the results
        if not own:
            ws = topk_idx.new_empty(max(ws_bytes, 256), dtype=torch.uint8)
            ws_ptr = ws.data_ptr()
    # the results share one allocation, each from a 16-byte boundary on
    pad = -E % 4
    counts, _, mean_prob, _, loss, _, tail = topk_idx.new_empty(2 * (E + pad) + 4 + own // 4).split_with_sizes(
        [E, pad, E, pad, 2, 2, own // 4])
    if own:
        ws_ptr = tail.data_ptr()
    mean_prob, loss = mean_prob.view(torch.float32), loss.view(torch.float32)
    _run("moe_balance_loss", dev, logits.data_ptr(), _XTYPES[logits.dtype], T, E, topk_idx.data_ptr(), k,
         None if mask is None else mask.data_ptr(), loss.data_ptr(), counts.data_ptr(), mean_prob.data_ptr(),
         ws_ptr, ws_bytes)
    return loss, counts, mean_prob


def balance_loss_backward(logits, topk_idx, counts, d_loss, topk_w=None, d_topk_w=None, mask=None, grad_dtype=None):
    """moe_balance_loss_backward: d_logits [T, E] for the gradients d_loss fp32 [2] of the two losses
    and, with topk_w and d_topk_w fp32 [T, k], of the renormalised routing weights.  grad_dtype:
    float32 or bfloat16 (None: the logits' type, float32 for float64 logits)."""
    dev, T, E, k = _batch(logits, topk_idx, mask)
    _need("counts", counts, _I32, (E,), dev)
    _need("d_loss", d_loss, _F32, (2,), dev)
    if (topk_w is None) != (d_topk_w is None):
        raise ValueError("topk_w and d_topk_w go together")
    if topk_w is not None:
        _need("topk_w", topk_w, _F32, (T, k), dev)
        _need("d_topk_w", d_topk_w, _F32, (T, k), dev)
    if grad_dtype is None:
        grad_dtype = torch.float32 if logits.dtype == torch.float64 else logits.dtype
    if grad_dtype not in _FLOATS:
        raise TypeError(f"grad_dtype must be float32 or bfloat16, got {grad_dtype}")
    d_logits = torch.empty_like(logits, dtype=grad_dtype)
    _run("moe_balance_loss_backward", dev, logits.data_ptr(), _XTYPES[logits.dtype], T, E, topk_idx.data_ptr(), k,
         None if mask is None else mask.data_ptr(), counts.data_ptr(), d_loss.data_ptr(),
         None if topk_w is None else topk_w.data_ptr(), None if topk_w is None else d_topk_w.data_ptr(),
         d_logits.data_ptr(), _XTYPES[grad_dtype])
    return d_logits


def read_intermediates(T: int, k: int, experts: dict, act: int, flags: int, ws, with_router: bool = True):
    """moe_read_intermediates: the h (fp32 [T k + S T, d_ff], pair order) the last layer call on
    `ws` left there; with a prefill flag also (codes uint8 [rows, d_ff], row scales fp32 [rows])."""
    S = int(experts.get("n_shared", 0))
    rows, d_ff = T * k + S * T, int(experts["d_ff"])
    dev = ws.device
    h = torch.empty((rows, d_ff), dtype=torch.float32, device=dev)
    prefill = bool(flags & (F_PREFILL_I8 | F_PREFILL_FP8))
    hq = torch.empty((rows, d_ff), dtype=torch.uint8, device=dev) if prefill else None
    sh = torch.empty(rows, dtype=torch.float32, device=dev) if prefill else None
    s = experts_struct(experts)
    _check("moe_read_intermediates",
           lib().moe_read_intermediates(T, k, ctypes.byref(s), act, flags, 1 if with_router else 0, _p(ws),
                                        ws.numel(), _p(h), _p(hq), _p(sh), _stream()))
    return (h, hq, sh) if prefill else h


def profile_enable(on: bool = True) -> None:
    """Bracket every library kernel launch with HIP events (see include/moe.h)."""
    _check("moe_profile_enable", lib().moe_profile_enable(1 if on else 0))


def profile_reset() -> None:
    lib().moe_profile_reset()


def profile_collect() -> dict:
    """Wait for the recorded events; {kernel name: (launches, total ms)} since the last reset."""
    L = lib()
    _check("moe_profile_collect", L.moe_profile_collect())
    res = {}
    for kind in range(L.moe_profile_kinds()):
        name = ctypes.c_char_p()
        n = ctypes.c_int64()
        ms = ctypes.c_double()
        _check("moe_profile_get", L.moe_profile_get(kind, ctypes.byref(name), ctypes.byref(n),
                                                    ctypes.byref(ms)))
        if n.value:
            res[name.value.decode()] = (int(n.value), float(ms.value))
    return res
