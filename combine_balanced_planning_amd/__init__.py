"""MI355X-native balanced expert-parallel planning, dispatch and combine.

A thin ctypes binding of ``libmoon.so`` (C ABI in ``include/moon.h``).  The
functions carry the C names and only marshal arguments: tensors become device
pointers (after dtype / device / contiguity / size checks), the stream
defaults to torch's current stream.  Every step of the path runs in the HIP
kernels of the library; there is no fallback.  torch is imported first so
the library binds to the HIP runtime torch has already loaded.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoon.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
_lib = ctypes.CDLL(LIB_PATH)

MOON_OK = 0
MOON_ERR_INVALID_ARG = -1
MOON_ERR_TOPOLOGY = -2
MOON_ERR_UNSUPPORTED = -3
MOON_ERR_OOM = -4
MOON_ERR_HIP = -5
MOON_ERR_PLAN_MISMATCH = -6
MOON_ERR_BAD_EXPERT = -7
MOON_ERR_SLOT_BUDGET = -8
MOON_ERR_HISTOGRAM = -9
MOON_ERR_NOT_PLANNED = -10
MOON_ERR_INTERNAL = -11

MOON_COMBINE_WEIGHTED = 0x1
MOON_DISPATCH_FUSED_DUPS = 0x2  # the default dispatch, named explicitly
MOON_COMBINE_DUP_PROLOGUE = 0x4
MOON_DISPATCH_DEDUP_EPILOGUE = 0x8

MOON_DTYPE_F32 = 0
MOON_DTYPE_BF16 = 1
MOON_ROUTE_SIGMOID = 0x1
MOON_ROUTE_RENORM = 0x2

_i32, _u32, _vp = ctypes.c_int32, ctypes.c_uint32, ctypes.c_void_p


class moon_config(ctypes.Structure):
    _fields_ = [("R", _i32), ("E", _i32), ("K", _i32), ("S", _i32), ("H", _i32), ("B", _i32),
                ("token_padding", _i32), ("flags", _u32)]


class moon_layout(ctypes.Structure):
    _fields_ = [("N", _i32), ("NvS", _i32), ("NvS_padded", _i32), ("E_plus_B", _i32),
                ("B", _i32), ("hidden_windows", _vp), ("weight_windows", _vp)]


class moon_plan_arrays(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dst", "experts_to_copy", "zero_fill_ranges", "remote_stats",
                                   "dup_groups", "dup_loffs", "dup_counts", "cu_seqlens",
                                   "status")] + \
               [(n, _i32) for n in ("N", "R", "E", "B", "NvS", "K")] + \
               [("prefetch_index", _vp)]


class moon_weight_tensor(ctypes.Structure):
    _fields_ = [("experts", _vp), ("slots", _vp), ("row_bytes", ctypes.c_int64)]


class moon_grad_tensor(ctypes.Structure):
    _fields_ = [("expert_grads", _vp), ("slot_grads", _vp), ("row_elems", ctypes.c_int64)]


class moon_route_config(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("R", "S", "E", "K", "dtype")] + \
               [("flags", _u32), ("scale", ctypes.c_float), ("loss_coef", ctypes.c_float)]


class moon_mx4_weight(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("expert_q", "expert_scales", "slot_q", "slot_scales")]


_P = ctypes.POINTER
_lib.moon_ctx_create.argtypes = [_P(moon_config), _P(_vp)]
_lib.moon_ctx_layout.argtypes = [_vp, _P(moon_layout)]
_lib.moon_ctx_destroy.argtypes = [_P(_vp)]
_lib.moon_ctx_destroy.restype = None
_lib.moon_plan_create.argtypes = [_vp, _P(_vp)]
_lib.moon_plan_clone.argtypes = [_vp, _P(_vp), _vp]
_lib.moon_plan_destroy.argtypes = [_P(_vp)]
_lib.moon_plan_destroy.restype = None
_lib.moon_plan_view.argtypes = [_vp, _P(moon_plan_arrays)]
_lib.moon_plan_status.argtypes = [_vp, _vp]
_lib.moon_plan.argtypes = [_vp, _vp, _vp, _vp, _vp]
_lib.moon_dispatch.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _u32, _vp]
_lib.moon_combine.argtypes = [_vp, _vp, _vp, _vp, _u32, _vp, _vp, _vp]
_lib.moon_prefetch_index.argtypes = [_vp, _vp, _vp, _vp]
_lib.moon_prefetch_weight.argtypes = [_vp, _vp, _P(moon_weight_tensor), _i32, _vp]
_lib.moon_reduce_grad.argtypes = [_vp, _vp, _P(moon_grad_tensor), _i32, _vp]
_lib.moon_status_str.argtypes = [_i32]
_lib.moon_status_str.restype = ctypes.c_char_p
_lib.moon_debug_tile_counts.argtypes = [_vp, _vp, _P(_i32), _P(_i32), _vp]
_lib.moon_plan_noalloc.argtypes = [_P(moon_config), _vp, _vp, _P(moon_plan_arrays), _vp]
_i64, _sz = ctypes.c_int64, ctypes.c_size_t
_lib.moon_route_workspace.argtypes = [_P(moon_route_config), _P(_sz)]
_lib.moon_route.argtypes = [_P(moon_route_config)] + [_vp] * 10 + [_sz, _vp]
_lib.moon_route_backward.argtypes = [_P(moon_route_config)] + [_vp] * 9
_lib.moon_mx4_quantize.argtypes = [_vp, _i32, _i64, _i32, _P(moon_plan_arrays), _vp, _vp, _vp]
_lib.moon_mx4_dequantize.argtypes = [_vp, _vp, _i64, _i32, _P(moon_plan_arrays), _i32, _vp, _vp]
_lib.moon_expert_gemm_mx4.argtypes = [_P(moon_plan_arrays), _vp, _vp, _i32, _P(moon_mx4_weight),
                                      _i32, _vp, _vp]
_lib.moon_expert_swiglu_mx4.argtypes = [_P(moon_plan_arrays), _vp, _vp, _i32, _P(moon_mx4_weight),
                                        _P(moon_mx4_weight), _i32, _vp, _vp, _vp]
_lib.moon_swiglu_save8.argtypes = [_P(moon_plan_arrays), _vp, _vp, _i32, _vp, _vp, _vp, _vp]
_lib.moon_swiglu_grad8.argtypes = [_P(moon_plan_arrays), _vp, _vp, _vp, _vp, _i32, _vp, _vp, _vp]
for _f in ("moon_ctx_create", "moon_ctx_layout", "moon_plan_create", "moon_plan_clone",
           "moon_plan_view", "moon_plan_status", "moon_plan", "moon_dispatch", "moon_combine",
           "moon_prefetch_index", "moon_prefetch_weight", "moon_reduce_grad",
           "moon_debug_tile_counts", "moon_plan_noalloc", "moon_route_workspace", "moon_route",
           "moon_route_backward", "moon_mx4_quantize", "moon_mx4_dequantize",
           "moon_expert_gemm_mx4", "moon_expert_swiglu_mx4", "moon_swiglu_save8",
           "moon_swiglu_grad8"):
    getattr(_lib, _f).restype = _i32


class MoonError(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {moon_status_str(status)} ({status})")
        self.status = status


def moon_status_str(status):
    return _lib.moon_status_str(int(status)).decode()


def _check(status, what):
    if status != MOON_OK:
        raise MoonError(status, what)


class Ctx:
    """Handle of a moon_ctx (windows + planner scratch on one device)."""

    def __init__(self, ptr, cfg, layout, device):
        self.ptr, self.cfg, self.layout, self.device = ptr, cfg, layout, device

    @property
    def NvS(self):
        return self.layout.NvS

    @property
    def B(self):
        return self.layout.B


class Plan:
    """Handle of a moon_comm_plan bound to its context."""

    def __init__(self, ptr, ctx):
        self.ptr, self.ctx = ptr, ctx


def _stream(stream, device=None):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return _vp(s.cuda_stream)


def _ptr(t, dtype, numel, name, optional=False):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, got {t.numel()}")
    return _vp(t.data_ptr())


def moon_ctx_create(R, E, K, S, H, B=0, token_padding=1, flags=0):
    cfg = moon_config(R, E, K, S, H, B, token_padding, flags)
    out = _vp()
    _check(_lib.moon_ctx_create(ctypes.byref(cfg), ctypes.byref(out)), "moon_ctx_create")
    lay = moon_layout()
    _check(_lib.moon_ctx_layout(out, ctypes.byref(lay)), "moon_ctx_layout")
    return Ctx(out, cfg, lay, torch.cuda.current_device())


def moon_ctx_layout(ctx):
    lay = moon_layout()
    _check(_lib.moon_ctx_layout(ctx.ptr, ctypes.byref(lay)), "moon_ctx_layout")
    return lay


def moon_ctx_destroy(ctx):
    p = _vp(ctx.ptr.value if ctx.ptr is not None else None)
    _lib.moon_ctx_destroy(ctypes.byref(p))
    ctx.ptr = _vp()


def moon_plan_create(ctx):
    out = _vp()
    _check(_lib.moon_plan_create(ctx.ptr, ctypes.byref(out)), "moon_plan_create")
    return Plan(out, ctx)


def moon_plan_clone(plan, stream=None):
    out = _vp()
    _check(_lib.moon_plan_clone(plan.ptr, ctypes.byref(out), _stream(stream)), "moon_plan_clone")
    return Plan(out, plan.ctx)


def moon_plan_destroy(plan):
    p = _vp(plan.ptr.value if plan.ptr is not None else None)
    _lib.moon_plan_destroy(ctypes.byref(p))
    plan.ptr = _vp()


def moon_plan_view(plan):
    v = moon_plan_arrays()
    _check(_lib.moon_plan_view(plan.ptr, ctypes.byref(v)), "moon_plan_view")
    return v


def moon_plan_status(plan, stream=None):
    """Synchronises the stream; returns the plan's status code (0 = valid)."""
    return int(_lib.moon_plan_status(plan.ptr, _stream(stream)))


def moon_plan(ctx, topk, tokens_per_expert, plan, stream=None):
    c = ctx.cfg
    _check(_lib.moon_plan(ctx.ptr, _ptr(topk, torch.int32, c.R * c.S * c.K, "topk"),
                          _ptr(tokens_per_expert, torch.int32, c.R * c.E, "tokens_per_expert",
                               optional=True), plan.ptr, _stream(stream)), "moon_plan")


def moon_dispatch(ctx, plan, hidden, weights=None, hidden_out=None, weights_out=None, flags=0,
                  stream=None):
    c, rows = ctx.cfg, ctx.cfg.R * ctx.NvS
    _check(_lib.moon_dispatch(
        ctx.ptr, plan.ptr, _ptr(hidden, torch.bfloat16, c.R * c.S * c.H, "hidden"),
        _ptr(weights, torch.float32, c.R * c.S * c.K, "weights", optional=True),
        _ptr(hidden_out, torch.bfloat16, rows * c.H, "hidden_out", optional=True),
        _ptr(weights_out, torch.float32, rows, "weights_out", optional=True), flags,
        _stream(stream)), "moon_dispatch")


def moon_combine(ctx, plan, y, w_nvs, flags, out, w_rsk_out=None, stream=None):
    c, rows = ctx.cfg, ctx.cfg.R * ctx.NvS
    _check(_lib.moon_combine(
        ctx.ptr, plan.ptr, _ptr(y, torch.bfloat16, rows * c.H, "y"),
        _ptr(w_nvs, torch.float32, rows, "w_nvs", optional=True), flags,
        _ptr(out, torch.bfloat16, c.R * c.S * c.H, "out"),
        _ptr(w_rsk_out, torch.float32, c.R * c.S * c.K, "w_rsk_out", optional=True),
        _stream(stream)), "moon_combine")


def moon_prefetch_index(ctx, plan, out, stream=None):
    c = ctx.cfg
    _check(_lib.moon_prefetch_index(ctx.ptr, plan.ptr,
                                    _ptr(out, torch.int32, c.R * ctx.B * 2, "out"),
                                    _stream(stream)), "moon_prefetch_index")


def moon_debug_tile_counts(ctx, out=None, stream=None):
    """Test hook: the planner's per-tile histogram of the latest moon_plan call
    (see include/moon.h).  Returns (tile_tokens, tiles_per_rank); when `out`
    (int32 [E+1, R*tiles_per_rank] on the GPU) is given, fills it."""
    c = ctx.cfg
    tt, tpr = _i32(0), _i32(0)
    _check(_lib.moon_debug_tile_counts(ctx.ptr, None, ctypes.byref(tt), ctypes.byref(tpr), None),
           "moon_debug_tile_counts")
    if out is not None:
        n = (c.E + 1) * c.R * tpr.value
        _check(_lib.moon_debug_tile_counts(ctx.ptr, _ptr(out, torch.int32, n, "out"), None, None,
                                           _stream(stream)), "moon_debug_tile_counts")
    return tt.value, tpr.value


def _expert_pair(ctx, rows, slots, name, dtype=None):
    """Check an ([E, ...], [R, B, ...]) tensor pair; returns (ptrs, row elements)."""
    c = ctx.cfg
    for t, what in ((rows, f"{name} rows"), (slots, f"{name} slots")):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous CUDA tensor")
        if dtype is not None and t.dtype != dtype:
            raise ValueError(f"{what} must be {dtype}, got {t.dtype}")
    if rows.dtype != slots.dtype:
        raise ValueError(f"{name}: rows and slots differ in dtype")
    if rows.shape[0] != c.E or tuple(slots.shape[:2]) != (c.R, ctx.B) or \
            tuple(slots.shape[2:]) != tuple(rows.shape[1:]):
        raise ValueError(f"{name}: expected rows [E={c.E}, ...] and slots [R={c.R}, B={ctx.B}, "
                         f"...] of one row shape, got {tuple(rows.shape)} and "
                         f"{tuple(slots.shape)}")
    return _vp(rows.data_ptr()), _vp(slots.data_ptr()), rows[0].numel()


def moon_prefetch_weight(ctx, plan, experts, slots, stream=None):
    """experts: list of [E, ...] tensors (rows [0, E) of each weight tensor);
    slots: list of [R, B, ...] tensors of the same dtypes, written in place."""
    if len(experts) != len(slots):
        raise ValueError("experts and slots must pair up")
    arr = (moon_weight_tensor * max(len(experts), 1))()
    for i, (x, sl) in enumerate(zip(experts, slots)):
        px, ps, n = _expert_pair(ctx, x, sl, f"tensor {i}")
        arr[i] = moon_weight_tensor(px, ps, n * x.element_size())
    _check(_lib.moon_prefetch_weight(ctx.ptr, plan.ptr, arr, len(experts), _stream(stream)),
           "moon_prefetch_weight")


def moon_reduce_grad(ctx, plan, grads, slot_grads, stream=None):
    """grads: list of [E, ...] float32 tensors (updated); slot_grads: list of
    [R, B, ...] float32 tensors (used slots cleared)."""
    if len(grads) != len(slot_grads):
        raise ValueError("grads and slot_grads must pair up")
    arr = (moon_grad_tensor * max(len(grads), 1))()
    for i, (g, sg) in enumerate(zip(grads, slot_grads)):
        pg, ps, n = _expert_pair(ctx, g, sg, f"gradient {i}", torch.float32)
        arr[i] = moon_grad_tensor(pg, ps, n)
    _check(_lib.moon_reduce_grad(ctx.ptr, plan.ptr, arr, len(grads), _stream(stream)),
           "moon_reduce_grad")


# ---------------------------------------------------------------------------
# Routing and expert operators.  `plan` is a Plan, or a dict of the arrays that
# moon_plan_noalloc filled ("cu_seqlens", "zero_fill_ranges", "experts_to_copy",
# "status"; "dst" where at hand, for its size).  All tensors of a call live on one device, which need not be the
# current one; the stream defaults to that device's current stream.
_DTYPES = {torch.float32: MOON_DTYPE_F32, torch.bfloat16: MOON_DTYPE_BF16}


def _device_of(t, name):
    """Device index of a call's first tensor."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return dev


def _addr(t, dtype, numel, name, dev):
    """Device address of a tensor after the checks of _ptr, on device `dev`."""
    if t.dtype is not dtype or t.numel() != numel or t.get_device() != dev or \
            not t.is_contiguous():
        _ptr(t, dtype, numel, name)
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")
    return t.data_ptr()


def _opt(t, dtype, numel, name, dev):
    return None if t is None else _addr(t, dtype, numel, name, dev)


def _dtype_code(t, name):
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be torch.float32 or torch.bfloat16, got {t.dtype}")
    return _DTYPES[t.dtype]


# The raw handle of a device's current stream without building a Stream object,
# and the current device without the check for a first use (a call has tensors
# on a device).  Small calls are bound by the host: 8 us, 3 of them the launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(dev, fn, *args, stream=None):
    """Calls the library with `dev` current (switching to it and back if it is not)."""
    s = _raw_stream(dev) if stream is None else stream.cuda_stream
    if _current_device() == dev:
        st = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, s)
    if st != MOON_OK:
        raise MoonError(st, fn.__name__)


def _groups(plan, rows, dev):
    """moon_plan_arrays of a Plan or a dict of plan arrays on device `dev`, for
    window tensors of `rows` rows."""
    if isinstance(plan, Plan):
        pa = moon_plan_view(plan)
        if plan.ctx.device != dev:
            raise ValueError(f"the plan is on cuda:{plan.ctx.device}, the tensors on cuda:{dev}")
    else:
        cu, etc, dst = plan["cu_seqlens"], plan["experts_to_copy"], plan.get("dst")
        cs, es = cu.shape, etc.shape
        if len(cs) != 2 or len(es) != 2 or es[0] != cs[0] or cs[0] < 1 or cs[1] <= es[1] or \
                es[1] < 1:
            raise ValueError("cu_seqlens must be [R, E+B] and experts_to_copy [R, B]")
        R, EB = cs
        pa = moon_plan_arrays()
        pa.R, pa.B, pa.E, pa.NvS = R, es[1], EB - es[1], rows // R
        pa.N = dst.numel() // R if dst is not None else 0
        pa.cu_seqlens = _addr(cu, torch.int32, R * EB, "cu_seqlens", dev)
        pa.zero_fill_ranges = _addr(plan["zero_fill_ranges"], torch.int32, 2 * R * EB,
                                    "zero_fill_ranges", dev)
        pa.status = _addr(plan["status"], torch.int32, 1, "status", dev)
    if rows != pa.R * pa.NvS:
        raise ValueError(f"window tensors must have R*NvS = {pa.R * pa.NvS} rows, got {rows}")
    return pa


def _route_config(logits, topk, flags, scale, loss_coef):
    """(moon_route_config, R, S, E, K) of logits [R, S, E] and topk [R, S, K]."""
    ls, ts = logits.shape, topk.shape
    if len(ls) != 3:
        raise ValueError(f"logits must be [R, S, E], got {tuple(ls)}")
    R, S, E = ls
    if len(ts) != 3 or ts[0] != R or ts[1] != S:
        raise ValueError(f"topk must be [R, S, K], got {tuple(ts)}")
    K = ts[2]
    code = _dtype_code(logits, "logits")
    return moon_route_config(R, S, E, K, code, flags, scale, loss_coef), R, S, E, K


def _flags8(valid, n, dev):
    if valid is None:
        return None
    if valid.dtype not in (torch.bool, torch.uint8):
        raise ValueError(f"valid must be torch.bool or torch.uint8, got {valid.dtype}")
    return _addr(valid, valid.dtype, n, "valid", dev)


def moon_route(logits, topk, weights, flags=0, scale=1.0, bias=None, valid=None,
               tokens_per_expert=None, valid_tokens=None, prob_sums=None, loss=None,
               loss_coef=0.0, workspace=None, stream=None):
    """Top-k routing of logits [R, S, E] (float32 or bfloat16) into topk
    [R, S, K] int32 and weights [R, S, K] float32; the optional outputs are
    described at moon_route in include/moon.h.  workspace: a uint8 tensor of at
    least moon_route_workspace(...) bytes; allocated for the call when None."""
    cfg, R, S, E, K = _route_config(logits, topk, flags, scale, loss_coef)
    dev, i32, f32 = _device_of(logits, "logits"), torch.int32, torch.float32
    if workspace is None and S > 32 and not (tokens_per_expert is None and valid_tokens is None
                                              and prob_sums is None and loss is None):
        n = _route_workspace(cfg)
        if n > 0 and stream is None:
            workspace = torch.empty(n, dtype=torch.uint8, device=logits.device)
        elif n > 0:  # from the pool of the stream that uses it, so nothing else still does
            with torch.cuda.stream(stream):
                workspace = torch.empty(n, dtype=torch.uint8, device=logits.device)
    ws_bytes = 0 if workspace is None else workspace.numel()
    _call(dev, _lib.moon_route, ctypes.byref(cfg), _addr(logits, logits.dtype, R * S * E, "logits", dev),
          _opt(bias, f32, E, "bias", dev), _flags8(valid, R * S, dev),
          _addr(topk, i32, R * S * K, "topk", dev), _addr(weights, f32, R * S * K, "weights", dev),
          _opt(tokens_per_expert, i32, R * E, "tokens_per_expert", dev),
          _opt(valid_tokens, i32, R, "valid_tokens", dev),
          _opt(prob_sums, f32, R * E, "prob_sums", dev), _opt(loss, f32, R, "loss", dev),
          _opt(workspace, torch.uint8, ws_bytes, "workspace", dev), ws_bytes, stream=stream)


def _route_workspace(cfg):
    n = _sz(0)
    _check(_lib.moon_route_workspace(ctypes.byref(cfg), ctypes.byref(n)), "moon_route_workspace")
    return n.value


def moon_route_workspace(R, S, E, K):
    """Bytes of workspace that moon_route needs for these sizes."""
    return _route_workspace(moon_route_config(R, S, E, K, MOON_DTYPE_F32, 0, 1.0, 0.0))


def moon_route_backward(logits, topk, d_logits, flags=0, scale=1.0, valid=None, d_weights=None,
                        tokens_per_expert=None, valid_tokens=None, d_loss=None, loss_coef=0.0,
                        stream=None):
    """Gradient of moon_route to d_logits (the shape and dtype of logits) from
    d_weights [R, S, K] and d_loss [R], either of which may be None."""
    cfg, R, S, E, K = _route_config(logits, topk, flags, scale, loss_coef)
    dev, i32, f32 = _device_of(logits, "logits"), torch.int32, torch.float32
    _call(dev, _lib.moon_route_backward, ctypes.byref(cfg),
          _addr(logits, logits.dtype, R * S * E, "logits", dev), _flags8(valid, R * S, dev),
          _addr(topk, i32, R * S * K, "topk", dev),
          _opt(d_weights, f32, R * S * K, "d_weights", dev),
          _opt(tokens_per_expert, i32, R * E, "tokens_per_expert", dev),
          _opt(valid_tokens, i32, R, "valid_tokens", dev), _opt(d_loss, f32, R, "d_loss", dev),
          _addr(d_logits, logits.dtype, R * S * E, "d_logits", dev), stream=stream)


def _mx4_call(fn, x, q, scales, plan, stream):
    if x.dim() < 2:
        raise ValueError("values must be [rows, cols]")
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    dev = _device_of(x, "values")
    pa = None if plan is None else ctypes.byref(_groups(plan, rows, dev))
    px = _addr(x, x.dtype, rows * cols, "values", dev)
    pq = _addr(q, torch.uint8, rows * (cols // 2), "q", dev)
    ps = _addr(scales, torch.uint8, rows * (cols // 32), "scales", dev)
    code = _dtype_code(x, "values")
    if fn is _lib.moon_mx4_quantize:
        _call(dev, fn, px, code, rows, cols, pa, pq, ps, stream=stream)
    else:
        _call(dev, fn, pq, ps, rows, cols, pa, code, px, stream=stream)


def moon_mx4_quantize(x, q, scales, plan=None, stream=None):
    """x [..., cols] (float32 or bfloat16) to MXFP4 codes q [..., cols/2] and
    scales [..., cols/32] (uint8).  With a plan x is window rows [R*NvS, cols]."""
    _mx4_call(_lib.moon_mx4_quantize, x, q, scales, plan, stream)


def moon_mx4_dequantize(q, scales, y, plan=None, stream=None):
    """The values of MXFP4 codes and scales, to y [..., cols]."""
    _mx4_call(_lib.moon_mx4_dequantize, y, q, scales, plan, stream)


def _mx4_weight(pa, w, N, K, name, dev):
    """moon_mx4_weight of (expert codes, expert scales, slot codes, slot scales)."""
    eq, es, sq, ss = w
    u8, E, RB = torch.uint8, pa.E, pa.R * pa.B
    return moon_mx4_weight(_addr(eq, u8, E * N * (K // 2), f"{name} expert codes", dev),
                           _addr(es, u8, E * N * (K // 32), f"{name} expert scales", dev),
                           _addr(sq, u8, RB * N * (K // 2), f"{name} slot codes", dev),
                           _addr(ss, u8, RB * N * (K // 32), f"{name} slot scales", dev))


def _rows_of(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be [R*NvS, values], got {tuple(t.shape)}")
    return t.shape


def moon_expert_gemm_mx4(plan, xq, xs, weight, y, stream=None):
    """y [R*NvS, N] bfloat16 = the MXFP4 rows (xq [R*NvS, K/2], xs) times the
    weights of their groups; weight = (expert_q [E, N, K/2], expert_scales
    [E, N, K/32], slot_q [R, B, N, K/2], slot_scales [R, B, N, K/32])."""
    rows, half = _rows_of(xq, "xq")
    N, K, dev = _rows_of(y, "y")[1], 2 * half, _device_of(xq, "xq")
    pa = _groups(plan, rows, dev)
    w = _mx4_weight(pa, weight, N, K, "weight", dev)
    _call(dev, _lib.moon_expert_gemm_mx4, ctypes.byref(pa),
          _addr(xq, torch.uint8, rows * half, "xq", dev),
          _addr(xs, torch.uint8, rows * (K // 32), "xs", dev), K, ctypes.byref(w), N,
          _addr(y, torch.bfloat16, rows * N, "y", dev), stream=stream)


def moon_expert_swiglu_mx4(plan, xq, xs, gate, up, h, row_weights=None, stream=None):
    """h [R*NvS, F] bfloat16: the gated activation of two such products; gate
    and up as the weight of moon_expert_gemm_mx4, row_weights [R*NvS] float32."""
    rows, half = _rows_of(xq, "xq")
    F, K, dev = _rows_of(h, "h")[1], 2 * half, _device_of(xq, "xq")
    pa = _groups(plan, rows, dev)
    wg = _mx4_weight(pa, gate, F, K, "gate", dev)
    wu = _mx4_weight(pa, up, F, K, "up", dev)
    _call(dev, _lib.moon_expert_swiglu_mx4, ctypes.byref(pa),
          _addr(xq, torch.uint8, rows * half, "xq", dev),
          _addr(xs, torch.uint8, rows * (K // 32), "xs", dev), K, ctypes.byref(wg),
          ctypes.byref(wu), F, _opt(row_weights, torch.float32, rows, "row_weights", dev),
          _addr(h, torch.bfloat16, rows * F, "h", dev), stream=stream)


def moon_swiglu_save8(plan, gate_up, h, saved, saved_scales, row_weights=None, stream=None):
    """Gated activation of gate_up [R*NvS, 2F] (gate first) to h [R*NvS, F],
    both bfloat16, keeping gate_up in 8 bits: saved [R*NvS, 2F] and
    saved_scales [R*NvS, 2F/32], uint8."""
    rows, F = _rows_of(h, "h")
    dev = _device_of(h, "h")
    pa = _groups(plan, rows, dev)
    _call(dev, _lib.moon_swiglu_save8, ctypes.byref(pa),
          _addr(gate_up, torch.bfloat16, rows * 2 * F, "gate_up", dev),
          _opt(row_weights, torch.float32, rows, "row_weights", dev), F,
          _addr(h, torch.bfloat16, rows * F, "h", dev),
          _addr(saved, torch.uint8, rows * 2 * F, "saved", dev),
          _addr(saved_scales, torch.uint8, rows * (2 * F // 32), "saved_scales", dev),
          stream=stream)


def moon_swiglu_grad8(plan, dh, saved, saved_scales, d_gate_up, row_weights=None,
                      d_row_weights=None, stream=None):
    """d_gate_up [R*NvS, 2F] bfloat16 and d_row_weights [R*NvS] float32
    (optional) from dh [R*NvS, F] and what moon_swiglu_save8 kept."""
    rows, F = _rows_of(dh, "dh")
    dev = _device_of(dh, "dh")
    pa = _groups(plan, rows, dev)
    _call(dev, _lib.moon_swiglu_grad8, ctypes.byref(pa),
          _addr(dh, torch.bfloat16, rows * F, "dh", dev),
          _addr(saved, torch.uint8, rows * 2 * F, "saved", dev),
          _addr(saved_scales, torch.uint8, rows * (2 * F // 32), "saved_scales", dev),
          _opt(row_weights, torch.float32, rows, "row_weights", dev), F,
          _addr(d_gate_up, torch.bfloat16, rows * 2 * F, "d_gate_up", dev),
          _opt(d_row_weights, torch.float32, rows, "d_row_weights", dev), stream=stream)


# ---------------------------------------------------------------------------
# Zero-copy tensor views of memory the library owns (they alias it: keep the
# context / plan alive while a view is in use).
class _CudaArray:
    def __init__(self, ptr, shape, typestr):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr,
                                         "data": (int(ptr), False), "version": 2}


def device_view(ptr, shape, dtype, device=None):
    typestr = {torch.int32: "<i4", torch.float32: "<f4", torch.int16: "<i2"}[
        torch.int16 if dtype == torch.bfloat16 else dtype]
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    t = torch.as_tensor(_CudaArray(ptr, shape, typestr), device=dev)
    return t.view(torch.bfloat16) if dtype == torch.bfloat16 else t


def plan_array_shapes(R, E, K, S, B, token_padding):
    """Shapes of the plan arrays (all int32) for moon_plan_noalloc, with the
    capacity NvS = round_up(S*K + (E/R + B)*(P - 1), P) documented at
    moon_ctx_create and B <= 0 meaning E/R.  Returns (shapes, NvS, B)."""
    B = B if B > 0 else E // R
    P = token_padding
    NvS = (S * K + (E // R + B) * (P - 1) + P - 1) // P * P
    EB = E + B
    return ({"dst": (R, S * K), "experts_to_copy": (R, B), "zero_fill_ranges": (R, EB, 2),
             "remote_stats": (R, 2), "dup_groups": (R, NvS, 3), "dup_loffs": (R, NvS),
             "dup_counts": (R, 2), "cu_seqlens": (R, EB), "status": (1,),
             "prefetch_index": (R, B, 2)}, NvS, B)


def moon_plan_noalloc(R, E, K, S, H, B, token_padding, topk, tokens_per_expert, arrays,
                      stream=None):
    """Planning without a context into caller-owned arrays (a dict of int32
    device tensors with the shapes of plan_array_shapes); allocates nothing."""
    shapes, NvS, Bx = plan_array_shapes(R, E, K, S, B, token_padding)
    cfg = moon_config(R, E, K, S, H, B, token_padding, 0)
    pa = moon_plan_arrays()
    for k, shp in shapes.items():
        n = 1
        for x in shp:
            n *= x
        setattr(pa, k, _ptr(arrays[k], torch.int32, n, k))
    pa.N, pa.R, pa.E, pa.B, pa.NvS, pa.K = S * K, R, E, Bx, NvS, K
    _check(_lib.moon_plan_noalloc(ctypes.byref(cfg), _ptr(topk, torch.int32, R * S * K, "topk"),
                                  _ptr(tokens_per_expert, torch.int32, R * E, "tokens_per_expert",
                                       optional=True), ctypes.byref(pa), _stream(stream)),
           "moon_plan_noalloc")


def plan_tensors(plan):
    """Views of the plan arrays, each with a leading R (see include/moon.h)."""
    v = moon_plan_view(plan)
    c = plan.ctx.cfg
    R, EB, NvS = c.R, c.E + v.B, v.NvS
    dev = torch.device("cuda", plan.ctx.device)
    shapes = {"dst": (R, v.N), "experts_to_copy": (R, v.B), "zero_fill_ranges": (R, EB, 2),
              "remote_stats": (R, 2), "dup_groups": (R, NvS, 3), "dup_loffs": (R, NvS),
              "dup_counts": (R, 2), "cu_seqlens": (R, EB), "status": (1,),
              "prefetch_index": (R, v.B, 2)}
    return {k: device_view(getattr(v, k), s, torch.int32, dev) for k, s in shapes.items()}


def window_tensors(ctx):
    """(hidden windows [R*NvS, H] bf16, weight windows [R*NvS] fp32) of the context."""
    lay, c = ctx.layout, ctx.cfg
    dev = torch.device("cuda", ctx.device)
    rows = c.R * lay.NvS_padded
    return (device_view(lay.hidden_windows, (rows, c.H), torch.bfloat16, dev),
            device_view(lay.weight_windows, (rows,), torch.float32, dev))
