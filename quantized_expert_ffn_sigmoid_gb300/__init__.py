"""Python binding of libcolimoe (the routed-MoE layer on sm_103a).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  Functions carry the names of the C entry points declared in
``include/coli_moe.h``; tensors are torch CUDA tensors (device memory and
streams come from torch), and calls are enqueued on the current torch stream
unless ``stream`` is given.  There is no CPU fallback: importing this module
raises if the compiled library is missing.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libcolimoe.so")

COLI_OK = 0
COLI_EINVAL = -1
COLI_EALIGN = -2
COLI_EWORKSPACE = -3
COLI_ECUDA = -4
COLI_EUNSUPPORTED = -5
STATUS_NONFINITE = 1
STATUS_BADIDX = 2
STATUS_TIMEOUT = 4

EXPORTS = (
    "coli_moe_workspace_size", "coli_moe_workspace_init", "coli_moe_route",
    "coli_moe_quantize_act", "coli_moe_forward", "coli_moe_dispatch", "coli_moe_experts",
    "coli_moe_status", "coli_moe_strerror", "coli_moe_workspace_layout",
    "coli_moe_forward_dump", "coli_moe_forward_static", "coli_moe_layer",
    "coli_moe_stack_forward",
    "coli_mx4_quantize", "coli_mx4_dequantize", "coli_mx4_product", "coli_mx4_workspace_size",
    "coli_mx4_forward", "coli_moe_block_norm",
)
STATIC_WS_BYTES = 24 << 20
MX4_PRODUCT_WS_BYTES = 8704
COLI_F32, COLI_BF16, COLI_F16, COLI_MX4 = 0, 1, 2, 3


class Cfg(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("n_groups", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("n_shared", ctypes.c_int32), ("shared_inter", ctypes.c_int32),
                ("weight_bits", ctypes.c_int32), ("routed_scaling_factor", ctypes.c_float),
                ("group_size", ctypes.c_int32), ("ep_rank", ctypes.c_int32), ("ep_size", ctypes.c_int32)]
    _OPTIONAL = ("group_size", "ep_rank", "ep_size")

    @classmethod
    def of(cls, shape, ep_rank: int = 0, ep_size: int = 0) -> "Cfg":
        """From any object with the same field names (e.g. synth.LayerShape);
        a missing group_size means per-row scales.  ``ep_rank`` / ``ep_size``
        select one shard of an expert-parallel layer (0 / 0: the whole layer)."""
        vals = {"ep_rank": ep_rank, "ep_size": ep_size}
        return cls(*(vals[f] if f in vals else getattr(shape, f, 0) if f in cls._OPTIONAL else getattr(shape, f)
                     for f, _ in cls._fields_))


class Weights(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_void_p), ("expert_scales", ctypes.c_void_p),
                ("shared", ctypes.c_void_p), ("shared_scales", ctypes.c_void_p)]


class StackLayer(ctypes.Structure):
    _fields_ = [("cfg", Cfg), ("weights", Weights), ("router_w", ctypes.c_void_p), ("corr_bias", ctypes.c_void_p)]


class Mx4Weights(ctypes.Structure):
    """Four addresses, as in C.  ``make_mx4_weights`` also leaves the bytes behind each of them in
    ``sizes`` and their GPU in ``device``, which ``coli_mx4_forward`` compares with the call, and holds the
    tensors; a struct filled by hand has none of these."""
    _fields_ = [("experts", ctypes.c_void_p), ("expert_scales", ctypes.c_void_p),
                ("shared", ctypes.c_void_p), ("shared_scales", ctypes.c_void_p)]
    sizes = device = tensors = None


class NormArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
                ("gate", ctypes.c_void_p), ("ld_gate", ctypes.c_int64),
                ("x_out", ctypes.c_void_p), ("ld_x_out", ctypes.c_int64),
                ("n_out", ctypes.c_void_p), ("ld_n_out", ctypes.c_int64),
                ("post_w", ctypes.c_void_p), ("pre_w", ctypes.c_void_p),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("res_scale", ctypes.c_float), ("eps", ctypes.c_float), ("type", ctypes.c_int32), ("n_type", ctypes.c_int32)]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "status", "n_entries", "entry_expert", "entry_count", "entry_offset", "pair_token",
        "pair_slot_of", "qx", "dx", "qh", "dh", "o", "total")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                          "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, S, I32, U32P = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32)
    I64 = ctypes.c_int64
    CP, WP = ctypes.POINTER(Cfg), ctypes.POINTER(Weights)
    sig = {
        "coli_moe_workspace_size": ([CP, I32], ctypes.c_size_t),
        "coli_moe_workspace_init": ([P, S, P], ctypes.c_int),
        "coli_moe_route": ([CP, P, I32, P, P, P, P, P, S, P], ctypes.c_int),
        "coli_moe_quantize_act": ([P, I32, I32, P, P, P], ctypes.c_int),
        "coli_moe_forward": ([CP, WP, P, I32, P, P, P, P, S, P], ctypes.c_int),
        "coli_moe_dispatch": ([CP, P, I32, P, P, S, P], ctypes.c_int),
        "coli_moe_experts": ([CP, WP, I32, P, P, P, S, P], ctypes.c_int),
        "coli_moe_status": ([P, P, U32P], ctypes.c_int),
        "coli_moe_strerror": ([ctypes.c_int], ctypes.c_char_p),
        "coli_moe_workspace_layout": ([CP, I32, ctypes.POINTER(WsLayout)], ctypes.c_int),
        "coli_moe_forward_dump": ([CP, WP, P, I32, P, P, P, P, S, P, P, P], ctypes.c_int),
        "coli_moe_forward_static": ([CP, WP, P, I32, P, P, P, P], ctypes.c_int),
        "coli_moe_layer": ([CP, WP, P, I32, P, P, P, P, P, P, S, P], ctypes.c_int),
        "coli_moe_stack_forward": ([ctypes.POINTER(StackLayer), I32, I32, P, P, I32, P, P, P, P, S, P],
                                   ctypes.c_int),
        "coli_mx4_quantize": ([P, I32, I64, I32, I32, P, P, P], ctypes.c_int),
        "coli_mx4_dequantize": ([P, P, I32, I32, P, I32, I64, P], ctypes.c_int),
        "coli_mx4_product": ([P, P, I32, P, P, I32, I32, I32, P, P, I32, I64, P, S, P], ctypes.c_int),
        "coli_mx4_workspace_size": ([CP, I32], ctypes.c_size_t),
        "coli_mx4_forward": ([CP, ctypes.POINTER(Mx4Weights), P, I32, P, I32, P, P, P, I32, P, S, P], ctypes.c_int),
        "coli_moe_block_norm": ([ctypes.POINTER(NormArgs), I32, I32, P], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()


class ColiError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {lib.coli_moe_strerror(code).decode()} ({code})")
        self.code = code


def _check(rc: int, where: str):
    if rc != COLI_OK:
        raise ColiError(rc, where)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _cfg(cfg) -> Cfg:
    return cfg if isinstance(cfg, Cfg) else Cfg.of(cfg)


def make_weights(experts, expert_scales, shared=None, shared_scales=None) -> Weights:
    """A weights struct from torch tensors (keep the tensors alive)."""
    return Weights(experts.data_ptr(), expert_scales.data_ptr(),
                   shared.data_ptr() if shared is not None else None,
                   shared_scales.data_ptr() if shared_scales is not None else None)


# ----------------------------------------------------------------- entry points
def coli_moe_workspace_size(cfg, max_T: int) -> int:
    return int(lib.coli_moe_workspace_size(ctypes.byref(_cfg(cfg)), int(max_T)))


def coli_moe_workspace_init(ws, stream=None):
    _check(lib.coli_moe_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "coli_moe_workspace_init")


def new_workspace(cfg, max_T: int, device="cuda"):
    """Allocate (with torch) and initialise a workspace for up to max_T positions."""
    import torch
    n = coli_moe_workspace_size(cfg, max_T)
    if n == 0:
        raise ColiError(COLI_EINVAL, "coli_moe_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    coli_moe_workspace_init(ws)
    return ws


def coli_moe_route(cfg, x, router_w, corr_bias, topk_idx, topk_w, ws, stream=None):
    T = x.shape[0]
    _check(lib.coli_moe_route(ctypes.byref(_cfg(cfg)), _ptr(x), T, _ptr(router_w), _ptr(corr_bias),
                              _ptr(topk_idx), _ptr(topk_w), _ptr(ws), ws.numel(), _stream(stream)),
           "coli_moe_route")


def coli_moe_quantize_act(x, q, d, stream=None):
    T, K = x.shape
    _check(lib.coli_moe_quantize_act(_ptr(x), T, K, _ptr(q), _ptr(d), _stream(stream)),
           "coli_moe_quantize_act")


def coli_moe_forward(cfg, weights: Weights, x, topk_idx, topk_w, y, ws, stream=None):
    _check(lib.coli_moe_forward(ctypes.byref(_cfg(cfg)), ctypes.byref(weights), _ptr(x), x.shape[0],
                                _ptr(topk_idx), _ptr(topk_w), _ptr(y), _ptr(ws), ws.numel(),
                                _stream(stream)), "coli_moe_forward")


def coli_moe_layer(cfg, weights: Weights, x, router_w, corr_bias, topk_idx, topk_w, y, ws, stream=None):
    _check(lib.coli_moe_layer(ctypes.byref(_cfg(cfg)), ctypes.byref(weights), _ptr(x), x.shape[0],
                              _ptr(router_w), _ptr(corr_bias), _ptr(topk_idx), _ptr(topk_w), _ptr(y),
                              _ptr(ws), ws.numel(), _stream(stream)), "coli_moe_layer")


def coli_moe_dispatch(cfg, x, topk_idx, ws, stream=None):
    _check(lib.coli_moe_dispatch(ctypes.byref(_cfg(cfg)), _ptr(x), x.shape[0], _ptr(topk_idx),
                                 _ptr(ws), ws.numel(), _stream(stream)), "coli_moe_dispatch")


def coli_moe_experts(cfg, weights: Weights, T: int, topk_w, y, ws, stream=None):
    _check(lib.coli_moe_experts(ctypes.byref(_cfg(cfg)), ctypes.byref(weights), int(T), _ptr(topk_w),
                                _ptr(y), _ptr(ws), ws.numel(), _stream(stream)), "coli_moe_experts")


def coli_moe_forward_dump(cfg, weights: Weights, x, topk_idx, topk_w, y, ws, acc_gu=None, acc_d=None,
                          stream=None):
    _check(lib.coli_moe_forward_dump(ctypes.byref(_cfg(cfg)), ctypes.byref(weights), _ptr(x), x.shape[0],
                                     _ptr(topk_idx), _ptr(topk_w), _ptr(y), _ptr(ws), ws.numel(),
                                     _ptr(acc_gu), _ptr(acc_d), _stream(stream)), "coli_moe_forward_dump")


def coli_moe_status(ws, stream=None) -> int:
    v = ctypes.c_uint32(0)
    _check(lib.coli_moe_status(_ptr(ws), _stream(stream), ctypes.byref(v)), "coli_moe_status")
    return int(v.value)


def coli_moe_strerror(code: int) -> str:
    return lib.coli_moe_strerror(int(code)).decode()


def coli_moe_workspace_layout(cfg, T: int) -> WsLayout:
    out = WsLayout()
    _check(lib.coli_moe_workspace_layout(ctypes.byref(_cfg(cfg)), int(T), ctypes.byref(out)),
           "coli_moe_workspace_layout")
    return out


def coli_moe_forward_static(cfg, weights: Weights, x, topk_idx, topk_w, y, stream=None):
    """coli_moe_forward without a caller workspace: the library's static
    24 MiB device scratch is used instead (for callers that cannot allocate;
    calls must not overlap on the GPU)."""
    _check(lib.coli_moe_forward_static(ctypes.byref(_cfg(cfg)), ctypes.byref(weights), _ptr(x), x.shape[0],
                                       _ptr(topk_idx), _ptr(topk_w), _ptr(y), _stream(stream)),
           "coli_moe_forward_static")


def stack_layers(layers):
    """A ctypes array of StackLayer from (cfg, weights, router_w, corr_bias)
    tuples (keep the tensors alive)."""
    arr = (StackLayer * len(layers))()
    for i, (cfg, w, wr, b) in enumerate(layers):
        arr[i] = StackLayer(_cfg(cfg), w, wr.data_ptr(), b.data_ptr())
    return arr


def coli_moe_stack_forward(layers, xs, residual, topk_idx, topk_w, y, ws, add_output=False, stream=None):
    """One step through a stack of layers (``layers`` from stack_layers):
    xs [L+1, T, H] (xs[0] read, the rest written), residual [L, T, H] or
    None, topk_idx / topk_w [L, T, k] and y [L, T, H] written."""
    n, T = len(layers), xs.shape[1]
    _check(lib.coli_moe_stack_forward(layers, n, T, _ptr(xs), _ptr(residual), int(bool(add_output)),
                                      _ptr(topk_idx), _ptr(topk_w), _ptr(y), _ptr(ws), ws.numel(),
                                      _stream(stream)), "coli_moe_stack_forward")


def capture_stack_step(layers, xs, residual, topk_idx, topk_w, y, ws, add_output=False):
    """The stack step captured once as a CUDA graph (torch.cuda.CUDAGraph);
    ``graph.replay()`` runs it again on the same buffers.  Runs the step once
    first, outside capture (the first call of some kernels sets attributes)."""
    import torch
    coli_moe_stack_forward(layers, xs, residual, topk_idx, topk_w, y, ws, add_output)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        coli_moe_stack_forward(layers, xs, residual, topk_idx, topk_w, y, ws, add_output)
    return g


# ------------------------------------------------------------------ MX4 experts
# Single-position calls take a few microseconds on the GPU, so these bindings
# keep their own cost to about that: one look at each tensor, plain integers
# to ctypes, the raw handle of the current stream.
#
# The library launches on the current device, so the tensors of a call are all
# on that one: anything else is refused here, before their addresses reach it.
_TYPES = {}
_raw_stream = _raw_device = _F32 = _I32 = None


def _torch_names():
    global _raw_stream, _raw_device, _F32, _I32
    import torch
    _raw_stream, _raw_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _F32, _I32 = torch.float32, torch.int32
    _TYPES.update({torch.float32: COLI_F32, torch.bfloat16: COLI_BF16, torch.float16: COLI_F16})


def _type(t) -> int:
    if not _TYPES:
        _torch_names()
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"values are float32, bfloat16 or float16, not {t.dtype}")
    return code


def _on(dev: int, stream) -> int:
    """The stream to enqueue on: the given one, else the current one; either of GPU `dev`, which must be the current device."""
    if dev < 0:
        raise ValueError("the tensors must be GPU tensors")
    if _raw_device is None:
        _torch_names()
    if _raw_device() != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{_raw_device()}: make theirs current (torch.cuda.device)")
    if stream is None:
        return _raw_stream(dev)
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"the stream is of cuda:{stream.device_index}, the tensors are on cuda:{dev}")
    return stream.cuda_stream


def _refuse(t, what: str, shape, name: str, dev: int):
    if dev < 0:
        raise ValueError("the tensors must be GPU tensors")
    raise ValueError(f"{name} must be a {what}GPU tensor on cuda:{dev} of shape {tuple(shape)}, not {t.dtype} {tuple(t.shape)} on {t.device}")


def _beyond(*sizes):
    raise ValueError(f"sizes beyond 32 bits: {sizes}")


def _pitch(t, shape, name: str):
    """The row stride of a tensor of two dimensions whose rows have consecutive elements."""
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have consecutive elements in each row")
    return ld if shape[0] > 1 or ld > shape[1] else shape[1]


# `dev` is the device of the tensor that gives a call its shape; _on looks at it last.
def _rows(t, shape, name: str, dev: int):
    """The row stride of a tensor of `shape` (two dimensions) on `dev`."""
    if t.shape != shape or t.get_device() != dev:
        _refuse(t, "", shape, name, dev)
    return _pitch(t, shape, name)


def _bytes(t, shape, name: str, dev: int) -> int:
    """The address of a contiguous uint8 tensor of `shape` on `dev`."""
    if t.shape != shape or t.element_size() != 1 or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, "contiguous uint8 ", shape, name, dev)
    return t.data_ptr()


def _flat(t, shape, dtype, name: str, dev: int) -> int:
    """The address of a contiguous tensor of `shape` and `dtype` on `dev`."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _refuse(t, "contiguous ", shape, name, dev)
    return t.data_ptr()


def _space(ws, dev: int):
    """Address and bytes of a workspace on `dev`."""
    if ws.get_device() != dev or not ws.is_contiguous():
        _refuse(ws, "contiguous ", ws.shape, "ws", dev)
    return ws.data_ptr(), ws.nbytes


def coli_mx4_quantize(x, codes, scales, stream=None):
    """MX4 of the rows of x [T, K] (any row stride) into codes [T, K/2] and scales [T, K/32]."""
    T, K = shape = x.shape
    if (T | K) >> 31:
        _beyond(T, K)
    ty, dev = _type(x), x.get_device()
    rc = lib.coli_mx4_quantize(x.data_ptr(), ty, _pitch(x, shape, "x"), T, K, _bytes(codes, (T, K // 2), "codes", dev),
                               _bytes(scales, (T, K // 32), "scales", dev), _on(dev, stream))
    if rc:
        _check(rc, "coli_mx4_quantize")


def coli_mx4_dequantize(codes, scales, out, stream=None):
    """The values of codes [T, K/2] and scales [T, K/32] into out [T, K] (any row stride)."""
    T, K = shape = out.shape
    if (T | K) >> 31:
        _beyond(T, K)
    ty, dev = _type(out), out.get_device()
    rc = lib.coli_mx4_dequantize(_bytes(codes, (T, K // 2), "codes", dev), _bytes(scales, (T, K // 32), "scales", dev), T, K,
                                 out.data_ptr(), ty, _pitch(out, shape, "out"), _on(dev, stream))
    if rc:
        _check(rc, "coli_mx4_dequantize")


def new_mx4_product_workspace(device="cuda"):
    """Allocate (with torch) and initialise a workspace for coli_mx4_product."""
    import torch
    ws = torch.empty(MX4_PRODUCT_WS_BYTES, dtype=torch.uint8, device=device)
    coli_moe_workspace_init(ws)
    return ws


def coli_mx4_product(x_codes, x_scales, w_codes, w_scales, y, ws, offsets=None, stream=None):
    """y[p] = w[group of p] x[p] for x_codes [P, K/2], w_codes [G, N, K/2] (or [N, K/2]) with their
    scales; ``offsets`` [G + 1] int32 on the device gives each group's first row (None: one group)."""
    P, k2 = shape = x_codes.shape
    w_shape = w_codes.shape
    if len(w_shape) == 3:
        G, N, _ = w_shape
        codes, scales = (G, N, k2), (G, N, k2 // 16)
    else:
        G, (N, _) = 1, w_shape
        codes, scales = (N, k2), (N, k2 // 16)
    if (P | G | N | 2 * k2) >> 31:
        _beyond(P, G, N, 2 * k2)
    yt, dev = _type(y), y.get_device()
    if y.shape != (P, N):
        _refuse(y, "", (P, N), "y", dev)
    wp, wn = _space(ws, dev)
    rc = lib.coli_mx4_product(_bytes(x_codes, shape, "x_codes", dev), _bytes(x_scales, (P, k2 // 16), "x_scales", dev), P,
                              _bytes(w_codes, codes, "w_codes", dev), _bytes(w_scales, scales, "w_scales", dev), G, N, 2 * k2,
                              None if offsets is None else _flat(offsets, (G + 1,), _I32, "offsets", dev),
                              y.data_ptr(), yt, _pitch(y, (P, N), "y"), wp, wn, _on(dev, stream))
    if rc:
        _check(rc, "coli_mx4_product")


def make_mx4_weights(experts, expert_scales, shared=None, shared_scales=None) -> Mx4Weights:
    """An MX4 weights struct from contiguous uint8 GPU tensors that hold exactly the records of the
    configuration they are used with: all experts, or those of its shard.  It keeps the tensors alive."""
    at, sizes, dev = [], [], experts.get_device()
    if dev < 0:
        raise ValueError(f"experts must be a contiguous uint8 GPU tensor, not on {experts.device}")
    for name, t in (("experts", experts), ("expert_scales", expert_scales), ("shared", shared), ("shared_scales", shared_scales)):
        n = 0 if t is None else t.numel()
        at.append(_bytes(t, t.shape, name, dev) if n else None)
        sizes.append(n)
    w = Mx4Weights(*at)
    w.sizes, w.device, w.tensors = tuple(sizes), dev, (experts, expert_scales, shared, shared_scales)
    return w


def _check_records(c, sizes):
    """Whether weights of these sizes are the records of configuration c (its shard's experts; the shared
    ones where they are used): the library sees addresses only."""
    def record(n, inter):
        return n * 3 * inter * c.hidden // 2, n * 3 * inter * c.hidden // 32

    n = c.n_experts if c.ep_size <= 1 else (c.n_experts - c.ep_rank + c.ep_size - 1) // c.ep_size
    want = record(n, c.inter)
    if sizes[:2] != want:
        raise ValueError(f"experts and expert_scales must be the records of {n} experts, {want} bytes, not {sizes[:2]}")
    if c.n_shared > 0 and c.ep_rank == 0 and any(sizes[2:]):
        want = record(c.n_shared, c.shared_inter)
        if sizes[2:] != want:
            raise ValueError(f"shared and shared_scales must be the records of {c.n_shared} shared experts, {want} bytes, not {sizes[2:]}")


def coli_mx4_workspace_size(cfg, max_T: int) -> int:
    if max_T >> 31 > 0:
        _beyond(max_T)
    return int(lib.coli_mx4_workspace_size(ctypes.byref(_cfg(cfg)), int(max_T)))


def new_mx4_workspace(cfg, max_T: int, device="cuda"):
    """Allocate (with torch) and initialise a workspace for coli_mx4_forward (and coli_moe_route)."""
    import torch
    n = coli_mx4_workspace_size(cfg, max_T)
    if n == 0:
        raise ColiError(COLI_EINVAL, "coli_mx4_workspace_size")
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    coli_moe_workspace_init(ws)
    return ws


def coli_mx4_forward(cfg, weights: Mx4Weights, x, topk_idx, topk_w, y, ws, x_scales=None, stream=None):
    """The MX4 expert layer: x [T, H] values, or codes [T, H/2] with ``x_scales`` [T, H/32]; y [T, H]."""
    c = _cfg(cfg)
    T, H = y.shape
    if H != c.hidden:
        raise ValueError(f"y must be [positions, {c.hidden}], not {tuple(y.shape)}")
    if T >> 31:
        _beyond(T)
    if not y.is_contiguous():
        raise ValueError("y must be contiguous")
    yt, dev = _type(y), y.get_device()
    if x_scales is None:
        xt, sp = _type(x), None
        xp = _flat(x, (T, H), x.dtype, "x", dev)
    else:
        xp, xt, sp = _bytes(x, (T, H // 2), "x", dev), COLI_MX4, _bytes(x_scales, (T, H // 32), "x_scales", dev)
    if weights.sizes is not None:
        _check_records(c, weights.sizes)
        if weights.device != dev:
            raise ValueError(f"the weights are on cuda:{weights.device}, y is not on that GPU but on {y.device}")
    k = c.top_k
    wp, wn = _space(ws, dev)
    rc = lib.coli_mx4_forward(ctypes.byref(c), ctypes.byref(weights), xp, xt, sp, T, _flat(topk_idx, (T, k), _I32, "topk_idx", dev),
                              _flat(topk_w, (T, k), _F32, "topk_w", dev), y.data_ptr(), yt,
                              wp, wn, _on(dev, stream))
    if rc:
        _check(rc, "coli_mx4_forward")


def coli_moe_block_norm(x, y=None, post_w=None, gate=None, res_scale=1.0, pre_w=None, eps=1e-6, x_out=None, n_out=None,
                        codes=None, scales=None, stream=None):
    """x' = x + res_scale * gate * (y, normed with post_w) and n = x' normed with pre_w, for rows of
    x [T, H]: writes whichever of x_out (may be x), n_out, codes + scales (MX4 of n) are given.
    ``gate`` is [H] or [T, H]."""
    T, H = shape = x.shape
    if (T | H) >> 31:
        _beyond(T, H)
    dtype, ty, dev = x.dtype, _type(x), x.get_device()
    yp = gp = xp = np = None
    ldy = ldg = ldx = ldn = 0
    nt = ty
    if y is not None:
        if y.dtype is not dtype:
            raise TypeError(f"y must have x's type {dtype}, not {y.dtype}")
        yp, ldy = y.data_ptr(), _rows(y, shape, "y", dev)
    if gate is not None:
        if gate.dtype is not dtype:
            raise TypeError(f"gate must have x's type {dtype}, not {gate.dtype}")
        if gate.dim() == 1:
            gp = _flat(gate, (H,), dtype, "gate", dev)
        else:
            gp, ldg = gate.data_ptr(), _rows(gate, shape, "gate", dev)
    if x_out is not None:
        if x_out.dtype is not dtype:
            raise TypeError(f"x_out must have x's type {dtype}, not {x_out.dtype}")
        xp, ldx = x_out.data_ptr(), _rows(x_out, shape, "x_out", dev)
    if n_out is not None:
        np, ldn = n_out.data_ptr(), _rows(n_out, shape, "n_out", dev)
        if n_out.dtype is not dtype:
            nt = _type(n_out)
    args = NormArgs(x.data_ptr(), _pitch(x, shape, "x"), yp, ldy, gp, ldg, xp, ldx, np, ldn,
                    None if post_w is None else _flat(post_w, (H,), _F32, "post_w", dev), None if pre_w is None else _flat(pre_w, (H,), _F32, "pre_w", dev),
                    None if codes is None else _bytes(codes, (T, H // 2), "codes", dev),
                    None if scales is None else _bytes(scales, (T, H // 32), "scales", dev), res_scale, eps, ty, nt)
    rc = lib.coli_moe_block_norm(args, T, H, _on(dev, stream))
    if rc:
        _check(rc, "coli_moe_block_norm")
