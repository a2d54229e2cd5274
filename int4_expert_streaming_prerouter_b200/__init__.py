"""Python binding of ``libe0moe.so``: argument marshalling only.

Every step of the MoE block runs in the library's CUDA kernels; this module turns torch
tensors into device pointers and CUDA streams, calls the C ABI declared in
``include/e0moe.h`` and raises :class:`E0Error` on a non-zero status.  PyTorch is used
for device memory, pinned host memory and streams only.

There is no fallback: if the shared library is missing this module raises at import of
:func:`lib` time, and every call needs a CUDA device.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libe0moe.so")

E0_OK, E0_ERR_INVALID_ARG = 0, -1
STATUS = {0: "OK", -1: "INVALID_ARG", -2: "CUDA", -3: "OOM", -4: "STAGING", -5: "SLOT_MISMATCH",
          -6: "TIMEOUT", -7: "DEVICE"}


class E0Error(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code
        self.status = STATUS.get(code, str(code))


class Dims(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int), ("n_experts", ctypes.c_int), ("d_ff", ctypes.c_int),
                ("top_k", ctypes.c_int), ("group", ctypes.c_int), ("lora_rank", ctypes.c_int),
                ("head_hidden", ctypes.c_int), ("head_onehot", ctypes.c_int),
                ("rms_eps", ctypes.c_float), ("lora_scale", ctypes.c_float)]


class Layer(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("experts", "shared", "lora_Ag", "lora_Bg", "lora_Au", "lora_Bu", "lora_Ad", "lora_Bd",
                 "router_w", "norm_w")]


class Head(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_lin", "fc1_w", "fc1_b", "fc2_w", "fc2_b")]


class Int4Mat(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("min", ctypes.c_void_p),
                ("n", ctypes.c_int), ("k", ctypes.c_int), ("group", ctypes.c_int),
                ("lora_A", ctypes.c_void_p), ("lora_B", ctypes.c_void_p), ("lora_rank", ctypes.c_int),
                ("lora_scale", ctypes.c_float)]


class Stats(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_uint64), ("staged_experts", ctypes.c_uint64),
                ("staged_bytes", ctypes.c_uint64), ("prefetched_experts", ctypes.c_uint64),
                ("ondemand_experts", ctypes.c_uint64), ("dropped", ctypes.c_uint64),
                ("stage_ms", ctypes.c_double), ("exposed_wait_ms", ctypes.c_double),
                ("kernel_launches", ctypes.c_uint64), ("gemm_timed", ctypes.c_uint64),
                ("gemm_ms", ctypes.c_double), ("hit_experts", ctypes.c_uint64)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_LL = ctypes.c_longlong

# name -> (restype, argtypes); one entry per function declared in include/e0moe.h
_SIGS = {
    "e0_create": (_I, [ctypes.POINTER(Dims), _I, _I, ctypes.POINTER(_P)]),
    "e0_destroy": (_I, [_P]),
    "e0_register_model": (_I, [_P, ctypes.POINTER(Layer), ctypes.POINTER(Head)]),
    "e0_moe_layer_forward": (_I, [_P, _I, _P, _I, _P, _P, _P, _P, _P, _P]),
    "e0_prerouter_predict": (_I, [_P, _I, _P, _I, _P, _P, _P, _P, _P]),
    "e0_stream_register": (_I, [_P, _P, ctypes.c_size_t, _I, _I]),
    "e0_stage_experts": (_I, [_P, _I, ctypes.POINTER(ctypes.c_int32), _I, _P]),
    "e0_moe_stack_decode": (_I, [_P, _P, _I, _I, _P, _P, _I, _I, _P]),
    "e0_moe_stack_decode_host": (_I, [_P, _P, _I, _I, _P, _P, _I, _I, _P]),
    "e0_host_io_wait": (_I, [_P, _P]),
    "e0_get_routing": (_I, [_P, _I, _P, _P]),
    "e0_moe_prefill_stack": (_I, [_P, _P, _I, _P, _P, _P, _P]),
    "e0_moe_prefill_stack_host": (_I, [_P, _P, _I, _P, _P, _P, _P]),
    "e0_get_stats": (_I, [_P, ctypes.POINTER(Stats)]),
    "e0_sync_status": (_I, [_P]),
    "e0_last_error": (ctypes.c_char_p, []),
    "e0_moe_layer_forward_noalloc": (_I, [ctypes.POINTER(Dims), ctypes.POINTER(Layer), _P, _I, _P, _P, _P, _P,
                                          _P, _P, _P]),
    "e0_add_rmsnorm": (_I, [_P, _LL, _P, _I, _LL, _P, ctypes.c_float, _I, _I, _P, _LL, _P, _LL, _P, _I, _LL, _I, _P,
                            _P]),
    "e0_int4_linear": (_I, [ctypes.POINTER(Int4Mat), _P, _I, _LL, _P, _I, _I, _P, _I, _LL, _P]),
    "e0_moe_layer_few": (_I, [ctypes.POINTER(Dims), ctypes.POINTER(Layer), _P, _P, _I, _P, _P, _P, _P, _P, _P, _P,
                              ctypes.c_size_t, _P, _P]),
    "e0_moe_layer_few_workspace": (_I, [ctypes.POINTER(Dims), _I, ctypes.POINTER(ctypes.c_size_t)]),
    "e0_stream_mode": (_I, [_P, _I]),
    "e0_debug_stream_log": (_I, [_P, _P]),
    "e0_debug_pool_slot": (_I, [_P, _I, _I, ctypes.POINTER(_P)]),
    "e0_debug_fail_staging_after": (_I, [_P, _I]),
    "e0_debug_set_slot_tag": (_I, [_P, _I, _I, _I]),
    "e0_debug_decode_stall": (_I, [_P, _I, ctypes.c_ulonglong]),
    "e0_debug_force_general": (_I, [_P, _I]),
    "e0_debug_decode_trace": (_I, [_P, _P]),
    "e0_debug_prefill_path": (_I, [_P, _I]),
    "e0_prefill_fixed_order": (_I, [_P, _I]),
    "e0_debug_decode_mode": (_I, [_P, _I]),
    "e0_debug_decode_flat": (_I, [_P, _I]),
    "e0_debug_time_gemm": (_I, [_P, _I]),
    "e0_debug_phase_timing": (_I, [_P, _I]),
    "e0_debug_phase_times": (_I, [_P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_ulonglong)]),
    "e0_decode_items": (_I, [ctypes.POINTER(Dims), _I, ctypes.POINTER(ctypes.c_uint8), ctypes.POINTER(ctypes.c_uint8),
                             _I, _I, _I, _I, ctypes.POINTER(ctypes.c_uint64), _I, ctypes.POINTER(_I)]),
}


def lib():
    """Load ``libe0moe.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m int4_expert_streaming_prerouter_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _check(rc: int):
    if rc != E0_OK:
        raise E0Error(rc, lib().e0_last_error().decode(errors="replace"))


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def make_dims(d, E, I, k, r, head_hidden=0, head_onehot=0, eps=1e-6, lora_scale=1.0) -> Dims:
    return Dims(d, E, I, k, 64, r, head_hidden, head_onehot, eps, lora_scale)


def decode_items(dims: Dims, n_layers: int, has_head, has_lora, n_ctas: int, flat: bool, step0: bool, cta: int):
    """The one-launch decode kernel's work-item list of CTA `cta` (host only; see the C
    header): a list of (kind, first, layer, first_unit, n_units) with kind 0 router rows,
    1 top-k, 2 x rows, 3 gate/up units, 4 down rows."""
    cap = 512
    out = (ctypes.c_uint64 * cap)()
    n = ctypes.c_int(0)
    hh = (ctypes.c_uint8 * n_layers)(*[1 if v else 0 for v in has_head])
    hl = (ctypes.c_uint8 * n_layers)(*[1 if v else 0 for v in has_lora])
    _check(lib().e0_decode_items(ctypes.byref(dims), n_layers, hh, hl, n_ctas, int(flat), int(step0), cta, out, cap,
                                 ctypes.byref(n)))
    return [(w & 15, (w >> 4) & 1, (w >> 8) & 255, (w >> 16) & 0xFFFFFF, w >> 40) for w in out[:n.value]]


def moe_layer_forward_noalloc(dims: Dims, layer: dict, h, route_idx=None, y=None, y_f32=None, idx=None,
                              gates=None, dev_status=None, stream=None):
    """One MoE block without any device allocation by the library (see the C header).
    `layer` is a dict of torch tensors as for Context.register_model."""
    import torch
    L = Layer()
    for f, _ in Layer._fields_:
        setattr(L, f, _ptr(layer.get(f)))
    T = h.shape[0]
    if y is None:
        y = torch.empty((T, dims.d_model), dtype=torch.bfloat16, device=h.device)
    _check(lib().e0_moe_layer_forward_noalloc(ctypes.byref(dims), ctypes.byref(L), _ptr(h), T, _ptr(route_idx),
                                              _ptr(y), _ptr(y_f32), _ptr(idx), _ptr(gates), _ptr(dev_status),
                                              _stream(stream)))
    return y


# ---------------------------------------------------------------------------------------
# Operators around the attention of a decoder layer (no context; see the C header)
# ---------------------------------------------------------------------------------------
ACT_BF16, ACT_INT8, ACT_E4M3 = 0, 1, 2


class _Torch:
    """What these calls need of torch, looked up once: they take a few microseconds in all, of
    which every lookup is a part."""

    def __init__(self):
        import torch
        self.bf16, self.f32, self.i32, self.u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
        self.int8, self.e4m3 = torch.int8, torch.float8_e4m3fn
        self.act = {self.bf16: ACT_BF16, self.int8: ACT_INT8, self.e4m3: ACT_E4M3}
        self.empty, self.on_device, self.on_stream = torch.empty, torch.cuda.device, torch.cuda.stream
        self.current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        L = lib()
        self.add_rmsnorm, self.int4_linear, self.moe_layer_few = L.e0_add_rmsnorm, L.e0_int4_linear, L.e0_moe_layer_few
        # the handle of a device's current stream, without an object around it
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_torch_names = None


def _torch() -> _Torch:
    global _torch_names
    if _torch_names is None:
        _torch_names = _Torch()
    return _torch_names


def _act_format(t) -> int:
    f = _torch().act.get(t.dtype)
    if f is None:
        raise TypeError(f"expected a bfloat16, int8 or float8_e4m3fn tensor, got {t.dtype}")
    return f


def _rows(t, name, shape, d, dtype, dev):
    """(address, row stride in elements) of a matrix of `shape` whose rows of d are contiguous."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape or t.get_device() != dev:
        raise ValueError(f"{name}: expected shape {tuple(shape)} on the device of the other tensors, got {tuple(t.shape)} on "
                         f"{t.device}")
    if t.is_contiguous():
        return t.data_ptr(), d
    rs, cs = t.stride()
    if cs != 1 and d > 1:
        raise ValueError(f"{name}: the channels of a row must be contiguous")
    return t.data_ptr(), rs if t.shape[0] > 1 else max(rs, d)


def _flat(t, name, shape, dtype, dev) -> Optional[int]:
    """Address of a contiguous tensor of the given shape and type; None for None."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on the device of the other "
                         f"tensors, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """An uninitialised tensor of the pool of the stream that will write it first."""
    X = _torch()
    if stream is None:
        return X.empty(shape, dtype=dtype, device=device)
    with X.on_stream(stream):
        return X.empty(shape, dtype=dtype, device=device)


def _few_workspace(dims, T, device, stream=None):
    n = ctypes.c_size_t(0)
    _check(lib().e0_moe_layer_few_workspace(ctypes.byref(dims), T, ctypes.byref(n)))
    return _empty(n.value, _torch().u8, device, stream)


def _call(X, dev, stream, fn, *args):
    """Call a library function that enqueues on `stream` (default: the current one of device
    `dev`) with that device current."""
    if dev < 0:
        raise ValueError("CUDA tensors are needed")
    raw = X.raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == X.current_device():
        rc = fn(*args, raw)
    else:
        with X.on_device(dev):
            rc = fn(*args, raw)
    if rc:
        _check(rc)


def add_rmsnorm(h, norm_w, delta=None, eps=1e-6, h_out=None, x=None, q8=None, q8_scale=None, q8_group=0, stream=None):
    """h' = bf16(h + delta) and its RMSNorm, in bf16 and in 8 bits (see the C header).

    h [T, d] bf16, norm_w [d] bf16, delta [T, d] bf16 or fp32 or None.  Outputs, each a tensor
    to write or None: h_out [T, d] bf16 (may be h), x [T, d] bf16, q8 [T, d] int8 or
    float8_e4m3fn with q8_scale [T, groups] fp32, one group for each q8_group = 64 or 128
    channels or for a whole row (0).  x is allocated where none of the three is given, q8_scale
    where only q8 is.  Returns (h_out, x, q8, q8_scale)."""
    X = _torch()
    bf16, dev = X.bf16, h.get_device()
    shape = h.shape
    T, d = shape
    hp, hs = _rows(h, "h", shape, d, bf16, dev)
    if h_out is None and x is None and q8 is None:
        x = _empty(shape, bf16, h.device, stream)
    # (whole tensors of the right kind, as nearly every call has them, are told apart here; _rows
    # takes or refuses the others)
    dp = ds = f32 = op = os_ = xp = xs = qp = qs = fmt = sp = 0
    if delta is not None:
        f32 = delta.dtype is X.f32
        if (f32 or delta.dtype is bf16) and delta.shape == shape and delta.get_device() == dev and delta.is_contiguous():
            dp, ds = delta.data_ptr(), d
        else:
            dp, ds = _rows(delta, "delta", shape, d, X.f32 if f32 else bf16, dev)
    if h_out is not None:
        if h_out is h:
            op, os_ = hp, hs
        elif h_out.dtype is bf16 and h_out.shape == shape and h_out.get_device() == dev and h_out.is_contiguous():
            op, os_ = h_out.data_ptr(), d
        else:
            op, os_ = _rows(h_out, "h_out", shape, d, bf16, dev)
    if x is not None:
        if x.dtype is bf16 and x.shape == shape and x.get_device() == dev and x.is_contiguous():
            xp, xs = x.data_ptr(), d
        else:
            xp, xs = _rows(x, "x", shape, d, bf16, dev)
    if q8 is not None:
        fmt = _act_format(q8)
        if fmt == ACT_BF16:
            raise TypeError("q8: expected an int8 or float8_e4m3fn tensor")
        if q8_group not in (0, 64, 128):
            raise ValueError("q8_group must be 0, 64 or 128")
        groups = -(-d // q8_group) if q8_group else 1
        if q8_scale is None:
            q8_scale = _empty((T, groups), X.f32, h.device, stream)
        if q8.shape == shape and q8.get_device() == dev and q8.is_contiguous():
            qp, qs = q8.data_ptr(), d
        else:
            qp, qs = _rows(q8, "q8", shape, d, q8.dtype, dev)
        sp = _flat(q8_scale, "q8_scale", (T, groups), X.f32, dev)
    _call(X, dev, stream, X.add_rmsnorm, hp, hs, dp, f32, ds, _flat(norm_w, "norm_w", (d,), bf16, dev), eps, T, d, op, os_, xp, xs,
          qp, fmt, qs, q8_group, sp)
    return h_out, x, q8, q8_scale


class Int4Linear:
    """A matrix in the int4 affine group format with an optional unmerged LoRA, applied to few
    tokens (see e0_int4_linear in the C header): codes [n, k/2] uint8, scale and min [n, k/g]
    bf16 with g = 64 or 128, lora_A [r, k] and lora_B [n, r] bf16.  Keeps the tensors."""

    def __init__(self, codes, scale, min, lora_A=None, lora_B=None, lora_scale=1.0):
        X = _torch()
        bf16, dev = X.bf16, codes.get_device()
        self.device, self.n, self.k = codes.device, codes.shape[0], 2 * codes.shape[1]
        self.group = self.k // scale.shape[1] if scale.dim() == 2 and scale.shape[1] else 0
        if self.group not in (64, 128) or self.k % self.group:
            raise ValueError(f"scale [n, k/g] must have g = 64 or 128 for k = {self.k}, got {tuple(scale.shape)}")
        if (lora_A is None) != (lora_B is None):
            raise ValueError("LoRA needs both matrices")
        r = lora_A.shape[0] if lora_A is not None else 0
        shape = (self.n, self.k // self.group)
        self._keep = (codes, scale, min, lora_A, lora_B)
        self._mat = Int4Mat(_flat(codes, "codes", (self.n, self.k // 2), X.u8, dev),
                            _flat(scale, "scale", shape, bf16, dev), _flat(min, "min", shape, bf16, dev),
                            self.n, self.k, self.group, _flat(lora_A, "lora_A", (r, self.k), bf16, dev),
                            _flat(lora_B, "lora_B", (self.n, r), bf16, dev), r, lora_scale)
        self._ref, self._dev = ctypes.byref(self._mat), dev

    def __call__(self, x, x_scale=None, y=None, stream=None):
        """x [T, k] bf16, or int8 / float8_e4m3fn with x_scale [T, 1], [T, k/64] or [T, k/128]
        fp32 (as add_rmsnorm writes them) -> y [T, n], bf16 or fp32 (bf16 where it is
        allocated here)."""
        X = _torch()
        dev, k, n, T = self._dev, self.k, self.n, x.shape[0]
        fmt = _act_format(x)
        xp, xs = _rows(x, "x", (T, k), k, x.dtype, dev)
        x_group, sp = 0, None
        if x_scale is not None:
            groups = x_scale.shape[-1]
            x_group = 0 if groups <= 1 else k // groups
            if x_group not in (0, 64, 128):
                raise ValueError(f"x_scale: expected 1, k/64 or k/128 scales a row, got {groups}")
            sp = _flat(x_scale, "x_scale", (T, k // x_group if x_group else 1), X.f32, dev)
        if y is None:
            y = _empty((T, n), X.bf16, self.device, stream)
        f32 = y.dtype is X.f32
        yp, ys = _rows(y, "y", (T, n), n, X.f32 if f32 else X.bf16, dev)
        _call(X, dev, stream, X.int4_linear, self._ref, xp, fmt, xs, sp, x_group, T, yp, f32, ys)
        return y


def _layer_shapes(dims):
    """Shapes of a layer's tensors: the experts' bytes as uint8, the others bf16."""
    d, E, I, r = dims.d_model, dims.n_experts, dims.d_ff, dims.lora_rank
    blob = 3 * (I * d // 2 + 4 * I * (d // 64))         # codes, scales and mins of gate, up and down
    return {"experts": (E, blob), "shared": (blob,), "router_w": (E, d), "norm_w": (d,),
            "lora_Ag": (r, d), "lora_Bg": (I, r), "lora_Au": (r, d), "lora_Bu": (I, r), "lora_Ad": (r, I), "lora_Bd": (d, r)}


class MoeLayer:
    """One MoE layer's resident weights, for few tokens without a context (see
    e0_moe_layer_few in the C header).  `layer` is a dict of torch tensors as for
    Context.register_model, all on one device; it keeps them."""

    def __init__(self, dims: Dims, layer: dict):
        X = _torch()
        self.dims = Dims.from_buffer_copy(dims)
        self._keep = {f: layer.get(f) for f, _ in Layer._fields_}
        there = {f: t for f, t in self._keep.items() if t is not None}
        self.device = next((t.device for t in there.values()), None)
        self._dev = -1 if self.device is None or self.device.type != "cuda" else next(iter(there.values())).get_device()
        shapes = _layer_shapes(dims)
        self._layer = Layer()
        for f, t in there.items():
            if t.device != self.device:
                raise ValueError(f"{f}: on {t.device}, the layer's other tensors are on {self.device}")
            setattr(self._layer, f, _flat(t, f, shapes[f], X.u8 if f in ("experts", "shared") else X.bf16, t.get_device()))

    def few_workspace(self, T: int):
        """A workspace for calls of at most T tokens (calls that may overlap need one each)."""
        return _few_workspace(self.dims, T, self.device)

    def few(self, h, delta=None, route_idx=None, h_out=None, y=None, y_f32=None, idx=None, gates=None, workspace=None,
            dev_status=None, stream=None):
        """The MoE block of 1..64 tokens in one launch: h' = bf16(h + delta) [T, d] (to h_out
        where given; it may be h), y [T, d] bf16 = the block's output for h'.  Without
        `workspace` one is allocated for the call."""
        if h.get_device() != self._dev:
            raise ValueError(f"h: on {h.device}, the layer is on {self.device}")
        return _moe_layer_few(self.dims, self._layer, h, delta, route_idx, h_out, y, y_f32, idx, gates,
                              workspace, dev_status, stream)


def _moe_layer_few(dims, layer, h, delta, route_idx, h_out, y, y_f32, idx, gates, workspace, dev_status, stream):
    X = _torch()
    bf16, f32, i32, dev, T = X.bf16, X.f32, X.i32, h.get_device(), h.shape[0]
    shape, per_k = (T, dims.d_model), (T, dims.top_k)
    hp = _flat(h, "h", shape, bf16, dev)
    if y is None:
        y = _empty(shape, bf16, h.device, stream)
    if workspace is None:
        workspace = _few_workspace(dims, T, h.device, stream)
    _call(X, dev, stream, X.moe_layer_few, ctypes.byref(dims), ctypes.byref(layer), hp,
          _flat(delta, "delta", shape, bf16, dev), T, _flat(route_idx, "route_idx", per_k, i32, dev),
          _flat(h_out, "h_out", shape, bf16, dev), _flat(y, "y", shape, bf16, dev), _flat(y_f32, "y_f32", shape, f32, dev),
          _flat(idx, "idx", per_k, i32, dev), _flat(gates, "gates", per_k, f32, dev),
          _flat(workspace, "workspace", (workspace.numel(),), X.u8, dev), workspace.numel(),
          _flat(dev_status, "dev_status", (1,), i32, dev))
    return y


class Context:
    """One ``e0_ctx``: workspaces, routing tables and (optionally) the streaming pool."""

    def __init__(self, d, E, I, k, r, n_layers, max_tokens, head_hidden=0, head_onehot=0,
                 eps=1e-6, lora_scale=1.0):
        self.dims = make_dims(d, E, I, k, r, head_hidden, head_onehot, eps, lora_scale)
        self.n_layers, self.max_tokens = n_layers, max_tokens
        self._keep = []
        self._layers, self._few = [], {}
        h = _P()
        _check(lib().e0_create(ctypes.byref(self.dims), n_layers, max_tokens, ctypes.byref(h)))
        self._h = h

    # -- lifetime ---------------------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None):
            lib().e0_destroy(self._h)
            self._h = None
            self._keep = []
            self._layers, self._few = [], {}

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- weights ----------------------------------------------------------------------
    def register_model(self, layers: list, heads: Optional[list] = None):
        """layers[l]: dict with torch tensors experts [E, blob] (or None), shared [blob],
        router_w [E, d], norm_w [d], and optionally lora_Ag..lora_Bd.  heads[l]: dict with
        w_lin (and fc1_w, fc1_b, fc2_w, fc2_b) or None."""
        L = (Layer * self.n_layers)()
        H = (Head * self.n_layers)()
        for i, ly in enumerate(layers):
            for f, _ in Layer._fields_:
                t = ly.get(f)
                setattr(L[i], f, _ptr(t))
                self._keep.append(t)
            hd = heads[i] if heads is not None else None
            for f, _ in Head._fields_:
                t = hd.get(f) if hd else None
                setattr(H[i], f, _ptr(t))
                self._keep.append(t)
        _check(lib().e0_register_model(self._h, L, H))
        self._layers, self._few = [dict(ly) for ly in layers], {}

    # -- one MoE block ------------------------------------------------------------------
    def moe_layer_forward(self, layer, h, route_idx=None, y=None, y_f32=None, idx=None, gates=None,
                          stream=None):
        import torch
        T = h.shape[0]
        d, k = self.dims.d_model, self.dims.top_k
        if y is None:
            y = torch.empty((T, d), dtype=torch.bfloat16, device=h.device)
        _check(lib().e0_moe_layer_forward(self._h, layer, _ptr(h), T, _ptr(route_idx), _ptr(y), _ptr(y_f32),
                                          _ptr(idx), _ptr(gates), _stream(stream)))
        return y

    def moe_layer_few(self, layer, h, delta=None, route_idx=None, h_out=None, y=None, y_f32=None, idx=None, gates=None,
                      workspace=None, dev_status=None, stream=None):
        """The MoE block of a registered layer for 1..64 tokens in one launch (see MoeLayer.few;
        it uses none of the context's workspaces)."""
        if self._h is None:
            raise E0Error(E0_ERR_INVALID_ARG, "moe_layer_few: the context is closed")
        if not 0 <= layer < len(self._layers):
            raise IndexError(f"layer {layer} of {len(self._layers)} registered")
        if layer not in self._few:
            self._few[layer] = MoeLayer(self.dims, self._layers[layer])
        return self._few[layer].few(h, delta, route_idx, h_out, y, y_f32, idx, gates, workspace, dev_status, stream)

    def prerouter_predict(self, layer, x, cur=None, prev=None, pred=None, logits=None, stream=None):
        import torch
        T = x.shape[0]
        if pred is None:
            pred = torch.empty((T, self.dims.top_k), dtype=torch.int32, device=x.device)
        _check(lib().e0_prerouter_predict(self._h, layer, _ptr(x), T, _ptr(cur), _ptr(prev), _ptr(pred),
                                          _ptr(logits), _stream(stream)))
        return pred

    # -- streaming tier ------------------------------------------------------------------
    def stream_register(self, host_blob, pool_layers=2, slots_per_layer=None):
        if slots_per_layer is None:
            slots_per_layer = self.dims.top_k
        if not host_blob.is_pinned():
            raise ValueError("the host expert store must be pinned memory")
        self._keep.append(host_blob)
        blob = host_blob.shape[-1]
        _check(lib().e0_stream_register(self._h, _ptr(host_blob), blob, pool_layers, slots_per_layer))

    def stream_mode(self, reactive: bool):
        """False: prerouter prefetch (default); True: every layer routes itself and stages
        on demand (no prediction).  Starts a new sequence."""
        _check(lib().e0_stream_mode(self._h, int(reactive)))

    def debug_stream_log(self, log):
        """log: int32 CUDA tensor [L, slots_per_layer] or None."""
        self._keep.append(log)
        _check(lib().e0_debug_stream_log(self._h, _ptr(log)))

    def debug_pool_slot(self, pool_set, slot) -> int:
        out = _P()
        _check(lib().e0_debug_pool_slot(self._h, pool_set, slot, ctypes.byref(out)))
        return int(out.value)

    def stage_experts(self, layer, experts, stream=None):
        arr = (ctypes.c_int32 * len(experts))(*[int(e) for e in experts])
        _check(lib().e0_stage_experts(self._h, layer, arr, len(experts), _stream(stream)))

    # -- decode over the stack ------------------------------------------------------------
    def stack_decode(self, h_in, step, y_out=None, y_f32=None, streaming=False, chained=False, stream=None):
        import torch
        L, B, d = h_in.shape
        if y_out is None:
            y_out = torch.empty((L, B, d), dtype=torch.bfloat16, device=h_in.device)
        _check(lib().e0_moe_stack_decode(self._h, _ptr(h_in), B, step, _ptr(y_out), _ptr(y_f32),
                                         int(streaming), int(chained), _stream(stream)))
        return y_out

    def stack_decode_host(self, h_host, step, y_host, y_f32_host=None, streaming=False, chained=False, stream=None):
        """One decode step with host (pinned) tensors; the library overlaps the copies with
        the kernels.  The outputs are complete after host_io_wait(stream) and a
        synchronisation of the stream."""
        L, B, d = h_host.shape
        assert not h_host.is_cuda and not y_host.is_cuda and (y_f32_host is None or not y_f32_host.is_cuda)
        _check(lib().e0_moe_stack_decode_host(self._h, _ptr(h_host), B, step, _ptr(y_host), _ptr(y_f32_host),
                                              int(streaming), int(chained), _stream(stream)))
        return y_host

    def host_io_wait(self, stream=None):
        _check(lib().e0_host_io_wait(self._h, _stream(stream)))

    def prefill_stack_host(self, h_host, y_host, y_f32_host=None, idx=None, stream=None):
        """prefill_stack with pinned host tensors h_host, y_host [L, T, d] bf16 (y_f32_host
        [L, T, d] fp32 or None; idx a CUDA int32 tensor [L, T, k] or None).  The library
        overlaps each layer's copies with the neighbouring layers' kernels; the outputs are
        complete after host_io_wait(stream) and a synchronisation of the stream."""
        L, T, d = h_host.shape
        assert not h_host.is_cuda and not y_host.is_cuda and (y_f32_host is None or not y_f32_host.is_cuda)
        _check(lib().e0_moe_prefill_stack_host(self._h, _ptr(h_host), T, _ptr(y_host), _ptr(y_f32_host), _ptr(idx),
                                               _stream(stream)))
        return y_host

    def prefill_stack(self, h_in, y_out=None, y_f32=None, idx=None, stream=None):
        """h_in [L, T, d] bf16 -> y_out [L, T, d] bf16 (prediction-as-routing, one token ahead)."""
        import torch
        L, T, d = h_in.shape
        if y_out is None:
            y_out = torch.empty((L, T, d), dtype=torch.bfloat16, device=h_in.device)
        _check(lib().e0_moe_prefill_stack(self._h, _ptr(h_in), T, _ptr(y_out), _ptr(y_f32), _ptr(idx),
                                          _stream(stream)))
        return y_out

    def get_routing(self, B):
        import numpy as np
        k = self.dims.top_k
        idx = np.zeros((self.n_layers, B, k), dtype=np.int32)
        pred = np.zeros((self.n_layers, B, k), dtype=np.int32)
        _check(lib().e0_get_routing(self._h, B, idx.ctypes.data, pred.ctypes.data))
        return idx, pred

    def stats(self) -> dict:
        s = Stats()
        _check(lib().e0_get_stats(self._h, ctypes.byref(s)))
        return {f: getattr(s, f) for f, _ in Stats._fields_}

    def sync_status(self):
        _check(lib().e0_sync_status(self._h))

    # -- host-side fault injection (tests) ------------------------------------------------
    def debug_fail_staging_after(self, n):
        _check(lib().e0_debug_fail_staging_after(self._h, n))

    def debug_set_slot_tag(self, pool_set, slot, expert):
        _check(lib().e0_debug_set_slot_tag(self._h, pool_set, slot, expert))

    def debug_decode_stall(self, cta, timeout_ns):
        _check(lib().e0_debug_decode_stall(self._h, cta, timeout_ns))

    def debug_decode_trace(self, buf):
        """buf: int64 CUDA tensor [grid, L, 16] or None; returns the grid size."""
        return lib().e0_debug_decode_trace(self._h, _ptr(buf))

    def debug_decode_mode(self, mode: int):
        _check(lib().e0_debug_decode_mode(self._h, mode))

    def debug_phase_timing(self, on: bool):
        _check(lib().e0_debug_phase_timing(self._h, int(on)))

    def debug_phase_times(self):
        """(per-kernel summed ms of the phased decode kernels [norm, rows, route, gate/up,
        sums+t_d, down], steps timed)."""
        ms = (ctypes.c_double * 6)()
        n = ctypes.c_ulonglong(0)
        _check(lib().e0_debug_phase_times(self._h, ms, ctypes.byref(n)))
        return list(ms), int(n.value)

    def debug_time_gemm(self, on: bool):
        _check(lib().e0_debug_time_gemm(self._h, int(on)))

    def debug_decode_flat(self, on: bool):
        _check(lib().e0_debug_decode_flat(self._h, int(on)))

    def debug_prefill_path(self, mode: int):
        _check(lib().e0_debug_prefill_path(self._h, mode))

    def prefill_fixed_order(self, on: bool):
        """Tensor-core prefill combine in slot order (bit-reproducible y) instead of
        completion-order reductions."""
        _check(lib().e0_prefill_fixed_order(self._h, int(on)))

    def debug_force_general(self, on: bool):
        _check(lib().e0_debug_force_general(self._h, int(on)))
