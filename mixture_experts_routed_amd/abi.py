"""ctypes binding of libmoe_routed.so (the C ABI in include/moe_routed.h).

Argument marshalling only: every step of the layer runs in the library's HIP
kernels. PyTorch supplies device memory and the stream. The functions named
like the C entry points take torch tensors (and plain ints) in the C order
and raise MoeError on a non-OK status; the short-named helpers below them
allocate outputs with torch and call those.

There is no fallback: if the library is missing or no GPU tensor is given,
the call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# a different build of the same sources may be named here (the tests load a
# build whose host code carries AddressSanitizer this way)
LIB_PATH = os.environ.get("MOE_ROUTED_LIB_OVERRIDE") or os.path.join(HERE, "libmoe_routed.so")

MOE_F32, MOE_F16, MOE_BF16 = 0, 1, 2
MOE_W_GATE_UP, MOE_W_DOWN = 0, 1
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "HIP runtime error",
          4: "larger than the allocation-free call's fixed buffer"}
NOALLOC_WORKSPACE_BYTES = 64 << 20  # MOE_NOALLOC_WORKSPACE_BYTES
META_FIELDS = ("nent", "nblk", "nr", "nt", "nactive", "maxcnt", "nskip", "nbad", "tm", "E", "K")
META_N = 11
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}  # enum moe_act
MOE_GRAD_X, MOE_GRAD_W, MOE_GRAD_BIAS = 1, 2, 4
ACT8_BLOCK = 32  # MOE_ACT8_BLOCK
SCORES = {"softmax": 0, "sigmoid": 1}  # enum moe_score
GATES = {"none": 0, "token": 1, "channel": 2, "full": 3}  # enum moe_gate
NORM_GRADS = frozenset(("dr", "dy", "dgate", "dw_post", "dw_pre"))
MX4_KINDS = {"gate": MOE_W_GATE_UP, "down": MOE_W_DOWN}  # gate: gate and up matrices
STAGES = ("hist", "scan", "place", "gather", "worklist", "gateup", "down", "combine")
TORCH_DTYPE = {MOE_F32: torch.float32, MOE_F16: torch.float16, MOE_BF16: torch.bfloat16}
DTYPE_OF = {torch.float32: MOE_F32, torch.float16: MOE_F16, torch.bfloat16: MOE_BF16}
DTYPE_NAME = {"f32": MOE_F32, "f16": MOE_F16, "bf16": MOE_BF16}


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {STATUS.get(status, status)} (status {status})")
        self.status = status


class PlanSizes(ctypes.Structure):
    _fields_ = [("nent", ctypes.c_int64), ("nblk", ctypes.c_int64), ("max_rows", ctypes.c_int64),
                ("max_tiles", ctypes.c_int64), ("scratch_bytes", ctypes.c_size_t)]


class ForwardLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("cnt", "eoff", "tiles", "stok", "sw", "pos", "boff", "meta", "plan_scratch", "xs",
                 "h", "y", "ffn_scratch", "total")]


_lib = None
P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
F32 = ctypes.c_float

_SIGS = {
    "moe_route_topk": [P, I32, I32, I32, P, P, P],
    "moe_plan_sizes": [I32, I32, I32, I32, ctypes.POINTER(PlanSizes)],
    "moe_plan": [P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, P, SZ, P],
    "moe_gather": [P, I32, I32, I32, P, P, I64, P, P],
    "moe_ffn_scratch_bytes": [I32, I32, I32, I32, I64, I32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_ffn_splits": [I32, I32, I32, I32, I64, I32, ctypes.POINTER(ctypes.c_int),
                       ctypes.POINTER(ctypes.c_int)],
    "moe_ffn_big_cells": [I32, I32, I32, I32, I64, I32, ctypes.POINTER(ctypes.c_int)],
    "moe_expert_ffn": [P, P, P, P, I32, I32, I32, I32, I32, P, P, P, P, I64, P, P, P, SZ, P],
    "moe_combine": [P, I64, P, I32, I32, I32, P, P],
    "moe_forward_workspace": [I32, I32, I32, I32, I32, I32, I32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_forward_layout": [I32, I32, I32, I32, I32, I32, I32, ctypes.POINTER(ForwardLayout)],
    "moe_forward": [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, P, SZ, P, P],
    "moe_forward_timed": [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, P, SZ, P, P, P],
    "moe_timer_create": [ctypes.POINTER(P), I32, ctypes.c_uint],
    "moe_timer_destroy": [P],
    "moe_timer_read": [P, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)],
    "moe_packed_weight_bytes": [I32, I32, I32, I32, I32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_pack_weights": [P, I32, I32, I32, I32, I32, P, SZ, P],
    "moe_expert_ffn_packed": [P, P, P, P, I32, I32, I32, I32, I32, P, P, P, P, I64, P, P, P, SZ,
                              P],
    "moe_forward_packed": [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, P, SZ, P, P],
    "moe_host_cache_bytes": [I32, I32, I32, I32, I32, I32, I32, I32,
                             ctypes.POINTER(ctypes.c_size_t)],
    "moe_host_cache_init": [P, SZ, I32, I32, I32, I32, I32, I32, P],
    "moe_forward_host_weights": [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, I32, I32, P,
                                 SZ, P, SZ, P, P],
    "moe_forward_packed_timed": [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, P, SZ, P, P,
                                 P],
    "moe_linear_workspace": [I32, I32, I32, I64, I64, I32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_linear_shape": [I32, I32, I32, I32, ctypes.POINTER(ctypes.c_int),
                         ctypes.POINTER(ctypes.c_int)],
    "moe_linear": [P, I64, P, I64, P, P, I64, I32, I32, I32, I32, I32, I32, P, SZ, P, I64, I32, P],
    "moe_linear_backward_workspace": [I32, I32, I32, I64, I64, I64, I32, I32,
                                      ctypes.POINTER(ctypes.c_size_t)],
    "moe_linear_backward": [P, I64, P, I64, P, I64, I32, I32, I32, I32, P, SZ, P, I64, P, I64, P,
                            I32, P],
    "moe_balance_workspace": [I32, I32, I32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_balance_loss": [P, P, I32, I32, I32, P, SZ, P, P, P, P],
    "moe_route_backward": [P, P, P, P, P, P, I32, I32, I32, P, I32, P],
    "moe_act_forward": [P, I64, P, I64, I32, I32, I32, I32, P, I64, P, P, P, P, P],
    "moe_act_backward": [P, P, P, P, P, I64, I32, I32, I32, I32, P, I64, P, I64, P, I64, P],
    "moe_mx4_weight_bytes": [I32, I32, I32, I32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_mx4_quantize": [P, I32, I32, I32, I32, I32, P, SZ, P],
    "moe_mx4_dequantize": [P, SZ, I32, I32, I32, I32, P, I32, P],
    "moe_forward_mx4": [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, P, SZ, P, I32, P],
    "moe_route_scored": [P, P, I32, I32, I32, I32, I32, I32, I32, I32, F32, P, P, P],
    "moe_route_scored_backward": [P, P, P, P, I32, I32, I32, I32, I32, F32, P, I32, P],
    "moe_norm": [P, I64, I32, P, I64, I32, P, P, I64, I32, P, I32, I32, I32, F32, F32, P, I64, P,
                 I64, P, P],
    "moe_norm_backward_workspace": [I32, I32, ctypes.POINTER(ctypes.c_size_t)],
    "moe_norm_backward": [P, I64, P, I64, P, I64, I32, P, I64, I32, P, P, I64, I32, P, P, I32, I32,
                          I32, F32, P, SZ, P, I64, P, I64, P, I64, P, P, I32, P],
    "moe_forward_packed_noalloc": [P, P, P, P, P, P, I32, I32, I32, I32, I32, I32, I32, P, P],
}

EXPORTS = tuple(_SIGS) + ("moe_status_str",)


def lib():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoeError("load", 3) from FileNotFoundError(
                f"{LIB_PATH} is missing: build it with mixture_experts_routed_amd.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = I32
        L.moe_status_str.argtypes = [I32]
        L.moe_status_str.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(fn: str, rc: int):
    if rc != 0:
        raise MoeError(fn, rc)


def _dev(t, name):
    """device address of a CUDA tensor (or None)"""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _mat(t, name, dev, rows, cols, dtype, other=None, read=True):
    """(device address, row stride) of a row-major matrix [rows, cols] of dtype (or
    `other`) on GPU `dev`; (None, 0) for None. read: by this call, or written"""
    if t is None:
        return None, 0
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a GPU tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected GPU {dev}")
    if t.dtype is not dtype and (other is None or t.dtype is not other):
        raise TypeError(f"{name}: expected {dtype}{f' or {other}' if other else ''}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: expected {(rows, cols)}, got {tuple(t.shape)}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name}: expected contiguous rows")
    if rows <= 1:
        s0 = cols
    elif s0 < cols:
        raise ValueError(f"{name}: overlapping rows")
    p = t.data_ptr()
    if p & 15 and read:
        raise ValueError(f"{name}: the first element is not 16-byte aligned")
    return p, s0


def _vec(t, name, dev, n, dtype, align=1):
    """device address of a contiguous array of n elements of dtype on GPU `dev` (or None)"""
    if t is None:
        return None
    p = _dev(t, name)
    if p % align:
        raise ValueError(f"{name}: the first element is not {align}-byte aligned")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected GPU {dev}")
    if t.numel() != n or t.dtype is not dtype:
        raise ValueError(f"{name}: expected {n} elements of {dtype}, got {tuple(t.shape)} {t.dtype}")
    return p


def _dtype(name, dtype):
    """the C ABI's code of a torch type"""
    if dtype not in DTYPE_OF:
        raise TypeError(f"{name}: expected float32, float16 or bfloat16, got {dtype}")
    return DTYPE_OF[dtype]


def _act(act):
    """the C ABI's code of an activation's name"""
    return _named("act", act, ACTS)


def _named(name, value, of):
    """the C ABI's code of a named choice"""
    if value not in of:
        raise ValueError(f"{name}: expected one of {', '.join(of)}, got {value!r}")
    return of[value]


def _host(t, name):
    """address of a host tensor (the library checks that it is pinned)"""
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f"{name}: expected a host tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


# --------------------------------------------------------- host-only sizes --

def moe_plan_sizes(T: int, K: int, E: int, tm: int) -> PlanSizes:
    z = PlanSizes()
    _check("moe_plan_sizes", lib().moe_plan_sizes(T, K, E, tm, ctypes.byref(z)))
    return z


def moe_ffn_scratch_bytes(E: int, d: int, f: int, tm: int, max_rows: int, dtype: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_ffn_scratch_bytes",
           lib().moe_ffn_scratch_bytes(E, d, f, tm, max_rows, dtype, ctypes.byref(v)))
    return v.value


def moe_ffn_splits(E: int, d: int, f: int, tm: int, max_rows: int, dtype: int):
    """(gate/up splits, down splits) of the reduction for these sizes."""
    a, b = ctypes.c_int(), ctypes.c_int()
    _check("moe_ffn_splits",
           lib().moe_ffn_splits(E, d, f, tm, max_rows, dtype, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def moe_ffn_big_cells(E: int, d: int, f: int, tm: int, max_rows: int, dtype: int) -> int:
    """which packed 16-bit projections run their runs of 4 items on the 8-wavefront
    kernel: bit 0 gate/up, bit 1 down"""
    on = ctypes.c_int()
    _check("moe_ffn_big_cells",
           lib().moe_ffn_big_cells(E, d, f, tm, max_rows, dtype, ctypes.byref(on)))
    return on.value


def moe_forward_workspace(T, K, E, d, f, tm, dtype: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_forward_workspace", lib().moe_forward_workspace(T, K, E, d, f, tm, dtype,
                                                                ctypes.byref(v)))
    return v.value


def moe_forward_layout(T, K, E, d, f, tm, dtype: int) -> ForwardLayout:
    L = ForwardLayout()
    _check("moe_forward_layout", lib().moe_forward_layout(T, K, E, d, f, tm, dtype, ctypes.byref(L)))
    return L


def moe_status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


# ------------------------------------------------ entry points (same names) --

def moe_route_topk(logits, T, E, K, ids, w, stream=None):
    _check("moe_route_topk", lib().moe_route_topk(_dev(logits, "logits"), T, E, K, _dev(ids, "ids"),
                                                  _dev(w, "w"), _stream(stream)))


def moe_plan(ids, w, T, K, E, tm, cnt, eoff, tiles, stok, sw, pos, boff, meta, scratch,
             stream=None):
    _check("moe_plan", lib().moe_plan(
        _dev(ids, "ids"), _dev(w, "w"), T, K, E, tm, _dev(cnt, "cnt"), _dev(eoff, "eoff"),
        _dev(tiles, "tiles"), _dev(stok, "stok"), _dev(sw, "sw"), _dev(pos, "pos"),
        _dev(boff, "boff"), _dev(meta, "meta"), _dev(scratch, "scratch"),
        scratch.numel() * scratch.element_size(), _stream(stream)))


def moe_gather(x, dtype, T, d, stok, meta, max_rows, xs, stream=None):
    _check("moe_gather", lib().moe_gather(_dev(x, "x"), dtype, T, d, _dev(stok, "stok"),
                                          _dev(meta, "meta"), max_rows, _dev(xs, "xs"),
                                          _stream(stream)))


def moe_packed_weight_bytes(E: int, d: int, f: int, dtype: int, kind: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_packed_weight_bytes",
           lib().moe_packed_weight_bytes(E, d, f, dtype, kind, ctypes.byref(v)))
    return v.value


def moe_pack_weights(w, kind: int, packed=None, stream=None):
    """Pack one set of expert matrices (W_gate/W_up [E, d, f] with kind
    MOE_W_GATE_UP, W_down [E, f, d] with MOE_W_DOWN); returns the packed bytes."""
    E = w.shape[0]
    d, f = (w.shape[1], w.shape[2]) if kind == MOE_W_GATE_UP else (w.shape[2], w.shape[1])
    dtype = DTYPE_OF[w.dtype]
    need = moe_packed_weight_bytes(E, d, f, dtype, kind)
    if packed is None:
        packed = torch.empty(need, dtype=torch.uint8, device=w.device)
    _check("moe_pack_weights", lib().moe_pack_weights(
        _dev(w, "w"), dtype, E, d, f, kind, _dev(packed, "packed"),
        packed.numel() * packed.element_size(), _stream(stream)))
    return packed


def pack(w_gate, w_up, w_down, stream=None) -> dict:
    """The three packed matrix sets of a layer, keyed gate / up / down."""
    return {"gate": moe_pack_weights(w_gate, MOE_W_GATE_UP, stream=stream),
            "up": moe_pack_weights(w_up, MOE_W_GATE_UP, stream=stream),
            "down": moe_pack_weights(w_down, MOE_W_DOWN, stream=stream)}


def moe_expert_ffn_packed(xs, pw_gate, pw_up, pw_down, dtype, E, d, f, tm, eoff, stok, sw, meta,
                          max_rows, h, y, scratch, stream=None):
    _check("moe_expert_ffn_packed", lib().moe_expert_ffn_packed(
        _dev(xs, "xs"), _dev(pw_gate, "pw_gate"), _dev(pw_up, "pw_up"), _dev(pw_down, "pw_down"),
        dtype, E, d, f, tm, _dev(eoff, "eoff"), _dev(stok, "stok"), _dev(sw, "sw"),
        _dev(meta, "meta"), max_rows, _dev(h, "h"), _dev(y, "y"), _dev(scratch, "scratch"),
        scratch.numel() * scratch.element_size(), _stream(stream)))


def moe_expert_ffn(xs, w_gate, w_up, w_down, dtype, E, d, f, tm, eoff, stok, sw, meta, max_rows,
                   h, y, scratch, stream=None):
    _check("moe_expert_ffn", lib().moe_expert_ffn(
        _dev(xs, "xs"), _dev(w_gate, "w_gate"), _dev(w_up, "w_up"), _dev(w_down, "w_down"), dtype,
        E, d, f, tm, _dev(eoff, "eoff"), _dev(stok, "stok"), _dev(sw, "sw"), _dev(meta, "meta"),
        max_rows, _dev(h, "h"), _dev(y, "y"), _dev(scratch, "scratch"),
        scratch.numel() * scratch.element_size(), _stream(stream)))


def moe_combine(y, max_rows, pos, T, K, d, out, stream=None):
    _check("moe_combine", lib().moe_combine(_dev(y, "y"), max_rows, _dev(pos, "pos"), T, K, d,
                                            _dev(out, "out"), _stream(stream)))


def moe_forward(x, ids, w, w_gate, w_up, w_down, dtype, T, K, E, d, f, tm, workspace, out,
                stream=None, timer=None, packed: bool = False):
    """packed=True: w_gate / w_up / w_down are packed matrix sets (moe_pack_weights)."""
    args = (_dev(x, "x"), _dev(ids, "ids"), _dev(w, "w"), _dev(w_gate, "w_gate"),
            _dev(w_up, "w_up"), _dev(w_down, "w_down"), dtype, T, K, E, d, f, tm,
            _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
            _dev(out, "out"), _stream(stream))
    name = "moe_forward_packed" if packed else "moe_forward"
    if timer is None:
        _check(name, getattr(lib(), name)(*args))
    else:
        _check(name + "_timed", getattr(lib(), name + "_timed")(*args, timer.handle))


def moe_forward_packed_noalloc(x, ids, w, pw_gate, pw_up, pw_down, dtype, T, K, E, d, f, tm, out,
                               stream=None):
    """moe_forward_packed with the library's fixed workspace (no workspace argument)."""
    _check("moe_forward_packed_noalloc", lib().moe_forward_packed_noalloc(
        _dev(x, "x"), _dev(ids, "ids"), _dev(w, "w"), _dev(pw_gate, "pw_gate"),
        _dev(pw_up, "pw_up"), _dev(pw_down, "pw_down"), dtype, T, K, E, d, f, tm,
        _dev(out, "out"), _stream(stream)))


def moe_host_cache_bytes(T: int, K: int, E: int, d: int, f: int, dtype: int, packed: bool,
                         slots: int = 0) -> int:
    n = ctypes.c_size_t()
    _check("moe_host_cache_bytes", lib().moe_host_cache_bytes(T, K, E, d, f, dtype, int(packed),
                                                              slots, ctypes.byref(n)))
    return n.value


def moe_host_cache_init(cache, E, d, f, dtype, packed: bool, slots: int, stream=None):
    _check("moe_host_cache_init", lib().moe_host_cache_init(
        _dev(cache, "cache"), cache.numel() * cache.element_size(), E, d, f, dtype, int(packed),
        slots, _stream(stream)))


def moe_forward_host_weights(x, ids, w, hw_gate, hw_up, hw_down, packed: bool, dtype, T, K, E, d,
                             f, tm, slots, cache, workspace, out, stream=None):
    """moe_forward / moe_forward_packed with the expert weights in pinned host tensors."""
    _check("moe_forward_host_weights", lib().moe_forward_host_weights(
        _dev(x, "x"), _dev(ids, "ids"), _dev(w, "w"), _host(hw_gate, "hw_gate"),
        _host(hw_up, "hw_up"), _host(hw_down, "hw_down"), int(packed), dtype, T, K, E, d, f, tm,
        slots, _dev(cache, "cache"), cache.numel() * cache.element_size(),
        _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
        _dev(out, "out"), _stream(stream)))


class Timer:
    """Per-kernel HIP-event timer of moe_forward_timed."""

    def __init__(self, capacity: int = 256, stages=STAGES):
        h = ctypes.c_void_p()
        mask = 0
        for s in stages:
            mask |= 1 << STAGES.index(s)
        _check("moe_timer_create", lib().moe_timer_create(ctypes.byref(h), capacity, mask))
        self.handle = h
        self.total_ms = (ctypes.c_double * len(STAGES))()
        self.launches = (ctypes.c_int64 * len(STAGES))()

    def read(self) -> dict:
        """Wait for the recorded events and accumulate; returns {stage: (ms_total, launches)}."""
        _check("moe_timer_read", lib().moe_timer_read(self.handle, self.total_ms, self.launches))
        return {s: (self.total_ms[i], self.launches[i]) for i, s in enumerate(STAGES)}

    def reset(self):
        for i in range(len(STAGES)):
            self.total_ms[i] = 0.0
            self.launches[i] = 0

    def close(self):
        if self.handle:
            lib().moe_timer_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------ allocating helpers --

def _empty(n, dtype, device):
    return torch.empty(int(max(n, 1)), dtype=dtype, device=device)


def route(logits, K: int, stream=None):
    """Router on GPU logits [T, E] fp32: returns (ids [T, K] int32, w [T, K] fp32)."""
    T, E = logits.shape
    ids = torch.empty((T, K), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, K), dtype=torch.float32, device=logits.device)
    moe_route_topk(logits, T, E, K, ids, w, stream)
    return ids, w


def plan(ids, w, E: int, tm: int = 16, stream=None) -> dict:
    """Run moe_plan on ids/w ([T, K] int32 / fp32 GPU tensors); returns the outputs."""
    T, K = ids.shape
    z = moe_plan_sizes(T, K, E, tm)
    dev = ids.device
    o = dict(cnt=_empty(E, torch.int32, dev), eoff=_empty(E + 1, torch.int32, dev),
             tiles=_empty(z.max_tiles, torch.int32, dev), stok=_empty(z.max_rows, torch.int32, dev),
             sw=_empty(z.max_rows, torch.float32, dev), pos=_empty(T * K, torch.int32, dev),
             boff=_empty(z.nblk * E, torch.int32, dev), meta=_empty(META_N, torch.int32, dev),
             scratch=_empty(z.scratch_bytes, torch.uint8, dev))
    moe_plan(ids, w, T, K, E, tm, o["cnt"], o["eoff"], o["tiles"], o["stok"], o["sw"], o["pos"],
             o["boff"], o["meta"], o["scratch"], stream)
    o["sizes"] = z
    return o


def forward(x, ids, w, w_gate, w_up, w_down, tm: int = 16, workspace=None, out=None, stream=None,
            timer=None, packed=None):
    """One routed MoE layer on GPU tensors; returns (out [T, d] fp32, workspace).
    packed: optional dict of packed matrix sets (see pack()); the layer then reads
    those instead of w_gate / w_up / w_down, which still give the shapes."""
    T, d = x.shape
    K = ids.shape[1]
    E, _, f = w_gate.shape
    dtype = DTYPE_OF[x.dtype]
    need = moe_forward_workspace(T, K, E, d, f, tm, dtype)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if out is None:
        out = torch.empty((T, d), dtype=torch.float32, device=x.device)
    if packed is not None:
        moe_forward(x, ids, w, packed["gate"], packed["up"], packed["down"], dtype, T, K, E, d, f,
                    tm, workspace, out, stream, timer, packed=True)
    else:
        moe_forward(x, ids, w, w_gate, w_up, w_down, dtype, T, K, E, d, f, tm, workspace, out,
                    stream, timer)
    return out, workspace


def forward_host(x, ids, w, hw_gate, hw_up, hw_down, tm: int = 16, packed: bool = False,
                 shapes=None, slots: int = 0, cache=None, workspace=None, out=None, stream=None):
    """One routed MoE layer whose expert weights are pinned host tensors (row-major
    [E, d, f] / [E, f, d], or packed arrays with shapes=(E, d, f)), through a device
    cache of `slots` experts (0: the fewest for T tokens); a new cache is made and
    cleared here, a given one must have been made for the same sizes and slots.
    Returns (out, cache, workspace)."""
    T, d = x.shape
    K = ids.shape[1]
    E, _, f = shapes if shapes is not None else hw_gate.shape
    dtype = DTYPE_OF[x.dtype]
    slots = slots or min(E, T * K)
    need = moe_forward_workspace(T, K, E, d, f, tm, dtype)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    if cache is None:
        cache = torch.empty(moe_host_cache_bytes(T, K, E, d, f, dtype, packed, slots),
                            dtype=torch.uint8, device=x.device)
        moe_host_cache_init(cache, E, d, f, dtype, packed, slots, stream)
    if out is None:
        out = torch.empty((T, d), dtype=torch.float32, device=x.device)
    moe_forward_host_weights(x, ids, w, hw_gate, hw_up, hw_down, packed, dtype, T, K, E, d, f, tm,
                             slots, cache, workspace, out, stream)
    return out, cache, workspace


# ---------------------------------------------- dense operators (C entry points) --

def moe_linear_shape(M: int, N: int, K: int, dtype: int):
    """(tile, splits along K) of a product of M x N outputs over K."""
    a, b = ctypes.c_int(), ctypes.c_int()
    _check("moe_linear_shape",
           lib().moe_linear_shape(M, N, K, dtype, ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


@functools.lru_cache(maxsize=1024)
def moe_linear_workspace(T: int, d: int, n: int, ldx: int, ldw: int, dtype: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_linear_workspace",
           lib().moe_linear_workspace(T, d, n, ldx, ldw, dtype, ctypes.byref(v)))
    return v.value


@functools.lru_cache(maxsize=1024)
def moe_linear_backward_workspace(T, d, n, ldx, ldw, lddz, dtype: int, grads: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_linear_backward_workspace",
           lib().moe_linear_backward_workspace(T, d, n, ldx, ldw, lddz, dtype, grads,
                                               ctypes.byref(v)))
    return v.value


@functools.lru_cache(maxsize=1024)
def moe_balance_workspace(T: int, E: int, K: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_balance_workspace", lib().moe_balance_workspace(T, E, K, ctypes.byref(v)))
    return v.value


# The short-named helpers take row-major GPU matrices (rows may be strided, the
# first element lies at a 16-byte boundary), check shapes and types, allocate what
# is not given, on the stream that the kernels run on, and launch on the tensors'
# device. `workspace` may be kept from call to call; it is replaced when it is too
# small.

class _On:
    """Device and stream of one call: the tensors' device made current, `handle` the
    stream to launch on. empty() allocates on that stream."""
    __slots__ = ("index", "handle", "stream", "before")

    def __init__(self, t, name, stream):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name}: expected a GPU tensor")
        self.index, self.stream, self.before = t.get_device(), stream, -1
        # (a handle does not say where it belongs)
        there = getattr(stream, "device_index", self.index)
        if there != self.index:
            raise ValueError(f"stream: on GPU {there}, expected GPU {self.index}")

    def __enter__(self):
        if self.index != torch._C._cuda_getDevice():
            self.before = torch._C._cuda_getDevice()
            torch.cuda.set_device(self.index)
        self.handle = (torch._C._cuda_getCurrentRawStream(self.index) if self.stream is None
                       else _stream(self.stream))
        return self

    def __exit__(self, *exc):
        if self.before >= 0:
            torch.cuda.set_device(self.before)

    def empty(self, shape, dtype):
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.index))
        # (ExternalStream(0) is not the default stream, but one of torch's own)
        s = (self.stream if hasattr(self.stream, "cuda_stream")
             else torch.cuda.ExternalStream(self.handle) if self.handle
             else torch.cuda.default_stream(self.index))
        with torch.cuda.stream(s):
            return torch.empty(shape, dtype=dtype, device=torch.device("cuda", self.index))

    def workspace(self, given, need):
        """(the tensor, its address, its bytes)"""
        if given is not None:
            p, have = _dev(given, "workspace"), given.numel() * given.element_size()
            if given.get_device() != self.index:
                raise ValueError(f"workspace: on {given.device}, expected GPU {self.index}")
            if have >= need:
                return given, p, have
        given = self.empty((need,), torch.uint8)
        return given, given.data_ptr(), need


def _matrix_shape(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a matrix, got {tuple(t.shape)}")
    return t.shape


def linear(x, w, bias=None, residual=None, act: str = "none", out_dtype=None, workspace=None,
           out=None, stream=None):
    """out = act(x w + bias) + residual for x [T, d], w [d, n] of one type, in out_dtype
    (x's type, or torch.float32); returns (out, workspace). residual may be out itself."""
    with _On(x, "x", stream) as at:
        dev, D = at.index, x.dtype
        T, d = _matrix_shape(x, "x")
        n = _matrix_shape(w, "w")[1]
        if out is None:
            out = at.empty((T, n), out_dtype or D)
        elif out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
        px, ldx = _mat(x, "x", dev, T, d, D)
        pw, ldw = _mat(w, "w", dev, d, n, D)
        pr, ldr = _mat(residual, "residual", dev, T, n, D, torch.float32)
        po, ldo = _mat(out, "out", dev, T, n, D, torch.float32)
        dtype = _dtype("x", D)
        workspace, ws, have = at.workspace(workspace,
                                           moe_linear_workspace(T, d, n, ldx, ldw, dtype))
        rc = lib().moe_linear(px, ldx, pw, ldw, _vec(bias, "bias", dev, n, D, 16), pr, ldr,
                              dtype if pr is None else DTYPE_OF[residual.dtype], dtype, _act(act),
                              T, d, n, ws, have, po, ldo, DTYPE_OF[out.dtype], at.handle)
    _check("moe_linear", rc)
    return out, workspace


def linear_backward(x, w, dz, grads=("dx", "dw", "db"), grad_dtype=None, workspace=None, dx=None,
                    dw=None, db=None, stream=None):
    """Gradients of z = x w + bias from dz [T, n]: dx [T, d] (dz's type), dw [d, n] and db
    [n] in grad_dtype (dz's type, or torch.float32). `grads` names what is computed; a
    given dx, dw or db is filled. x may be None without dw, w without dx (not both).
    Returns (dict of the gradients, workspace)."""
    if not grads or set(grads) - {"dx", "dw", "db"}:
        raise ValueError(f"grads: expected some of dx, dw, db, got {grads}")
    if ("dw" in grads and x is None) or ("dx" in grads and w is None) or (x is None and w is None):
        raise ValueError("dw needs x, dx needs w, and one of them gives d")
    with _On(dz, "dz", stream) as at:
        dev, D = at.index, dz.dtype
        T, n = _matrix_shape(dz, "dz")
        d = _matrix_shape(x, "x")[1] if x is not None else _matrix_shape(w, "w")[0]
        px, ldx = _mat(x, "x", dev, T, d, D, read="dw" in grads)
        pw, ldw = _mat(w, "w", dev, d, n, D, read="dx" in grads)
        pz, lddz = _mat(dz, "dz", dev, T, n, D)
        G = grad_dtype or (dw.dtype if dw is not None else db.dtype if db is not None else D)
        if G is not D and G is not torch.float32:
            raise TypeError(f"grad_dtype: expected {D} or torch.float32, got {G}")
        got, mask = {}, 0
        if "dx" in grads:
            got["dx"] = at.empty((T, d), D) if dx is None else dx
            mask = MOE_GRAD_X
        if "dw" in grads:
            got["dw"] = at.empty((d, n), G) if dw is None else dw
            mask |= MOE_GRAD_W
        if "db" in grads:
            got["db"] = at.empty((n,), G) if db is None else db
            mask |= MOE_GRAD_BIAS
        pdx, lddx = _mat(got.get("dx"), "dx", dev, T, d, D)
        pdw, lddw = _mat(got.get("dw"), "dw", dev, d, n, G)
        pdb = _vec(got.get("db"), "db", dev, n, G, 16)
        dtype = _dtype("dz", D)
        workspace, ws, have = at.workspace(
            workspace, moe_linear_backward_workspace(T, d, n, ldx, ldw, lddz, dtype, mask))
        rc = lib().moe_linear_backward(px, ldx, pw, ldw, pz, lddz, dtype, T, d, n, ws, have, pdx,
                                       lddx, pdw, lddw, pdb, DTYPE_OF[G], at.handle)
    _check("moe_linear_backward", rc)
    return got, workspace


def balance_loss(logits, ids, workspace=None, cnt=None, prob=None, loss=None, stream=None):
    """Router losses of logits [T, E] fp32 and ids [T, K] int32. Returns (dict, workspace):
    loss [2] (balance, z), cnt [E + 2] int32 (entries per expert, valid tokens, valid
    entries), prob [E] (mean probability over the valid tokens)."""
    with _On(logits, "logits", stream) as at:
        dev = at.index
        T, E = _matrix_shape(logits, "logits")
        K = _matrix_shape(ids, "ids")[1]
        cnt = at.empty((E + 2,), torch.int32) if cnt is None else cnt
        prob = at.empty((E,), torch.float32) if prob is None else prob
        loss = at.empty((2,), torch.float32) if loss is None else loss
        workspace, ws, have = at.workspace(workspace, moe_balance_workspace(T, E, K))
        rc = lib().moe_balance_loss(
            _vec(logits, "logits", dev, T * E, torch.float32),
            _vec(ids, "ids", dev, T * K, torch.int32), T, E, K, ws, have,
            _vec(cnt, "cnt", dev, E + 2, torch.int32), _vec(prob, "prob", dev, E, torch.float32),
            _vec(loss, "loss", dev, 2, torch.float32), at.handle)
    _check("moe_balance_loss", rc)
    return {"loss": loss, "cnt": cnt, "prob": prob}, workspace


def route_backward(logits, ids, w, dw, cnt, dloss, out_dtype=None, out=None, stream=None):
    """Gradient of the router logits [T, E] from dw [T, K], the gradient of route()'s weights
    w (None: no such term), and dloss [2], the gradient by balance_loss()'s two losses
    (None: no such term); cnt as balance_loss() gave it. out_dtype: fp32, or the type of
    the router's product."""
    with _On(logits, "logits", stream) as at:
        dev = at.index
        T, E = _matrix_shape(logits, "logits")
        K = _matrix_shape(ids, "ids")[1]
        if out is None:
            out = at.empty((T, E), out_dtype or torch.float32)
        elif out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
        rc = lib().moe_route_backward(
            _vec(logits, "logits", dev, T * E, torch.float32),
            _vec(ids, "ids", dev, T * K, torch.int32), _vec(w, "w", dev, T * K, torch.float32),
            _vec(dw, "dw", dev, T * K, torch.float32), _vec(cnt, "cnt", dev, E + 2, torch.int32),
            _vec(dloss, "dloss", dev, 2, torch.float32), T, E, K,
            _vec(out, "out", dev, T * E, out.dtype), _dtype("out", out.dtype), at.handle)
    _check("moe_route_backward", rc)
    return out


def act_forward(g, u=None, act: str = "silu", ckpt=None, h=None, stream=None):
    """h = act(g) * u (or act(g)) for matrices [T, f]; h may be g or u itself. ckpt: None (nothing kept), True (a
    new 8-bit checkpoint) or an earlier call's, which is overwritten. Returns (h, ckpt);
    a checkpoint is a dict of e4m3 codes g8, u8 [T, f] and scale bytes gs, us [T,
    ceil(f / 32)], code * 2^(scale - 127) the values they stand for."""
    with _On(g, "g", stream) as at:
        dev, D = at.index, g.dtype
        T, f = _matrix_shape(g, "g")
        if ckpt is True:
            ckpt = {}
            for k in ("g", "u")[:1 if u is None else 2]:
                ckpt[k + "8"] = at.empty((T, f), torch.float8_e4m3fn)
                ckpt[k + "s"] = at.empty((T, -(-f // ACT8_BLOCK)), torch.uint8)
        h = at.empty((T, f), D) if h is None else h
        pg, ldg = _mat(g, "g", dev, T, f, D)
        pu, ldu = _mat(u, "u", dev, T, f, D)
        ph, ldh = _mat(h, "h", dev, T, f, D)
        g8, gs, u8, us = _ckpt(dev, ckpt, T, f, u is not None)
        rc = lib().moe_act_forward(pg, ldg, pu, ldu, _dtype("g", D), _act(act), T, f, ph, ldh, g8,
                                   gs, u8, us, at.handle)
    _check("moe_act_forward", rc)
    return h, ckpt


def act_backward(ckpt, dh, act: str = "silu", dg=None, du=None, h=None, need_h: bool = True,
                 stream=None):
    """From act_forward()'s checkpoint and dh [T, f]: a dict of dg, du (if there was a u) and
    h, the forward's output as the checkpoint gives it (not with need_h=False). One of
    them may be dh itself."""
    with _On(dh, "dh", stream) as at:
        dev, D = at.index, dh.dtype
        T, f = _matrix_shape(dh, "dh")
        gated = "u8" in ckpt
        if du is not None and not gated:
            raise ValueError("du: the checkpoint has no u")
        got = {"dg": at.empty((T, f), D) if dg is None else dg}
        if gated:
            got["du"] = at.empty((T, f), D) if du is None else du
        if need_h or h is not None:
            got["h"] = at.empty((T, f), D) if h is None else h
        pz, lddh = _mat(dh, "dh", dev, T, f, D)
        pdg, lddg = _mat(got["dg"], "dg", dev, T, f, D)
        pdu, lddu = _mat(got.get("du"), "du", dev, T, f, D)
        ph, ldh = _mat(got.get("h"), "h", dev, T, f, D)
        g8, gs, u8, us = _ckpt(dev, ckpt, T, f, gated)
        rc = lib().moe_act_backward(g8, gs, u8, us, pz, lddh, _dtype("dh", D), _act(act), T, f, pdg,
                                    lddg, pdu, lddu, ph, ldh, at.handle)
    _check("moe_act_backward", rc)
    return got


def _ckpt(dev, ckpt, T, f, gated):
    """device addresses g8, gs, u8, us of a checkpoint (None where there is none)"""
    if ckpt is None:
        return None, None, None, None
    if ("u8" in ckpt) != gated:
        raise ValueError("ckpt: made for another kind of activation (with or without u)")
    nb = T * -(-f // ACT8_BLOCK)
    g = (_vec(ckpt["g8"], "g8", dev, T * f, torch.float8_e4m3fn, 16),
         _vec(ckpt["gs"], "gs", dev, nb, torch.uint8))
    return g + ((_vec(ckpt["u8"], "u8", dev, T * f, torch.float8_e4m3fn, 16),
                 _vec(ckpt["us"], "us", dev, nb, torch.uint8)) if gated else (None, None))


# ------------------------------------- operators around the routed layer's block --

@functools.lru_cache(maxsize=1024)
def moe_mx4_weight_bytes(E: int, d: int, f: int, kind: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_mx4_weight_bytes", lib().moe_mx4_weight_bytes(E, d, f, kind, ctypes.byref(v)))
    return v.value


@functools.lru_cache(maxsize=1024)
def moe_norm_backward_workspace(T: int, d: int) -> int:
    v = ctypes.c_size_t()
    _check("moe_norm_backward_workspace", lib().moe_norm_backward_workspace(T, d, ctypes.byref(v)))
    return v.value


@functools.lru_cache(maxsize=1024)
def _forward_workspace(T, K, E, d, f, tm, dtype):
    return moe_forward_workspace(T, K, E, d, f, tm, dtype)


def route_scored(logits, K: int, bias=None, score: str = "softmax", groups: int = 1, keep=None,
                 group_top: int = 1, renorm: bool = True, scale: float = 1.0, ids=None, w=None,
                 stream=None):
    """Routing of logits [T, E] fp32 by softmax or sigmoid scores: the K experts with the
    largest score + bias [E] of the `keep` (None: all) of `groups` groups whose group_top
    best experts add up to most; weights are the scores (without the bias) times scale,
    renormalised to sum to it or not. Returns (ids [T, K] int32, w [T, K] fp32)."""
    with _On(logits, "logits", stream) as at:
        dev = at.index
        T, E = _matrix_shape(logits, "logits")
        ids = at.empty((T, K), torch.int32) if ids is None else ids
        w = at.empty((T, K), torch.float32) if w is None else w
        rc = lib().moe_route_scored(
            _vec(logits, "logits", dev, T * E, torch.float32),
            _vec(bias, "bias", dev, E, torch.float32), _named("score", score, SCORES), T, E, K,
            groups, groups if keep is None else keep, group_top, int(bool(renorm)), scale,
            _vec(ids, "ids", dev, T * K, torch.int32), _vec(w, "w", dev, T * K, torch.float32),
            at.handle)
    _check("moe_route_scored", rc)
    return ids, w


def route_scored_backward(logits, ids, dw, score: str = "softmax", renorm: bool = True,
                          scale: float = 1.0, add=None, out_dtype=None, out=None, stream=None):
    """Gradient of the logits [T, E] from dw [T, K], that of route_scored()'s weights, for
    its ids. add [T, E], of the result's type, is added to it and may be out itself.
    out_dtype: fp32, or the type of the router's product."""
    with _On(logits, "logits", stream) as at:
        dev = at.index
        T, E = _matrix_shape(logits, "logits")
        K = _matrix_shape(ids, "ids")[1]
        if out is None:
            out = at.empty((T, E), out_dtype or (add.dtype if add is not None else torch.float32))
        elif out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
        rc = lib().moe_route_scored_backward(
            _vec(logits, "logits", dev, T * E, torch.float32),
            _vec(ids, "ids", dev, T * K, torch.int32), _vec(dw, "dw", dev, T * K, torch.float32),
            _vec(add, "add", dev, T * E, out.dtype), _named("score", score, SCORES), T, E, K,
            int(bool(renorm)), scale, _vec(out, "out", dev, T * E, out.dtype),
            _dtype("out", out.dtype), at.handle)
    _check("moe_route_scored_backward", rc)
    return out


def _mx4_shape(name, w, kind):
    if w.dim() != 3:
        raise ValueError(f"{name}: expected [E, in, out] matrices, got {tuple(w.shape)}")
    E, a, b = w.shape
    return (E, a, b) if kind == MOE_W_GATE_UP else (E, b, a)


def mx4_quantize(w, kind: str, packed=None, stream=None):
    """Expert matrices in microscaled 4-bit floating point: w [E, d, f] (kind "gate": gate
    or up matrices) or [E, f, d] ("down"). Returns the packed bytes, in the layout that
    forward_mx4 streams; a given `packed` is filled."""
    with _On(w, "w", stream) as at:
        k = _named("kind", kind, MX4_KINDS)
        E, d, f = _mx4_shape("w", w, k)
        need = moe_mx4_weight_bytes(E, d, f, k)
        packed = at.empty((need,), torch.uint8) if packed is None else packed
        rc = lib().moe_mx4_quantize(
            _vec(w, "w", at.index, E * d * f, w.dtype, 16), _dtype("w", w.dtype), E, d, f, k,
            _vec(packed, "packed", at.index, need, torch.uint8, 16), need, at.handle)
    _check("moe_mx4_quantize", rc)
    return packed


def mx4_dequantize(packed, E: int, d: int, f: int, kind: str, dtype=None, out=None, stream=None):
    """The values of packed matrices, row-major in `dtype` (out's, or bfloat16): [E, d, f]
    (kind "gate") or [E, f, d] ("down")."""
    with _On(packed, "packed", stream) as at:
        k = _named("kind", kind, MX4_KINDS)
        need = moe_mx4_weight_bytes(E, d, f, k)
        shape = (E, d, f) if k == MOE_W_GATE_UP else (E, f, d)
        if out is None:
            out = at.empty(shape, dtype or torch.bfloat16)
        elif dtype is not None and out.dtype is not dtype:
            raise TypeError(f"out: expected {dtype}, got {out.dtype}")
        elif tuple(out.shape) != shape:
            raise ValueError(f"out: expected {shape}, got {tuple(out.shape)}")
        rc = lib().moe_mx4_dequantize(
            _vec(packed, "packed", at.index, need, torch.uint8, 16), need, E, d, f, k,
            _vec(out, "out", at.index, E * d * f, out.dtype, 16), _dtype("out", out.dtype),
            at.handle)
    _check("moe_mx4_dequantize", rc)
    return out


def pack_mx4(w_gate, w_up, w_down, stream=None) -> dict:
    """The three matrix sets of a layer in 4 bits, keyed gate / up / down."""
    return {"gate": mx4_quantize(w_gate, "gate", stream=stream),
            "up": mx4_quantize(w_up, "gate", stream=stream),
            "down": mx4_quantize(w_down, "down", stream=stream)}


def forward_mx4(x, ids, w, packed, E: int, f: int, tm: int = 16, out_dtype=None, workspace=None,
                out=None, stream=None):
    """One routed MoE layer with expert weights in 4 bits (pack_mx4()'s dict, for E experts
    of intermediate size f): x [T, d] float16 or bfloat16, ids and w [T, K]; out [T, d] in
    x's type or torch.float32. Returns (out, workspace)."""
    with _On(x, "x", stream) as at:
        dev, D = at.index, x.dtype
        T, d = _matrix_shape(x, "x")
        K = _matrix_shape(ids, "ids")[1]
        if out is None:
            out = at.empty((T, d), out_dtype or D)
        elif out_dtype is not None and out.dtype is not out_dtype:
            raise TypeError(f"out: expected {out_dtype}, got {out.dtype}")
        dtype = _dtype("x", D)
        bgu = moe_mx4_weight_bytes(E, d, f, MOE_W_GATE_UP)
        bdn = moe_mx4_weight_bytes(E, d, f, MOE_W_DOWN)
        workspace, ws, have = at.workspace(workspace, _forward_workspace(T, K, E, d, f, tm, dtype))
        rc = lib().moe_forward_mx4(
            _vec(x, "x", dev, T * d, D, 16), _vec(ids, "ids", dev, T * K, torch.int32),
            _vec(w, "w", dev, T * K, torch.float32),
            _vec(packed["gate"], "packed['gate']", dev, bgu, torch.uint8, 16),
            _vec(packed["up"], "packed['up']", dev, bgu, torch.uint8, 16),
            _vec(packed["down"], "packed['down']", dev, bdn, torch.uint8, 16), dtype, T, K, E, d,
            f, tm, ws, have, _vec(out, "out", dev, T * d, out.dtype, 16),
            _dtype("out", out.dtype), at.handle)
    _check("moe_forward_mx4", rc)
    return out, workspace


def _gate(gate, kind, name, dev, T, d, dtype, channel=None):
    """(address, row stride) of a gate or its gradient; channel: a per-channel one's type"""
    if gate is None:
        return None, 0
    if kind == GATES["full"]:
        return _mat(gate, name, dev, T, d, dtype)
    per_channel = kind == GATES["channel"]
    return _vec(gate, name, dev, d if per_channel else T, channel if per_channel and channel
                else dtype, 16), 0


def _norm_dtype(r, y, *weights):
    """the type that the weights and the gate share; without any, that of y, or of the
    residual stream r next to an fp32 y"""
    for t in weights:
        if t is not None:
            return t.dtype
    if y is None:
        raise ValueError("y or w_pre is needed")
    return y.dtype if y.dtype is not torch.float32 else r.dtype


def norm(r, y=None, w_post=None, gate=None, gate_kind: str = "none", w_pre=None,
         alpha: float = 1.0, eps: float = 1e-6, z=None, h=None, stats=None, stream=None):
    """The norms after and before a block (root mean square over a row), its gate, scale and
    residual in one pass: n = y / rms(y) * w_post (or y), z = r + alpha * gate * n (or r
    without y), h = z / rms(z) * w_pre. r [T, d], the residual stream, and y [T, d], the
    block's output, each in the weights' type or torch.float32; gate [T] ("token"), [d]
    ("channel") or [T, d] ("full"). z may be r itself, h may be y. stats: a [T, 2] fp32
    tensor, or True for a new one, that receives 1 / rms(y) and 1 / rms(z) for
    norm_backward. Returns a dict of z (with y), h (with w_pre) and stats (if asked for)."""
    with _On(r, "r", stream) as at:
        dev, R = at.index, r.dtype
        T, d = _matrix_shape(r, "r")
        D = _norm_dtype(r, y, w_pre, w_post, gate)
        kind = _named("gate_kind", gate_kind, GATES)
        got = {}
        if y is not None:
            got["z"] = at.empty((T, d), R) if z is None else z
        elif z is not None:
            raise ValueError("z: there is no y, z is r")
        if w_pre is not None:
            got["h"] = at.empty((T, d), D) if h is None else h
        elif h is not None:
            raise ValueError("h: there is no w_pre")
        if stats is not None:
            got["stats"] = at.empty((T, 2), torch.float32) if stats is True else stats
        F = torch.float32
        pr, ldr = _mat(r, "r", dev, T, d, D, F)
        py, ldy = _mat(y, "y", dev, T, d, D, F)
        pg, ldg = _gate(gate, kind, "gate", dev, T, d, D)
        pz, ldz = _mat(got.get("z"), "z", dev, T, d, R)
        ph, ldh = _mat(got.get("h"), "h", dev, T, d, D)
        dtype = _dtype("the weights", D)
        rc = lib().moe_norm(
            pr, ldr, _dtype("r", R), py, ldy, dtype if y is None else _dtype("y", y.dtype),
            _vec(w_post, "w_post", dev, d, D, 16), pg, ldg, kind,
            _vec(w_pre, "w_pre", dev, d, D, 16), dtype, T, d, alpha, eps, pz, ldz, ph, ldh,
            _vec(got.get("stats"), "stats", dev, 2 * T, F), at.handle)
    _check("moe_norm", rc)
    return got


def norm_backward(z, stats, dz=None, dh=None, y=None, w_post=None, gate=None,
                  gate_kind: str = "none", w_pre=None, alpha: float = 1.0, grad_dtype=None,
                  grads=None, workspace=None, dr=None, dy=None, dgate=None, dw_post=None,
                  dw_pre=None, stream=None):
    """Gradients of norm() from dz (of z, from behind; or None) and dh (of h, given with
    w_pre), with its z (r where there was no y), stats and other arguments. Returns (dict,
    workspace): dr, and those of dy, dgate, dw_post, dw_pre that apply (or that `grads`
    names or a tensor is given for); dr may be dz itself. dw_post, dw_pre and a per-channel dgate are in
    grad_dtype (the weights' type, or torch.float32)."""
    with _On(z, "z", stream) as at:
        dev, R, F = at.index, z.dtype, torch.float32
        T, d = _matrix_shape(z, "z")
        D = _norm_dtype(z, y, w_pre, w_post, gate)
        kind = _named("gate_kind", gate_kind, GATES)
        every = grads is None

        def asked(name, given, able):
            if given is None and not (able if every else name in grads):
                return False
            if not able:
                raise ValueError(f"{name}: there is no such gradient in this call")
            return True

        if not every and not NORM_GRADS.issuperset(grads):
            raise ValueError(f"grads: expected some of {', '.join(sorted(NORM_GRADS))}")
        per_channel = gate is not None and gate_kind == "channel"
        G = grad_dtype
        if G is None:
            G = next((t.dtype for t in (dw_post, dw_pre, dgate if per_channel else None)
                      if t is not None), D)
        if G is not D and G is not F:
            raise TypeError(f"grad_dtype: expected {D} or torch.float32, got {G}")
        Y = D if y is None else y.dtype
        got = {"dr": at.empty((T, d), R) if dr is None else dr}
        if asked("dy", dy, y is not None):
            got["dy"] = dy = at.empty((T, d), Y) if dy is None else dy
        if asked("dgate", dgate, gate is not None):
            if dgate is None:
                dgate = at.empty(((T,), (d,), (T, d))[kind - 1], G if per_channel else D)
            got["dgate"] = dgate
        if asked("dw_post", dw_post, w_post is not None):
            got["dw_post"] = dw_post = at.empty((d,), G) if dw_post is None else dw_post
        if asked("dw_pre", dw_pre, w_pre is not None):
            got["dw_pre"] = dw_pre = at.empty((d,), G) if dw_pre is None else dw_pre
        pdz, lddz = _mat(dz, "dz", dev, T, d, R)
        pdh, lddh = _mat(dh, "dh", dev, T, d, D)
        pz, ldz = _mat(z, "z", dev, T, d, D, F)
        py, ldy = _mat(y, "y", dev, T, d, D, F)
        pg, ldg = _gate(gate, kind, "gate", dev, T, d, D)
        pdr, lddr = _mat(got["dr"], "dr", dev, T, d, R)
        pdy, lddy = _mat(dy, "dy", dev, T, d, Y)
        pdg, lddg = _gate(dgate, kind, "dgate", dev, T, d, D, G)
        workspace, ws, have = at.workspace(workspace, moe_norm_backward_workspace(T, d))
        dtype = _dtype("the weights", D)
        rc = lib().moe_norm_backward(
            pdz, lddz, pdh, lddh, pz, ldz, _dtype("z", R), py, ldy,
            _dtype("y", Y), _vec(w_post, "w_post", dev, d, D, 16), pg, ldg, kind,
            _vec(w_pre, "w_pre", dev, d, D, 16), _vec(stats, "stats", dev, 2 * T, F), dtype, T, d,
            alpha, ws, have, pdr, lddr, pdy, lddy, pdg, lddg,
            _vec(dw_post, "dw_post", dev, d, G, 16), _vec(dw_pre, "dw_pre", dev, d, G, 16),
            DTYPE_OF[G], at.handle)
    _check("moe_norm_backward", rc)
    return got, workspace
