"""Thin ctypes binding of libmoe (include/moe.h).

Argument marshalling only: every step of the layer runs in libmoe's CUDA
kernels.  Tensors are torch CUDA tensors; their data pointers and the current
torch stream are handed to the C entry points.  Missing outputs and
workspaces are allocated with torch (device memory is torch's job here), as
under torch.cuda.stream(stream) where a call is given a stream.  If libmoe.so
is missing this module raises on import: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with "
        "`python -c 'import __graft_entry__ as g; g.build()'` "
        "or `python routed_expert_ffn_02_gb300/_build.py`")

_lib = ctypes.CDLL(LIB_PATH)

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
                3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT",
                6: "MOE_ERR_BAD_INDEX"}

# Every function declared in include/moe.h.
EXPORTED = ("moe_route", "moe_permute_workspace_size", "moe_permute", "moe_permute_noalloc",
            "moe_expert_ffn_workspace_size", "moe_expert_ffn", "moe_combine",
            "moe_workspace_size", "moe_forward", "moe_forward_profiled",
            "moe_forward_launches", "moe_layer_weight_bytes", "moe_stager_create",
            "moe_stager_destroy", "moe_forward_offload", "moe_workspace_init",
            "moe_workspace_status", "moe_last_error", "moe_version",
            "moe_pipe_workspace_size", "moe_pipe_create", "moe_pipe_destroy",
            "moe_forward_host", "moe_cache_bytes", "moe_cache_create", "moe_cache_destroy",
            "moe_cache_stats", "moe_forward_cached", "moe_debug_set_wait_limit",
            "moe_quantize_rows", "moe_quantize_weights", "moe_grouped_gemm_fp8_workspace_size",
            "moe_grouped_gemm_fp8", "moe_expert_ffn_fp8_workspace_size", "moe_expert_ffn_fp8",
            "moe_fp8_workspace_size", "moe_forward_fp8", "moe_balance_workspace_size",
            "moe_balance", "moe_balance_backward",
            "moe_expert_ffn_train_workspace_size", "moe_expert_ffn_train",
            "moe_expert_ffn_backward_workspace_size", "moe_expert_ffn_backward",
            "moe_dequantize_rows", "moe_grouped_gemm_workspace_size", "moe_grouped_gemm")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("H", ctypes.c_int32), ("I", ctypes.c_int32),
                ("fat_threshold", ctypes.c_int32),
                ("thin_mma_min", ctypes.c_int32)]


class MoeFp8Experts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("gate", "gate_scales", "up", "up_scales",
                                               "down", "down_scales")]


class MoeSaved(ctypes.Structure):
    _fields_ = [("fp8", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
        "x", "x_scales", "gate", "gate_scales", "up", "up_scales")]


@dataclass(frozen=True)
class Shape:
    T: int
    E: int
    k: int
    H: int
    I: int
    fat_threshold: int = 32
    thin_mma_min: int = 0     # 0: library default; > fat_threshold - 1: CUDA cores only

    def c(self) -> MoeShape:
        c = self.__dict__.get("_c")
        if c is None:
            c = MoeShape(self.T, self.E, self.k, self.H, self.I, self.fat_threshold,
                         self.thin_mma_min)
            object.__setattr__(self, "_c", c)
        return c

    @property
    def P(self) -> int:
        return self.T * self.k


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = _lib.moe_last_error().decode()
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_P = ctypes.c_void_p
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t
_SP = ctypes.POINTER(MoeShape)

_WP = ctypes.POINTER(MoeFp8Experts)
_VP = ctypes.POINTER(MoeSaved)
_f32 = ctypes.c_float

_sig = {
    "moe_quantize_rows": ([_P, _i32, _i32, _P, _P, _P], _i32),
    "moe_quantize_weights": ([_P, _i32, _i32, _i32, _P, _P, _P], _i32),
    "moe_grouped_gemm_fp8_workspace_size": ([_i32, _i32], _sz),
    "moe_grouped_gemm_fp8": ([_P, _P, _i32, _P, _i32, _i32, _i32, _P, _P, _P, _P, _sz, _P], _i32),
    "moe_expert_ffn_fp8_workspace_size": ([_SP], _sz),
    "moe_expert_ffn_fp8": ([_SP, _P, _P, _P, _WP, _P, _P, _sz, _P], _i32),
    "moe_fp8_workspace_size": ([_SP], _sz),
    "moe_forward_fp8": ([_SP, _P, _P, _WP, _P, _P, _P, _P, _sz, _P], _i32),
    "moe_balance_workspace_size": ([_i32, _i32, _i32], _sz),
    "moe_balance": ([_P, _P, _i32, _i32, _i32, _P, _i32, _f32, _P, _P, _P, _P, _sz, _P], _i32),
    "moe_balance_backward": ([_P, _P, _P, _P, _i32, _i32, _i32, _i32, _f32, _P, _P, _P, _P, _P,
                              _P], _i32),
    "moe_expert_ffn_train_workspace_size": ([_SP], _sz),
    "moe_expert_ffn_train": ([_SP, _P, _P, _P, _P, _P, _P, _P, _VP, _P, _sz, _P], _i32),
    "moe_expert_ffn_backward_workspace_size": ([_SP], _sz),
    "moe_expert_ffn_backward": ([_SP, _P, _P, _VP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                 _sz, _P], _i32),
    "moe_dequantize_rows": ([_P, _P, _i32, _i32, _P, _P], _i32),
    "moe_grouped_gemm_workspace_size": ([_i32, _i32, _i32, _i32], _sz),
    "moe_grouped_gemm": ([_P, _i32, _P, _i32, _i32, _i32, _P, _P, _i32, _P, _P, _i32, _P, _sz, _P],
                         _i32),
    "moe_route": ([_P, _i32, _i32, _i32, _P, _P, _P], _i32),
    "moe_permute_workspace_size": ([_i32, _i32, _i32], _sz),
    "moe_permute": ([_P, _i32, _i32, _i32, _P, _P, _P, _P, _P, _sz, _P], _i32),
    "moe_permute_noalloc": ([_P, _i32, _i32, _i32, _P, _P, _P, _P, _P, _P], _i32),
    "moe_expert_ffn_workspace_size": ([_SP], _sz),
    "moe_expert_ffn": ([_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _sz, _P], _i32),
    "moe_combine": ([_P, _P, _P, _i32, _i32, _i32, _P, _P], _i32),
    "moe_workspace_size": ([_SP], _sz),
    "moe_forward": ([_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _sz, _P], _i32),
    "moe_forward_profiled": ([_SP, _P, _P, _P, _P, _P, _P, _P, _P, _P, _sz, _P,
                              ctypes.POINTER(ctypes.c_void_p), _i32], _i32),
    "moe_forward_launches": ([_SP], _i32),
    "moe_layer_weight_bytes": ([_SP], _sz),
    "moe_stager_create": ([_P, _i32, _sz, ctypes.POINTER(_P)], _i32),
    "moe_stager_destroy": ([_P], _i32),
    "moe_forward_offload": ([_P, _SP, _i32, ctypes.POINTER(_P), _P, ctypes.POINTER(_P),
                             ctypes.POINTER(_P), _P, _sz, _P, _P], _i32),
    "moe_workspace_init": ([_P, _sz, _P], _i32),
    "moe_pipe_workspace_size": ([_SP], _sz),
    "moe_cache_bytes": ([_SP, _i32, _i32], _sz),
    "moe_cache_create": ([_SP, _i32, _i32, _P, _sz, ctypes.POINTER(_P)], _i32),
    "moe_cache_destroy": ([_P], _i32),
    "moe_cache_stats": ([_P, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)], _i32),
    "moe_forward_cached": ([_P, _SP, _i32, ctypes.POINTER(_i32), ctypes.POINTER(_P), _P,
                            ctypes.POINTER(_P), ctypes.POINTER(_P), _P, _sz, _P, _P], _i32),
    "moe_pipe_create": ([ctypes.POINTER(_P)], _i32),
    "moe_pipe_destroy": ([_P], _i32),
    "moe_forward_host": ([_P, _SP, _P, _P, _P, _P, _P, _P, _P, _sz, _P, _P, _P], _i32),
    "moe_workspace_status": ([_P, _P, _i32], _i32),
    "moe_debug_set_wait_limit": ([ctypes.c_int64], _i32),
    "moe_last_error": ([], ctypes.c_char_p),
    "moe_version": ([], ctypes.c_char_p),
}
for _name, (_args, _ret) in _sig.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _ret


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "expected a contiguous CUDA tensor"
    return ctypes.c_void_p(t.data_ptr())


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """A tensor for a call on `stream` (None: the current one), out of that
    stream's memory: torch hands memory out again in its stream's order, so
    other streams' work is neither still using it nor given it before the call
    has run."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _host_ptr(t: torch.Tensor):
    assert not t.is_cuda and t.is_contiguous(), "expected a contiguous host tensor"
    return ctypes.c_void_p(t.data_ptr())


# The 8-bit operators and the balance loss run in microseconds, so their
# arguments take a short path: one condition and a plain integer per tensor.
_raw_stream = torch._C._cuda_getCurrentRawStream
_BF16, _F32, _I32, _U8, _E4M3 = (torch.bfloat16, torch.float32, torch.int32, torch.uint8,
                                 torch.float8_e4m3fn)


def _in(t: torch.Tensor, dtype, shape) -> int:
    """Address of a contiguous CUDA tensor of this type and shape."""
    if t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    raise AssertionError(f"expected a contiguous CUDA tensor {dtype} {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _opt(t: torch.Tensor | None, dtype, shape):
    return None if t is None else _in(t, dtype, shape)


def _out(t: torch.Tensor | None, shape, dtype, like: torch.Tensor, stream):
    """The caller's output tensor, checked, or a new one, and its address."""
    if t is None:
        t = (torch.empty(shape, dtype=dtype, device=like.device) if stream is None
             else _empty(shape, dtype, like.device, stream))
        return t, t.data_ptr()
    return t, _in(t, dtype, shape)


def _on(stream, t: torch.Tensor) -> int:
    """The stream to launch on: the caller's, or the current one of t's device."""
    return stream.cuda_stream if stream is not None else _raw_stream(t.get_device())


def _sequences(seq_offsets) -> int:
    if seq_offsets is None:
        return 1
    assert seq_offsets.dim() == 1 and seq_offsets.shape[0] >= 2, "seq_offsets is [S + 1], S >= 1"
    return seq_offsets.shape[0] - 1


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != MOE_OK:
        raise MoeError(status, where)


def version() -> str:
    return _lib.moe_version().decode()


def debug_set_wait_limit(cycles: int) -> None:
    """Test hook (moe_debug_set_wait_limit): main-loop waits of this thread's
    later expert-kernel launches give up after `cycles` SM cycles (0: the
    default bound).  Only for tests of the timeout path."""
    _check(_lib.moe_debug_set_wait_limit(int(cycles)), "moe_debug_set_wait_limit")


class Workspace:
    """Device scratch for libmoe calls on one stream (None: the current one): a
    256-byte-aligned torch buffer whose status word is cleared once at
    creation."""

    def __init__(self, nbytes: int, device=None, stream=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        assert torch.device(device).type == "cuda", f"workspace on {device}: expected a CUDA device"
        self._buf = _empty(nbytes + 256, torch.uint8, device, stream)
        off = (-self._buf.data_ptr()) % 256
        self.tensor = self._buf[off:off + nbytes]
        self.nbytes = nbytes
        self.addr = self.tensor.data_ptr()
        _check(_lib.moe_workspace_init(self.ptr, nbytes, _stream(stream)), "moe_workspace_init")

    @property
    def ptr(self):
        return ctypes.c_void_p(self.addr)

    def status(self, clear: bool = True, stream=None) -> int:
        """Synchronises the stream and returns the device status code."""
        return _lib.moe_workspace_status(self.ptr, _stream(stream), int(clear))


def workspace_size(shape: Shape) -> int:
    n = _lib.moe_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(1, "moe_workspace_size")
    return n


def permute_workspace_size(T: int, E: int, k: int) -> int:
    n = _lib.moe_permute_workspace_size(T, E, k)
    if n == 0:
        raise MoeError(1, "moe_permute_workspace_size")
    return n


def expert_ffn_workspace_size(shape: Shape) -> int:
    n = _lib.moe_expert_ffn_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(1, "moe_expert_ffn_workspace_size")
    return n


def moe_route(logits: torch.Tensor, k: int, topk_idx=None, gates=None, stream=None):
    T, E = logits.shape
    dev = logits.device
    topk_idx = topk_idx if topk_idx is not None else _empty((T, k), torch.int32, dev, stream)
    gates = gates if gates is not None else _empty((T, k), torch.float32, dev, stream)
    _check(_lib.moe_route(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(gates), _stream(stream)),
           "moe_route")
    return topk_idx, gates


def moe_permute(topk_idx: torch.Tensor, E: int, ws: Workspace | None = None, out=None,
                stream=None):
    """Returns (counts [E], offsets [E+1], perm [T*k], inv_perm [T*k])."""
    T, k = topk_idx.shape
    dev = topk_idx.device
    P = T * k
    if out is None:
        out = (_empty(E, torch.int32, dev, stream), _empty(E + 1, torch.int32, dev, stream),
               _empty(max(P, 1), torch.int32, dev, stream)[:P],
               _empty(max(P, 1), torch.int32, dev, stream)[:P])
    counts, offsets, perm, inv_perm = out
    ws = ws or Workspace(permute_workspace_size(T, E, k), dev, stream)
    _check(_lib.moe_permute(_ptr(topk_idx), T, E, k, _ptr(counts), _ptr(offsets), _ptr(perm),
                            _ptr(inv_perm), ws.ptr, ws.nbytes, _stream(stream)), "moe_permute")
    return counts, offsets, perm, inv_perm


def moe_permute_noalloc(topk_idx: torch.Tensor, E: int, out, device_status=None, stream=None):
    """moe_permute with the library's fixed scratch (no workspace, no device
    allocation inside the call).  `out` = (counts, offsets, perm, inv_perm)
    must be supplied by the caller; device_status (int32 [1]) is optional."""
    T, k = topk_idx.shape
    counts, offsets, perm, inv_perm = out
    _check(_lib.moe_permute_noalloc(_ptr(topk_idx), T, E, k, _ptr(counts), _ptr(offsets),
                                    _ptr(perm), _ptr(inv_perm), _ptr(device_status),
                                    _stream(stream)), "moe_permute_noalloc")
    return out


def moe_expert_ffn(shape: Shape, x, perm, offsets, counts, W_gate, W_up, W_down,
                   y_sorted=None, ws: Workspace | None = None, stream=None):
    dev = x.device
    y_sorted = y_sorted if y_sorted is not None else _empty(
        (shape.P, shape.H), torch.bfloat16, dev, stream)
    ws = ws or Workspace(expert_ffn_workspace_size(shape), dev, stream)
    _check(_lib.moe_expert_ffn(ctypes.byref(shape.c()), _ptr(x), _ptr(perm), _ptr(offsets),
                               _ptr(counts), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                               _ptr(y_sorted), ws.ptr, ws.nbytes, _stream(stream)),
           "moe_expert_ffn")
    return y_sorted


def moe_combine(y_sorted, inv_perm, gates, T: int, k: int, H: int, out=None, stream=None):
    out = out if out is not None else _empty((T, H), torch.bfloat16, y_sorted.device, stream)
    _check(_lib.moe_combine(_ptr(y_sorted), _ptr(inv_perm), _ptr(gates), T, k, H, _ptr(out),
                            _stream(stream)), "moe_combine")
    return out


def moe_forward(shape: Shape, logits, x, W_gate, W_up, W_down, out=None, topk_idx=None,
                gates=None, ws: Workspace | None = None, stream=None):
    dev = x.device
    out = out if out is not None else _empty((shape.T, shape.H), torch.bfloat16, dev, stream)
    ws = ws or Workspace(workspace_size(shape), dev, stream)
    _check(_lib.moe_forward(ctypes.byref(shape.c()), _ptr(logits), _ptr(x), _ptr(W_gate),
                            _ptr(W_up), _ptr(W_down), _ptr(out), _ptr(topk_idx), _ptr(gates),
                            ws.ptr, ws.nbytes, _stream(stream)), "moe_forward")
    return out


PROFILE_EVENTS = 9
PROFILE_STAGES = ("route", "permute", "gather", "gemm_gate_up", "thin_gate_up",
                  "gemm_down", "thin_down", "combine")


def moe_forward_profiled(shape: Shape, logits, x, W_gate, W_up, W_down, events, out=None,
                         topk_idx=None, gates=None, ws: Workspace | None = None,
                         stream=None):
    """moe_forward recording `events` (PROFILE_EVENTS torch.cuda.Event objects,
    created with enable_timing=True) at the stage boundaries."""
    assert len(events) == PROFILE_EVENTS
    dev = x.device
    out = out if out is not None else _empty((shape.T, shape.H), torch.bfloat16, dev, stream)
    ws = ws or Workspace(workspace_size(shape), dev, stream)
    for e in events:
        if e.cuda_event == 0:   # torch creates the CUDA event on first record
            e.record(stream if stream is not None else torch.cuda.current_stream())
    arr = (ctypes.c_void_p * PROFILE_EVENTS)(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(_lib.moe_forward_profiled(ctypes.byref(shape.c()), _ptr(logits), _ptr(x),
                                     _ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(out),
                                     _ptr(topk_idx), _ptr(gates), ws.ptr, ws.nbytes,
                                     _stream(stream), arr, PROFILE_EVENTS),
           "moe_forward_profiled")
    return out


def forward_launches(shape: Shape) -> int:
    """Kernels one moe_forward call launches for this shape."""
    return _lib.moe_forward_launches(ctypes.byref(shape.c()))


def layer_weight_bytes(shape: Shape) -> int:
    """Bytes of one layer's expert set (W_gate | W_up | W_down, bf16)."""
    return _lib.moe_layer_weight_bytes(ctypes.byref(shape.c()))


def pack_layer_weights(W_gate, W_up, W_down, pin: bool = True) -> torch.Tensor:
    """One layer's experts as the contiguous W_gate | W_up | W_down block the
    stager copies (pinned host memory by default)."""
    parts = [W_gate.reshape(-1), W_up.reshape(-1), W_down.reshape(-1)]
    out = torch.empty(sum(p.numel() for p in parts), dtype=torch.bfloat16, pin_memory=pin)
    off = 0
    for p in parts:   # straight into the (pinned) block, no intermediate copy
        out[off:off + p.numel()].copy_(p)
        off += p.numel()
    return out


class Stager:
    """Ring of `n_slots` device staging slots (allocated here with torch, owned
    by this object) plus the library's stager over them."""

    def __init__(self, shape: Shape, n_slots: int, device=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        self.slot_bytes = (layer_weight_bytes(shape) + 255) // 256 * 256
        self.n_slots = n_slots
        self._mem = torch.empty(n_slots * self.slot_bytes + 256, dtype=torch.uint8, device=device)
        off = (-self._mem.data_ptr()) % 256
        self.slots = self._mem[off:off + n_slots * self.slot_bytes]
        self._h = ctypes.c_void_p()
        _check(_lib.moe_stager_create(ctypes.c_void_p(self.slots.data_ptr()), n_slots,
                                      self.slot_bytes, ctypes.byref(self._h)), "moe_stager_create")

    def close(self):
        if self._h:
            _lib.moe_stager_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, shape: Shape, logits, x, host_weights, outs=None, ws: Workspace | None = None,
                compute=None, copy=None):
        """Runs len(host_weights) layers; logits[l] and outs[l] are device
        tensors, host_weights[l] pinned host blocks from pack_layer_weights.
        Returns the outputs."""
        L = len(host_weights)
        dev = x.device
        outs = outs if outs is not None else [
            _empty((shape.T, shape.H), torch.bfloat16, dev, compute) for _ in range(L)]
        ws = ws or Workspace(workspace_size(shape), dev, compute)
        compute = compute if compute is not None else torch.cuda.current_stream()
        copy = copy if copy is not None else torch.cuda.Stream(device=dev)
        PA = ctypes.c_void_p * max(L, 1)
        lg = PA(*[ctypes.c_void_p(t.data_ptr()) for t in logits])
        hw = PA(*[ctypes.c_void_p(t.data_ptr()) for t in host_weights])
        op = PA(*[ctypes.c_void_p(t.data_ptr()) for t in outs])
        _check(_lib.moe_forward_offload(self._h, ctypes.byref(shape.c()), L, lg, _ptr(x), hw, op,
                                        ws.ptr, ws.nbytes, ctypes.c_void_p(compute.cuda_stream),
                                        ctypes.c_void_p(copy.cuda_stream)), "moe_forward_offload")
        return outs


def pipe_workspace_size(shape: Shape) -> int:
    n = _lib.moe_pipe_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(1, "moe_pipe_workspace_size")
    return n


class Pipe:
    """The layer on activations in host memory: each forward() copies its
    inputs in on an h2d stream, computes on `compute` and copies the output
    back on a d2h stream, overlapping with the neighbouring calls.  Owns the
    library pipe, its workspace (with two staging slots) and the two copy
    streams; all calls use one shape and one compute stream."""

    def __init__(self, shape: Shape, device=None, compute=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        self.shape = shape
        self.compute = compute if compute is not None else torch.cuda.current_stream(device)
        self.h2d = torch.cuda.Stream(device=device)
        self.d2h = torch.cuda.Stream(device=device)
        self.ws = Workspace(pipe_workspace_size(shape), device, self.compute)
        self._h = ctypes.c_void_p()
        _check(_lib.moe_pipe_create(ctypes.byref(self._h)), "moe_pipe_create")

    def close(self):
        if self._h:
            _lib.moe_pipe_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, logits_h, x_h, W_gate, W_up, W_down, out_h):
        """Enqueues one layer: logits_h [T, E] fp32, x_h [T, H] bf16 and
        out_h [T, H] bf16 are (pinned) host tensors; out_h is written when
        the d2h stream reaches it (see synchronize())."""
        _check(_lib.moe_forward_host(self._h, ctypes.byref(self.shape.c()), _host_ptr(logits_h),
                                     _host_ptr(x_h), _ptr(W_gate), _ptr(W_up), _ptr(W_down),
                                     _host_ptr(out_h), self.ws.ptr, self.ws.nbytes,
                                     _stream(self.compute), _stream(self.h2d),
                                     _stream(self.d2h)), "moe_forward_host")
        return out_h

    def synchronize(self):
        self.d2h.synchronize()


class ExpertCache:
    """HBM expert cache (n_slots experts, least recently used evicted) over
    experts kept in pinned host memory; owns its device block (torch) and the
    library's cache."""

    def __init__(self, shape: Shape, n_slots: int, max_layers: int, device=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        self.shape = shape
        nbytes = _lib.moe_cache_bytes(ctypes.byref(shape.c()), n_slots, max_layers)
        if nbytes == 0:
            raise MoeError(1, "moe_cache_bytes")
        self._mem = torch.empty(nbytes + 256, dtype=torch.uint8, device=device)
        off = (-self._mem.data_ptr()) % 256
        self.mem = self._mem[off:off + nbytes]
        self._h = ctypes.c_void_p()
        _check(_lib.moe_cache_create(ctypes.byref(shape.c()), n_slots, max_layers,
                                     ctypes.c_void_p(self.mem.data_ptr()), nbytes,
                                     ctypes.byref(self._h)), "moe_cache_create")

    def close(self):
        if self._h:
            _lib.moe_cache_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stats(self):
        """(hits, misses) since creation."""
        h, m = ctypes.c_int64(), ctypes.c_int64()
        _check(_lib.moe_cache_stats(self._h, ctypes.byref(h), ctypes.byref(m)), "moe_cache_stats")
        return h.value, m.value

    def forward(self, layer_ids, logits, x, host_weights, outs=None, ws: Workspace | None = None,
                compute=None, copy=None):
        """Runs len(layer_ids) layers: logits[l], outs[l] device tensors,
        host_weights[l] pinned blocks from pack_layer_weights."""
        L = len(layer_ids)
        dev = x.device
        shape = self.shape
        outs = outs if outs is not None else [
            _empty((shape.T, shape.H), torch.bfloat16, dev, compute) for _ in range(L)]
        ws = ws or Workspace(workspace_size(shape), dev, compute)
        compute = compute if compute is not None else torch.cuda.current_stream()
        copy = copy if copy is not None else torch.cuda.Stream(device=dev)
        PA = ctypes.c_void_p * max(L, 1)
        ids = (ctypes.c_int32 * max(L, 1))(*layer_ids)
        lg = PA(*[ctypes.c_void_p(t.data_ptr()) for t in logits])
        hw = PA(*[ctypes.c_void_p(t.data_ptr()) for t in host_weights])
        op = PA(*[ctypes.c_void_p(t.data_ptr()) for t in outs])
        _check(_lib.moe_forward_cached(self._h, ctypes.byref(shape.c()), L, ids, lg, _ptr(x), hw,
                                       op, ws.ptr, ws.nbytes,
                                       ctypes.c_void_p(compute.cuda_stream),
                                       ctypes.c_void_p(copy.cuda_stream)), "moe_forward_cached")
        return outs


class DecodeGraph:
    """moe_forward for one fixed shape (a decode batch) captured once in a
    CUDA graph, as a serving engine runs decode steps: write the step's
    inputs into the static buffers `logits` [T, E] fp32 and `x` [T, H] bf16
    (device), call replay(), read `out` [T, H].  The weights are captured by
    address and must stay allocated."""

    def __init__(self, shape: Shape, W_gate, W_up, W_down, device=None):
        device = device or W_gate.device
        self.shape = shape
        self.logits = torch.zeros((shape.T, shape.E), dtype=torch.float32, device=device)
        self.x = torch.zeros((shape.T, shape.H), dtype=torch.bfloat16, device=device)
        self.out = torch.empty((shape.T, shape.H), dtype=torch.bfloat16, device=device)
        self.topk_idx = torch.empty((shape.T, shape.k), dtype=torch.int32, device=device)
        self.gates = torch.empty((shape.T, shape.k), dtype=torch.float32, device=device)
        self._W = (W_gate, W_up, W_down)
        self.stream = torch.cuda.Stream(device=device)
        self.ws = Workspace(workspace_size(shape), device, self.stream)
        self.stream.wait_stream(torch.cuda.current_stream(device))
        with torch.cuda.stream(self.stream):
            self._forward()                     # resolves lazy state before capture
        self.stream.synchronize()
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph, stream=self.stream):
            self._forward()

    def _forward(self):
        moe_forward(self.shape, self.logits, self.x, *self._W, out=self.out,
                    topk_idx=self.topk_idx, gates=self.gates, ws=self.ws, stream=self.stream)

    def replay(self):
        """Runs the captured layer on the current stream's timeline."""
        self.graph.replay()
        return self.out


def moe_quantize_rows(x: torch.Tensor, q=None, scales=None, stream=None):
    """x [rows, K] bf16 -> (q [rows, K] float8_e4m3fn, scales [rows, K/128]
    uint8): one power-of-two scale 2^(byte - 127) per 128 values of a row."""
    rows, K = x.shape
    q, qp = _out(q, (rows, K), _E4M3, x, stream)
    scales, sp = _out(scales, (rows, K // 128), _U8, x, stream)
    st = _lib.moe_quantize_rows(_in(x, _BF16, (rows, K)), rows, K, qp, sp, _on(stream, x))
    if st:
        raise MoeError(st, "moe_quantize_rows")
    return q, scales


def moe_quantize_weights(W: torch.Tensor, q=None, scales=None, stream=None):
    """W [E, N, K] bf16 -> (q [E, N, K] float8_e4m3fn, scales [E, N/128, K/128]
    uint8): one power-of-two scale per 128 x 128 block."""
    E, N, K = W.shape
    q, qp = _out(q, (E, N, K), _E4M3, W, stream)
    scales, sp = _out(scales, (E, N // 128, K // 128), _U8, W, stream)
    st = _lib.moe_quantize_weights(_in(W, _BF16, (E, N, K)), E, N, K, qp, sp, _on(stream, W))
    if st:
        raise MoeError(st, "moe_quantize_weights")
    return q, scales


def grouped_gemm_fp8_workspace_size(rows: int, E: int) -> int:
    n = _lib.moe_grouped_gemm_fp8_workspace_size(rows, E)
    if n == 0:
        raise MoeError(1, "moe_grouped_gemm_fp8_workspace_size")
    return n


def moe_grouped_gemm_fp8(x, x_scales, offsets, W, W_scales, y=None, ws: Workspace | None = None,
                         stream=None):
    """y[p] = x[p] . W[e]^T for the rows offsets[e] <= p < offsets[e + 1], both
    operands 8-bit with block scales (as moe_quantize_rows / _weights give
    them); y [rows, N] bf16.  E = 1 (offsets [0, rows]) is the dense product."""
    rows, K = x.shape
    E, N, _ = W.shape
    y, yp = _out(y, (rows, N), _BF16, x, stream)
    ws = ws or Workspace(grouped_gemm_fp8_workspace_size(rows, E), x.device, stream)
    st = _lib.moe_grouped_gemm_fp8(
        _in(x, _E4M3, (rows, K)), _in(x_scales, _U8, (rows, K // 128)), rows,
        _in(offsets, _I32, (E + 1,)), E, N, K, _in(W, _E4M3, (E, N, K)),
        _in(W_scales, _U8, (E, N // 128, K // 128)), yp, ws.addr, ws.nbytes,
        _on(stream, x))
    if st:
        raise MoeError(st, "moe_grouped_gemm_fp8")
    return y


@dataclass(frozen=True)
class Fp8Experts:
    """A layer's experts in 8 bits: gate, up [E, I, H] and down [E, H, I]
    float8_e4m3fn, each with its scales [E, rows/128, cols/128] uint8.  The
    tensors are checked here, and again by a call that finds one of them in
    another place (its storage was replaced)."""
    gate: torch.Tensor
    gate_scales: torch.Tensor
    up: torch.Tensor
    up_scales: torch.Tensor
    down: torch.Tensor
    down_scales: torch.Tensor

    def __post_init__(self):
        E, I, H = self.gate.shape
        a, b = (E, I // 128, H // 128), (E, H // 128, I // 128)
        at = (_in(self.gate, _E4M3, (E, I, H)), _in(self.gate_scales, _U8, a),
              _in(self.up, _E4M3, (E, I, H)), _in(self.up_scales, _U8, a),
              _in(self.down, _E4M3, (E, H, I)), _in(self.down_scales, _U8, b))
        object.__setattr__(self, "_sizes", (E, H, I))
        object.__setattr__(self, "_at", at)
        object.__setattr__(self, "_c", MoeFp8Experts(*at))

    def _tensors(self):
        return (self.gate, self.gate_scales, self.up, self.up_scales, self.down, self.down_scales)

    def __reduce__(self):
        """Copies and pickles are of the tensors, as bytes (torch's pickle does
        not read 8-bit floating point back)."""
        return Fp8Experts._of_bytes, tuple(t.view(_U8) for t in self._tensors())

    @staticmethod
    def _of_bytes(*parts):
        return Fp8Experts(*(t.view(_U8 if i % 2 else _E4M3) for i, t in enumerate(parts)))

    def ref(self, shape: Shape):
        """The C structure, for a layer of these sizes."""
        if tuple(t.data_ptr() for t in self._tensors()) != self._at:
            self.__post_init__()
        assert self._sizes == (shape.E, shape.H, shape.I), \
            f"experts of (E, H, I) = {self._sizes}, layer of {(shape.E, shape.H, shape.I)}"
        return ctypes.byref(self._c)


def quantize_experts(W_gate, W_up, W_down, stream=None) -> Fp8Experts:
    """bf16 experts (the layouts of moe_forward) -> Fp8Experts."""
    return Fp8Experts(*moe_quantize_weights(W_gate, stream=stream),
                      *moe_quantize_weights(W_up, stream=stream),
                      *moe_quantize_weights(W_down, stream=stream))


def expert_ffn_fp8_workspace_size(shape: Shape) -> int:
    n = _lib.moe_expert_ffn_fp8_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(1, "moe_expert_ffn_fp8_workspace_size")
    return n


def moe_expert_ffn_fp8(shape: Shape, x, perm, offsets, experts: Fp8Experts, y_sorted=None,
                       ws: Workspace | None = None, stream=None):
    """moe_expert_ffn on 8-bit experts (perm, offsets from moe_permute)."""
    P, T, H = shape.P, shape.T, shape.H
    y_sorted, yp = _out(y_sorted, (P, H), _BF16, x, stream)
    ws = ws or Workspace(expert_ffn_fp8_workspace_size(shape), x.device, stream)
    st = _lib.moe_expert_ffn_fp8(
        ctypes.byref(shape.c()), _in(x, _BF16, (T, H)), _in(perm, _I32, (P,)),
        _in(offsets, _I32, (shape.E + 1,)), experts.ref(shape), yp,
        ws.addr, ws.nbytes, _on(stream, x))
    if st:
        raise MoeError(st, "moe_expert_ffn_fp8")
    return y_sorted


def fp8_workspace_size(shape: Shape) -> int:
    n = _lib.moe_fp8_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(1, "moe_fp8_workspace_size")
    return n


def moe_forward_fp8(shape: Shape, logits, x, experts: Fp8Experts, out=None, topk_idx=None,
                    gates=None, ws: Workspace | None = None, stream=None):
    """moe_forward on 8-bit experts."""
    T, H, k = shape.T, shape.H, shape.k
    out, op = _out(out, (T, H), _BF16, x, stream)
    ws = ws or Workspace(fp8_workspace_size(shape), x.device, stream)
    st = _lib.moe_forward_fp8(
        ctypes.byref(shape.c()), _in(logits, _F32, (T, shape.E)), _in(x, _BF16, (T, H)),
        experts.ref(shape), op, _opt(topk_idx, _I32, (T, k)),
        _opt(gates, _F32, (T, k)), ws.addr, ws.nbytes, _on(stream, x))
    if st:
        raise MoeError(st, "moe_forward_fp8")
    return out


def balance_workspace_size(T: int, E: int, S: int = 1) -> int:
    n = _lib.moe_balance_workspace_size(T, E, S)
    if n == 0:
        raise MoeError(1, "moe_balance_workspace_size")
    return n


def moe_balance(logits, topk_idx, seq_offsets=None, coef: float = 1.0, loss=None, counts=None,
                stats=None, ws: Workspace | None = None, stream=None):
    """The router's balance loss over packed sequences (seq_offsets int32
    [S + 1], None: one sequence of all tokens).  Returns (loss [] fp32, counts
    [S, E] int32, stats [T, 2] fp32 for moe_balance_backward)."""
    T, E = logits.shape
    k = topk_idx.shape[1]
    S = _sequences(seq_offsets)
    loss, lp = _out(loss, (), _F32, logits, stream)
    counts, cp = _out(counts, (S, E), _I32, logits, stream)
    stats, sp = _out(stats, (T, 2), _F32, logits, stream)
    ws = ws or Workspace(balance_workspace_size(T, E, S), logits.device, stream)
    st = _lib.moe_balance(
        _in(logits, _F32, (T, E)), _in(topk_idx, _I32, (T, k)), T, E, k,
        _opt(seq_offsets, _I32, (S + 1,)), S, coef, lp, cp, sp, ws.addr, ws.nbytes, _on(stream, logits))
    if st:
        raise MoeError(st, "moe_balance")
    return loss, counts, stats


def moe_balance_backward(logits, stats, counts, k: int, seq_offsets=None, coef: float = 1.0,
                         d_loss=None, topk_idx=None, gates=None, d_gates=None, d_logits=None,
                         stream=None):
    """Gradient of the logits from the balance loss (d_loss: fp32 scalar on the
    device, None for 1) and, where topk_idx, gates and d_gates are given, from
    the router's gates.  Returns d_logits [T, E] fp32."""
    T, E = logits.shape
    S = _sequences(seq_offsets)
    d_logits, dp = _out(d_logits, (T, E), _F32, logits, stream)
    st = _lib.moe_balance_backward(
        _in(logits, _F32, (T, E)), _in(stats, _F32, (T, 2)), _in(counts, _I32, (S, E)),
        _opt(seq_offsets, _I32, (S + 1,)), T, E, k, S, coef, _opt(d_loss, _F32, ()),
        _opt(topk_idx, _I32, (T, k)), _opt(gates, _F32, (T, k)), _opt(d_gates, _F32, (T, k)),
        dp, _on(stream, logits))
    if st:
        raise MoeError(st, "moe_balance_backward")
    return d_logits


@dataclass(eq=False)
class SavedFfn:
    """What moe_expert_ffn_train keeps for moe_expert_ffn_backward, by sorted
    row: the two projections gate, up [P, I], with x [T, H].  In bf16 (the
    scales are None; x is the call's own input), or in 8 bits: float8_e4m3fn
    with scales [P, I/128] and [T, H/128] uint8.  A backward pass without the
    weights' gradients does not read x: it may be None there."""
    x: torch.Tensor | None
    gate: torch.Tensor
    up: torch.Tensor
    x_scales: torch.Tensor | None = None
    gate_scales: torch.Tensor | None = None
    up_scales: torch.Tensor | None = None

    def ref(self, shape: Shape, need_x: bool = True):
        """The C structure, for a layer of these sizes (need_x: with x)."""
        T, H, I = shape.T, shape.H, shape.I
        P = T * shape.k
        if self.gate_scales is None:
            x = _in(self.x, _BF16, (T, H)) if need_x else None
            return ctypes.byref(MoeSaved(0, x, None, _in(self.gate, _BF16, (P, I)), None, _in(self.up, _BF16, (P, I)), None))
        rows = (P, I // 128)
        x, x_scales = (_in(self.x, _E4M3, (T, H)), _in(self.x_scales, _U8, (T, H // 128))) if need_x else (None, None)
        return ctypes.byref(MoeSaved(1, x, x_scales, _in(self.gate, _E4M3, (P, I)), _in(self.gate_scales, _U8, rows),
                                     _in(self.up, _E4M3, (P, I)), _in(self.up_scales, _U8, rows)))

    @staticmethod
    def empty(shape: Shape, x: torch.Tensor, checkpoint: str = "bf16", stream=None) -> "SavedFfn":
        """Room for one forward call on x ("bf16" or "fp8" checkpoints)."""
        assert checkpoint in ("bf16", "fp8"), f"checkpoint = {checkpoint!r}: 'bf16' or 'fp8'"
        T, P, H, I, dev = shape.T, shape.P, shape.H, shape.I, x.device
        if checkpoint == "bf16":
            return SavedFfn(x, _empty((P, I), _BF16, dev, stream), _empty((P, I), _BF16, dev, stream))
        return SavedFfn(*(_empty(s, _E4M3, dev, stream) for s in ((T, H), (P, I), (P, I))),
                        *(_empty(s, _U8, dev, stream) for s in ((T, H // 128), (P, I // 128), (P, I // 128))))


def expert_ffn_train_workspace_size(shape: Shape) -> int:
    n = _lib.moe_expert_ffn_train_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(1, "moe_expert_ffn_train_workspace_size")
    return n


def moe_expert_ffn_train(shape: Shape, x, perm, offsets, W_gate, W_up, W_down,
                         checkpoint: str = "bf16", y_sorted=None, saved: SavedFfn | None = None,
                         ws: Workspace | None = None, stream=None):
    """moe_expert_ffn that keeps what the backward pass needs, in bf16 or
    ("fp8") in 8 bits.  perm and offsets from moe_permute, or None with
    E = k = 1: a dense block.  `saved`: room from an earlier call, whose kind
    then counts.  Returns (y_sorted [P, H] bf16, SavedFfn)."""
    T, E, H, I = shape.T, shape.E, shape.H, shape.I
    P = T * shape.k
    xp = _in(x, _BF16, (T, H))
    y_sorted, yp = _out(y_sorted, (P, H), _BF16, x, stream)
    if saved is None:
        saved = SavedFfn.empty(shape, x, checkpoint, stream)
    elif saved.gate_scales is None:      # the record of this call: its own x
        saved = SavedFfn(x, saved.gate, saved.up)
    up = (E, I, H)
    ws = ws or Workspace(expert_ffn_train_workspace_size(shape), x.device, stream)
    st = _lib.moe_expert_ffn_train(
        ctypes.byref(shape.c()), xp, _opt(perm, _I32, (P,)), _opt(offsets, _I32, (E + 1,)),
        _in(W_gate, _BF16, up), _in(W_up, _BF16, up), _in(W_down, _BF16, (E, H, I)),
        yp, saved.ref(shape), ws.addr, ws.nbytes, _on(stream, x))
    if st:
        raise MoeError(st, "moe_expert_ffn_train")
    return y_sorted, saved


def expert_ffn_backward_workspace_size(shape: Shape) -> int:
    n = _lib.moe_expert_ffn_backward_workspace_size(ctypes.byref(shape.c()))
    if n == 0:
        raise MoeError(1, "moe_expert_ffn_backward_workspace_size")
    return n


def moe_expert_ffn_backward(shape: Shape, d_out, saved: SavedFfn, perm, offsets, inv_perm, W_gate,
                            W_up, W_down, gates=None, need_x: bool = True,
                            need_weights: bool = True, d_x=None, d_gates=None, dW=None,
                            ws: Workspace | None = None, stream=None):
    """Gradients of the layer's experts and gates from d_out [T, H] bf16, the
    gradient of moe_combine's output (gates None: all 1); saved.x is read for the
    weights' gradients only.  Returns (d_x [T, H]
    bf16, d_gates [T, k] fp32, dW_gate, dW_up, dW_down bf16); None in the place
    of what is not needed, and of d_gates without gates."""
    T, E, k, H, I = shape.T, shape.E, shape.k, shape.H, shape.I
    P, up, down = T * k, (E, I, H), (E, H, I)
    dp = _in(d_out, _BF16, (T, H))
    xp = gp = wg = wu = wd = None
    if need_x:
        d_x, xp = _out(d_x, (T, H), _BF16, d_out, stream)
    if gates is not None:
        d_gates, gp = _out(d_gates, (T, k), _F32, d_out, stream)
    if need_weights:
        given = dW if dW is not None else (None, None, None)
        dWg, wg = _out(given[0], up, _BF16, d_out, stream)
        dWu, wu = _out(given[1], up, _BF16, d_out, stream)
        dWd, wd = _out(given[2], down, _BF16, d_out, stream)
    ws = ws or Workspace(expert_ffn_backward_workspace_size(shape), d_out.device, stream)
    st = _lib.moe_expert_ffn_backward(
        ctypes.byref(shape.c()), dp, _opt(gates, _F32, (T, k)), saved.ref(shape, need_weights),
        _opt(perm, _I32, (P,)), _opt(offsets, _I32, (E + 1,)), _opt(inv_perm, _I32, (P,)),
        _in(W_gate, _BF16, up), _in(W_up, _BF16, up), _in(W_down, _BF16, down),
        xp, gp, wg, wu, wd, ws.addr, ws.nbytes, _on(stream, d_out))
    if st:
        raise MoeError(st, "moe_expert_ffn_backward")
    return (d_x if need_x else None, d_gates if gates is not None else None,
            *((dWg, dWu, dWd) if need_weights else (None, None, None)))


def moe_dequantize_rows(q, scales, x=None, stream=None):
    """The values of 8-bit rows (q [rows, K] float8_e4m3fn, scales [rows, K/128]
    uint8) as bf16 [rows, K]."""
    rows, K = q.shape
    x, xp = _out(x, (rows, K), _BF16, q, stream)
    st = _lib.moe_dequantize_rows(_in(q, _E4M3, (rows, K)), _in(scales, _U8, (rows, K // 128)), rows, K,
                                  xp, _on(stream, q))
    if st:
        raise MoeError(st, "moe_dequantize_rows")
    return x


ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}


def grouped_gemm_workspace_size(rows: int, E: int, N: int, K: int) -> int:
    n = _lib.moe_grouped_gemm_workspace_size(rows, E, N, K)
    if n == 0:
        raise MoeError(1, "moe_grouped_gemm_workspace_size")
    return n


def moe_grouped_gemm(x, W, offsets=None, bias=None, activation: str = "none", residual=None,
                     out_dtype=torch.bfloat16, y=None, ws: Workspace | None = None, stream=None):
    """y[p] = act(x[p] . W[e]^T + bias[e]) + residual[p] for the rows
    offsets[e] <= p < offsets[e + 1] (None with E = 1: all); x [rows, K],
    W [E, N, K] and residual [rows, N] bf16, bias [E, N] fp32; y [rows, N] of
    out_dtype (bf16 or fp32).  activation: "none", "relu", "gelu" or "silu"."""
    rows, K = x.shape
    E, N, _ = W.shape
    assert activation in ACTIVATIONS, f"activation = {activation!r}: one of {', '.join(ACTIVATIONS)}"
    assert out_dtype in (_BF16, _F32), f"out_dtype = {out_dtype}: bfloat16 or float32"
    y, yp = _out(y, (rows, N), out_dtype, x, stream)
    ws = ws or Workspace(grouped_gemm_workspace_size(rows, E, N, K), x.device, stream)
    st = _lib.moe_grouped_gemm(
        _in(x, _BF16, (rows, K)), rows, _opt(offsets, _I32, (E + 1,)), E, N, K,
        _in(W, _BF16, (E, N, K)), _opt(bias, _F32, (E, N)), ACTIVATIONS[activation],
        _opt(residual, _BF16, (rows, N)), yp, int(out_dtype is _F32), ws.addr, ws.nbytes,
        _on(stream, x))
    if st:
        raise MoeError(st, "moe_grouped_gemm")
    return y


def raw_lib():
    """The loaded ctypes library (for callers that pass raw pointers)."""
    return _lib
