"""Python binding of libmoe.so, the MI355X MoE expert-layer library.

Argument marshalling only: every function here has the name of the C entry
point it calls (declared in include/moe.h), takes torch tensors that live on
the GPU, checks their dtype/shape/contiguity, and passes their device pointers
and the current HIP stream through ctypes.  Every step of the layer runs in the
library's HIP kernels; there is no fallback of any kind -- if libmoe.so is
missing or cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "Dims", "MoeError", "F32", "BF16", "lib_path", "load", "moe_init", "moe_status_str",
    "moe_last_error", "moe_workspace_bytes", "moe_route", "moe_dispatch", "moe_expert_ffn_up",
    "moe_expert_ffn_down", "moe_expert_ffn", "moe_combine", "moe_dispatch_ffn",
    "moe_ffn_combine", "moe_combine_bwd", "moe_expert_ffn_bwd_data",
    "moe_expert_ffn_bwd_weight", "moe_dispatch_bwd", "moe_route_bwd", "moe_expert_ffn_bwd_act",
    "moe_expert_ffn_bwd_input", "moe_expert_ffn_bwd_weight_gate_up", "moe_expert_ffn_bwd_weight_down",
    "moe_expert_ffn_bwd", "moe_sync_status", "moe_route_noalloc", "Tuning", "moe_get_tuning",
    "moe_tuning_predict", "moe_decode_workspace_bytes", "moe_decode", "moe_decode_mx", "moe_mx_bytes",
    "moe_mx_quantize", "moe_mx_dequantize", "moe_balance_workspace_bytes", "moe_balance", "moe_balance_bwd",
    "EXACT", "Newton", "MuonParams", "NEWTON_COEF", "moe_muon_workspace_bytes", "moe_orthogonalize", "moe_muon",
]

F32, BF16 = 0, 1
_TORCH_DTYPE = {F32: torch.float32, BF16: torch.bfloat16}

_PKG = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_PKG, "libmoe.so")


class Dims(ctypes.Structure):
    """moe_dims.  I_shared defaults to I when there are shared experts."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("K", ctypes.c_int32), ("I", ctypes.c_int32), ("n_shared", ctypes.c_int32),
                ("I_shared", ctypes.c_int32), ("dtype", ctypes.c_int32)]

    def __init__(self, T=0, H=0, E=0, K=0, I=0, n_shared=0, I_shared=None, dtype=BF16):
        if I_shared is None:
            I_shared = I if n_shared else 0
        super().__init__(T, H, E, K, I, n_shared, I_shared, dtype)

    @property
    def R(self) -> int:
        return self.T * self.K

    @property
    def RA(self) -> int:
        return self.T * self.K + self.n_shared * self.T

    @property
    def torch_dtype(self):
        return _TORCH_DTYPE[self.dtype]


class Tuning(ctypes.Structure):
    """moe_tuning: the schedule knobs (band heights, fused task sizes)."""
    _fields_ = [("band_up", ctypes.c_int32), ("band_act", ctypes.c_int32),
                ("small_group", ctypes.c_int32), ("band_wgrad_up", ctypes.c_int32),
                ("band_wgrad_down", ctypes.c_int32), ("combine_tokens", ctypes.c_int32),
                ("copy_tokens", ctypes.c_int32), ("copy_in_tiles", ctypes.c_int32)]

    def as_dict(self):
        return {f: int(getattr(self, f)) for f, _ in self._fields_}


class MoeError(RuntimeError):
    def __init__(self, status: int, name: str, detail: str):
        super().__init__(f"{name} failed: {moe_status_str(status)}: {detail}")
        self.status = status


_P = ctypes.c_void_p
_D = ctypes.POINTER(Dims)
_SIGS = {
    "moe_init": (ctypes.c_int, [ctypes.c_int]),
    "moe_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_workspace_bytes": (ctypes.c_size_t, [_D]),
    "moe_get_tuning": (ctypes.c_int, [_D, ctypes.POINTER(Tuning)]),
    "moe_tuning_predict": (ctypes.c_double, [_D, ctypes.c_char_p, ctypes.c_int]),
    "moe_sync_status": (ctypes.c_int, [_P]),
    "moe_route": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_route_noalloc": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P]),
    "moe_route_ranks_workspace_bytes": (ctypes.c_size_t, [_D, ctypes.c_int]),
    "moe_route_ranks": (ctypes.c_int, [_D, _P, ctypes.c_int, _P, _P, _P, _P, _P, _P, _P,
                                       ctypes.c_size_t, _P]),
    "moe_dispatch": (ctypes.c_int, [_D, _P, _P, _P, _P]),
    "moe_expert_ffn_up": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn_down": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                      ctypes.c_size_t, _P]),
    "moe_combine": (ctypes.c_int, [_D, _P, _P, _P, _P, _P]),
    "moe_dispatch_ffn": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                        ctypes.c_size_t, _P]),
    "moe_ffn_combine": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_combine_bwd": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P]),
    "moe_expert_ffn_bwd_data": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                               _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn_bwd_weight": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                                 _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn_bwd": (ctypes.c_int, [_D] + [_P] * 22 + [ctypes.c_size_t, _P]),
    "moe_expert_ffn_bwd_act": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn_bwd_input": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_expert_ffn_bwd_weight_gate_up": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                                         ctypes.c_size_t, _P]),
    "moe_expert_ffn_bwd_weight_down": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]),
    "moe_dispatch_bwd": (ctypes.c_int, [_D, _P, _P, _P, _P]),
    "moe_route_bwd": (ctypes.c_int, [_D, _P, _P, _P, _P, _P]),
    "moe_decode_workspace_bytes": (ctypes.c_size_t, [_D]),
    "moe_decode": (ctypes.c_int, [_D] + [_P] * 13 + [ctypes.c_size_t, _P]),
    "moe_decode_mx": (ctypes.c_int, [_D] + [_P] * 13 + [ctypes.c_size_t, _P]),
    "moe_mx_bytes": (ctypes.c_size_t, [ctypes.c_int] * 3),
    "moe_mx_quantize": (ctypes.c_int, [ctypes.c_int] * 4 + [_P, _P, _P]),
    "moe_mx_dequantize": (ctypes.c_int, [ctypes.c_int] * 4 + [_P, _P, _P]),
}

_lib = None


def load() -> ctypes.CDLL:
    """Load libmoe.so (once).  Raises if it is missing: there is no fallback."""
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with "
                               "`python -m combine_moe_route_histogram_amd.build`")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def moe_status_str(status: int) -> str:
    return load().moe_status_str(status).decode()


def moe_last_error() -> str:
    return load().moe_last_error().decode()


def moe_init(device: int = 0) -> None:
    st = load().moe_init(device)
    if st:
        raise MoeError(st, "moe_init", moe_last_error())


def moe_sync_status(stream=None) -> None:
    """Wait for `stream`; raise MoeError (MOE_ETIMEOUT) if a bounded wait inside
    a kernel gave up since the last check, or on a HIP error."""
    _call("moe_sync_status", _stream(stream))


def moe_get_tuning(d: Dims) -> Tuning:
    """The schedule knobs the library uses for these dims."""
    t = Tuning()
    _call("moe_get_tuning", ctypes.byref(d), ctypes.byref(t))
    return t


def moe_tuning_predict(d: Dims, knob: str, value: int) -> float:
    """The band model's predicted bytes beyond L2 per flop (negative: not modelled)."""
    return float(load().moe_tuning_predict(ctypes.byref(d), knob.encode(), int(value)))


def moe_workspace_bytes(d: Dims) -> int:
    return int(load().moe_workspace_bytes(ctypes.byref(d)))


# ---------------------------------------------------------------- marshalling

def _ptr(t, name, dtype=None, numel=None):
    if t is None:
        return None
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype == dtype)
            and (numel is None or t.numel() >= numel)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor or None")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (3 us a call), in the versions of
# torch that have it: it is not part of torch's public interface.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ws(ws):
    if ws is None:
        return None, 0
    return _ptr(ws, "ws", torch.uint8), ws.numel()


def _call(name, *args):
    st = getattr(load(), name)(*args)
    if st:
        raise MoeError(st, name, moe_last_error())


# ---------------------------------------------------------------- forward

def moe_route(d: Dims, logits, topk_idx, topk_w, counts, offsets, slot, slot_src, ws, stream=None):
    T, E, K, R = d.T, d.E, d.K, d.R
    wp, wn = _ws(ws)
    _call("moe_route", ctypes.byref(d), _ptr(logits, "logits", torch.float32, T * E),
          _ptr(topk_idx, "topk_idx", torch.int32, T * K), _ptr(topk_w, "topk_w", torch.float32, T * K),
          _ptr(counts, "counts", torch.int32, E), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(slot, "slot", torch.int32, T * K), _ptr(slot_src, "slot_src", torch.int32, R),
          wp, wn, _stream(stream))


def moe_route_noalloc(d: Dims, logits, topk_idx, topk_w, counts, offsets, slot, slot_src,
                      stream=None):
    T, E, K, R = d.T, d.E, d.K, d.R
    _call("moe_route_noalloc", ctypes.byref(d), _ptr(logits, "logits", torch.float32, T * E),
          _ptr(topk_idx, "topk_idx", torch.int32, T * K), _ptr(topk_w, "topk_w", torch.float32, T * K),
          _ptr(counts, "counts", torch.int32, E), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(slot, "slot", torch.int32, T * K), _ptr(slot_src, "slot_src", torch.int32, R),
          _stream(stream))


def moe_route_ranks_workspace_bytes(d: Dims, G: int) -> int:
    return int(load().moe_route_ranks_workspace_bytes(ctypes.byref(d), int(G)))


def moe_route_ranks(d: Dims, topk_idx, G: int, rank_counts, rank_base, counts, offsets, slot,
                    slot_src, ws, stream=None):
    T, E, K, R = d.T, d.E, d.K, d.R
    wp, wn = _ws(ws)
    _call("moe_route_ranks", ctypes.byref(d), _ptr(topk_idx, "topk_idx", torch.int32, T * K),
          int(G), _ptr(rank_counts, "rank_counts", torch.int32, G * E),
          _ptr(rank_base, "rank_base", torch.int32, G * E),
          _ptr(counts, "counts", torch.int32, E), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(slot, "slot", torch.int32, T * K), _ptr(slot_src, "slot_src", torch.int32, R),
          wp, wn, _stream(stream))


def moe_dispatch(d: Dims, x, slot, x_perm, stream=None):
    dt = d.torch_dtype
    _call("moe_dispatch", ctypes.byref(d), _ptr(x, "x", dt, d.T * d.H),
          _ptr(slot, "slot", torch.int32, d.T * d.K), _ptr(x_perm, "x_perm", dt, d.R * d.H),
          _stream(stream))


def moe_expert_ffn_up(d: Dims, x_perm, x, offsets, w1, w3, ws1, ws3, ab, h, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_up", ctypes.byref(d), _ptr(x_perm, "x_perm", dt, d.R * H),
          _ptr(x, "x", dt, d.T * H), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(w1, "w1", dt, E * H * I), _ptr(w3, "w3", dt, E * H * I),
          _ptr(ws1, "ws1", dt, Ns * H * I), _ptr(ws3, "ws3", dt, Ns * H * I),
          _ptr(ab, "ab", dt, d.RA * 2 * I), _ptr(h, "h", dt, d.RA * I), wp, wn, _stream(stream))


def moe_expert_ffn_down(d: Dims, h, offsets, w2, ws2, y, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_down", ctypes.byref(d), _ptr(h, "h", dt, d.RA * I),
          _ptr(offsets, "offsets", torch.int32, E + 1), _ptr(w2, "w2", dt, E * I * H),
          _ptr(ws2, "ws2", dt, Ns * I * H), _ptr(y, "y", dt, d.RA * H), wp, wn, _stream(stream))


def moe_expert_ffn(d: Dims, x_perm, x, offsets, w1, w3, w2, ws1, ws3, ws2, ab, h, y, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_expert_ffn", ctypes.byref(d), _ptr(x_perm, "x_perm", dt, d.R * H),
          _ptr(x, "x", dt, d.T * H), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(w1, "w1", dt, E * H * I), _ptr(w3, "w3", dt, E * H * I), _ptr(w2, "w2", dt, E * I * H),
          _ptr(ws1, "ws1", dt, Ns * H * I), _ptr(ws3, "ws3", dt, Ns * H * I),
          _ptr(ws2, "ws2", dt, Ns * I * H), _ptr(ab, "ab", dt, d.RA * 2 * I),
          _ptr(h, "h", dt, d.RA * I), _ptr(y, "y", dt, d.RA * H), wp, wn, _stream(stream))


def moe_combine(d: Dims, y, slot, topk_w, out, stream=None):
    dt = d.torch_dtype
    _call("moe_combine", ctypes.byref(d), _ptr(y, "y", dt, d.RA * d.H),
          _ptr(slot, "slot", torch.int32, d.T * d.K), _ptr(topk_w, "topk_w", torch.float32, d.T * d.K),
          _ptr(out, "out", dt, d.T * d.H), _stream(stream))


def moe_dispatch_ffn(d: Dims, x, slot_src, slot, offsets, w1, w3, ws1, ws3, x_perm, ab, h, ws,
                     stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_dispatch_ffn", ctypes.byref(d), _ptr(x, "x", dt, d.T * H),
          _ptr(slot_src, "slot_src", torch.int32, d.R), _ptr(slot, "slot", torch.int32, d.T * d.K),
          _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(w1, "w1", dt, E * H * I), _ptr(w3, "w3", dt, E * H * I),
          _ptr(ws1, "ws1", dt, Ns * H * I), _ptr(ws3, "ws3", dt, Ns * H * I),
          _ptr(x_perm, "x_perm", dt, d.R * H), _ptr(ab, "ab", dt, d.RA * 2 * I),
          _ptr(h, "h", dt, d.RA * I), wp, wn, _stream(stream))


def moe_ffn_combine(d: Dims, h, offsets, w2, ws2, slot, topk_w, y, out, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_ffn_combine", ctypes.byref(d), _ptr(h, "h", dt, d.RA * I),
          _ptr(offsets, "offsets", torch.int32, E + 1), _ptr(w2, "w2", dt, E * I * H),
          _ptr(ws2, "ws2", dt, Ns * I * H), _ptr(slot, "slot", torch.int32, d.T * d.K),
          _ptr(topk_w, "topk_w", torch.float32, d.T * d.K), _ptr(y, "y", dt, d.RA * H),
          _ptr(out, "out", dt, d.T * H), wp, wn, _stream(stream))


# ---------------------------------------------------------------- backward

def moe_combine_bwd(d: Dims, dout, y, slot, topk_w, dy, dtopk_w, stream=None):
    dt = d.torch_dtype
    _call("moe_combine_bwd", ctypes.byref(d), _ptr(dout, "dout", dt, d.T * d.H),
          _ptr(y, "y", dt, d.R * d.H), _ptr(slot, "slot", torch.int32, d.T * d.K),
          _ptr(topk_w, "topk_w", torch.float32, d.T * d.K), _ptr(dy, "dy", dt, d.R * d.H),
          _ptr(dtopk_w, "dtopk_w", torch.float32, d.T * d.K), _stream(stream))


def moe_expert_ffn_bwd_data(d: Dims, dy, dout, offsets, w1, w3, w2, ws1, ws3, ws2, ab, dab, dx_rows,
                            ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_bwd_data", ctypes.byref(d), _ptr(dy, "dy", dt, d.R * H),
          _ptr(dout, "dout", dt, d.T * H), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(w1, "w1", dt, E * H * I), _ptr(w3, "w3", dt, E * H * I), _ptr(w2, "w2", dt, E * I * H),
          _ptr(ws1, "ws1", dt, Ns * H * I), _ptr(ws3, "ws3", dt, Ns * H * I),
          _ptr(ws2, "ws2", dt, Ns * I * H), _ptr(ab, "ab", dt, d.RA * 2 * I),
          _ptr(dab, "dab", dt, d.RA * 2 * I), _ptr(dx_rows, "dx_rows", dt, d.RA * H), wp, wn,
          _stream(stream))


def moe_expert_ffn_bwd_weight(d: Dims, x_perm, x, h, dy, dout, dab, offsets, dw1, dw3, dw2,
                              dws1, dws3, dws2, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    f32 = torch.float32
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_bwd_weight", ctypes.byref(d), _ptr(x_perm, "x_perm", dt, d.R * H),
          _ptr(x, "x", dt, d.T * H), _ptr(h, "h", dt, d.RA * I), _ptr(dy, "dy", dt, d.R * H),
          _ptr(dout, "dout", dt, d.T * H), _ptr(dab, "dab", dt, d.RA * 2 * I),
          _ptr(offsets, "offsets", torch.int32, E + 1), _ptr(dw1, "dw1", f32, E * H * I),
          _ptr(dw3, "dw3", f32, E * H * I), _ptr(dw2, "dw2", f32, E * I * H),
          _ptr(dws1, "dws1", f32, Ns * H * I), _ptr(dws3, "dws3", f32, Ns * H * I),
          _ptr(dws2, "dws2", f32, Ns * I * H), wp, wn, _stream(stream))


def moe_expert_ffn_bwd(d: Dims, dy, dout, offsets, w1, w3, w2, ws1, ws3, ws2, ab, x_perm, x, h,
                       dab, dx_rows, dw1, dw3, dw2, dws1, dws3, dws2, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    f32 = torch.float32
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_bwd", ctypes.byref(d), _ptr(dy, "dy", dt, d.R * H),
          _ptr(dout, "dout", dt, d.T * H), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(w1, "w1", dt, E * H * I), _ptr(w3, "w3", dt, E * H * I), _ptr(w2, "w2", dt, E * I * H),
          _ptr(ws1, "ws1", dt, Ns * H * I), _ptr(ws3, "ws3", dt, Ns * H * I),
          _ptr(ws2, "ws2", dt, Ns * I * H), _ptr(ab, "ab", dt, d.RA * 2 * I),
          _ptr(x_perm, "x_perm", dt, d.R * H), _ptr(x, "x", dt, d.T * H), _ptr(h, "h", dt, d.RA * I),
          _ptr(dab, "dab", dt, d.RA * 2 * I), _ptr(dx_rows, "dx_rows", dt, d.RA * H),
          _ptr(dw1, "dw1", f32, E * H * I), _ptr(dw3, "dw3", f32, E * H * I),
          _ptr(dw2, "dw2", f32, E * I * H), _ptr(dws1, "dws1", f32, Ns * H * I),
          _ptr(dws3, "dws3", f32, Ns * H * I), _ptr(dws2, "dws2", f32, Ns * I * H), wp, wn,
          _stream(stream))


def moe_expert_ffn_bwd_act(d: Dims, dy, dout, offsets, w2, ws2, ab, dab, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_bwd_act", ctypes.byref(d), _ptr(dy, "dy", dt, d.R * H),
          _ptr(dout, "dout", dt, d.T * H), _ptr(offsets, "offsets", torch.int32, E + 1),
          _ptr(w2, "w2", dt, E * I * H), _ptr(ws2, "ws2", dt, Ns * I * H),
          _ptr(ab, "ab", dt, d.RA * 2 * I), _ptr(dab, "dab", dt, d.RA * 2 * I), wp, wn,
          _stream(stream))


def moe_expert_ffn_bwd_input(d: Dims, dab, offsets, w1, w3, ws1, ws3, dx_rows, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_bwd_input", ctypes.byref(d), _ptr(dab, "dab", dt, d.RA * 2 * I),
          _ptr(offsets, "offsets", torch.int32, E + 1), _ptr(w1, "w1", dt, E * H * I),
          _ptr(w3, "w3", dt, E * H * I), _ptr(ws1, "ws1", dt, Ns * H * I),
          _ptr(ws3, "ws3", dt, Ns * H * I), _ptr(dx_rows, "dx_rows", dt, d.RA * H), wp, wn,
          _stream(stream))


def moe_expert_ffn_bwd_weight_gate_up(d: Dims, x_perm, x, dab, offsets, dw1, dw3, dws1, dws3, ws,
                                      stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    f32 = torch.float32
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_bwd_weight_gate_up", ctypes.byref(d), _ptr(x_perm, "x_perm", dt, d.R * H),
          _ptr(x, "x", dt, d.T * H), _ptr(dab, "dab", dt, d.RA * 2 * I),
          _ptr(offsets, "offsets", torch.int32, E + 1), _ptr(dw1, "dw1", f32, E * H * I),
          _ptr(dw3, "dw3", f32, E * H * I), _ptr(dws1, "dws1", f32, Ns * H * I),
          _ptr(dws3, "dws3", f32, Ns * H * I), wp, wn, _stream(stream))


def moe_expert_ffn_bwd_weight_down(d: Dims, h, dy, dout, offsets, dw2, dws2, ws, stream=None):
    dt, H, I, E, Ns = d.torch_dtype, d.H, d.I, d.E, d.n_shared
    f32 = torch.float32
    wp, wn = _ws(ws)
    _call("moe_expert_ffn_bwd_weight_down", ctypes.byref(d), _ptr(h, "h", dt, d.RA * I),
          _ptr(dy, "dy", dt, d.R * H), _ptr(dout, "dout", dt, d.T * H),
          _ptr(offsets, "offsets", torch.int32, E + 1), _ptr(dw2, "dw2", f32, E * I * H),
          _ptr(dws2, "dws2", f32, Ns * I * H), wp, wn, _stream(stream))


def moe_dispatch_bwd(d: Dims, dx_rows, slot, dx, stream=None):
    dt = d.torch_dtype
    _call("moe_dispatch_bwd", ctypes.byref(d), _ptr(dx_rows, "dx_rows", dt, d.RA * d.H),
          _ptr(slot, "slot", torch.int32, d.T * d.K), _ptr(dx, "dx", dt, d.T * d.H), _stream(stream))


def moe_route_bwd(d: Dims, dtopk_w, topk_w, topk_idx, dlogits, stream=None):
    f32 = torch.float32
    _call("moe_route_bwd", ctypes.byref(d), _ptr(dtopk_w, "dtopk_w", f32, d.T * d.K),
          _ptr(topk_w, "topk_w", f32, d.T * d.K), _ptr(topk_idx, "topk_idx", torch.int32, d.T * d.K),
          _ptr(dlogits, "dlogits", f32, d.T * d.E), _stream(stream))


# ---------------------------------------------------------------- a few tokens, 4-bit weights

def moe_decode_workspace_bytes(d: Dims) -> int:
    return int(load().moe_decode_workspace_bytes(ctypes.byref(d)))


def _launch(name, stream, head, tensors, tail):
    """The call with the tensors' pointers between `head` and `tail`; tensors: (tensor, name,
    dtype, elements).  Tensors of another device than the one the work runs on are refused: a
    kernel would read memory that its device may not reach."""
    index = stream.device_index if isinstance(stream, torch.cuda.Stream) else torch.cuda.current_device()
    args = []
    for t, arg_name, dtype, numel in tensors:
        if t is None:
            args.append(None)
        elif (isinstance(t, torch.Tensor) and t.get_device() == index and t.dtype is dtype
              and t.is_contiguous() and t.numel() >= numel):
            args.append(t.data_ptr())
        else:   # says what is wrong
            _ptr(t, arg_name, dtype, numel)
            raise ValueError(f"{arg_name} is on {t.device}, the call runs on cuda:{index}")
    _call(name, *head, *args, *tail, _stream(stream))


def _decode(name, d, dt, n, ns, logits, x, w1, w3, w2, ws1, ws3, ws2, n_tokens, topk_idx, topk_w, out, ws, stream):
    T, H, K, act = d.T, d.H, d.K, d.torch_dtype
    i32, f32 = torch.int32, torch.float32
    _launch(name, stream, (ctypes.byref(d),),
            ((logits, "logits", f32, T * d.E), (x, "x", act, T * H), (w1, "w1", dt, n), (w3, "w3", dt, n),
             (w2, "w2", dt, n), (ws1, "ws1", dt, ns), (ws3, "ws3", dt, ns), (ws2, "ws2", dt, ns),
             (n_tokens, "n_tokens", i32, 1), (topk_idx, "topk_idx", i32, T * K), (topk_w, "topk_w", f32, T * K),
             (out, "out", act, T * H), (ws, "ws", torch.uint8, 0)), (0 if ws is None else ws.numel(),))


def moe_decode(d: Dims, logits, x, w1, w3, w2, ws1, ws3, ws2, n_tokens, topk_idx, topk_w, out, ws,
               stream=None):
    n, ns = d.E * d.H * d.I, d.n_shared * d.H * d.I
    _decode("moe_decode", d, d.torch_dtype, n, ns, logits, x, w1, w3, w2, ws1, ws3, ws2, n_tokens, topk_idx,
            topk_w, out, ws, stream)


def moe_decode_mx(d: Dims, logits, x, w1, w3, w2, ws1, ws3, ws2, n_tokens, topk_idx, topk_w, out, ws,
                  stream=None):
    """moe_decode on packed weights: uint8 tensors of moe_mx_bytes, as moe_mx_quantize writes them."""
    n, ns = _mx_numel(d.E, d.H, d.I), _mx_numel(d.n_shared, d.H, d.I)
    _decode("moe_decode_mx", d, torch.uint8, n, ns, logits, x, w1, w3, w2, ws1, ws3, ws2, n_tokens, topk_idx,
            topk_w, out, ws, stream)


def _mx_numel(G, K, N):
    return G * K * N // 32 * 17


def _fits_int32(v) -> bool:
    return -2 ** 31 <= v < 2 ** 31


def moe_mx_bytes(G: int, K: int, N: int) -> int:
    # ctypes would drop the bits above 32
    return int(load().moe_mx_bytes(G, K, N)) if _fits_int32(G) and _fits_int32(K) and _fits_int32(N) else 0


def _check_mx_sizes(G, K, N):
    """The C call must see the sizes that the tensors are held against: ctypes drops bits above 32."""
    for name, v in (("G", G), ("K", K), ("N", N)):
        if not _fits_int32(v):
            raise ValueError(f"{name} must fit into 32 bits (got {v})")


def _mx_dtype(w):
    """MOE_F32 or MOE_BF16 of a weight tensor, and its torch type (None: bf16, the call reports the NULL)."""
    if w is None:
        return BF16, None
    if not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor or None")
    for code, dt in _TORCH_DTYPE.items():
        if w.dtype is dt:
            return code, dt
    raise TypeError(f"w must be {torch.float32} or {torch.bfloat16} (got {w.dtype})")


def moe_mx_quantize(G: int, K: int, N: int, w, mx, stream=None):
    _check_mx_sizes(G, K, N)
    code, dt = _mx_dtype(w)
    _launch("moe_mx_quantize", stream, (G, K, N, code),
            ((w, "w", dt, G * K * N), (mx, "mx", torch.uint8, _mx_numel(G, K, N))), ())


def moe_mx_dequantize(G: int, K: int, N: int, mx, w, stream=None):
    _check_mx_sizes(G, K, N)
    code, dt = _mx_dtype(w)
    _launch("moe_mx_dequantize", stream, (G, K, N, code),
            ((mx, "mx", torch.uint8, _mx_numel(G, K, N)), (w, "w", dt, G * K * N)), ())


# ---------------------------------------------------------------- router losses

def moe_balance_workspace_bytes(d: Dims, seq_len: int) -> int:
    return int(load().moe_balance_workspace_bytes(ctypes.byref(d), seq_len)) if _fits_int32(seq_len) else 0


def _sequences(d, seq_len):
    """Number of sequences; seq_len as the C call must see it (ctypes drops bits above 32)."""
    if not _fits_int32(seq_len):
        raise ValueError(f"seq_len must fit into 32 bits (got {seq_len})")
    return -(-d.T // seq_len) if seq_len > 0 else 0      # the call refuses seq_len < 1


def _numel(ws):
    return ws.numel() if isinstance(ws, torch.Tensor) else 0


def _mask(mask):
    """A bool mask's bytes are 0 and 1."""
    return mask.view(torch.uint8) if isinstance(mask, torch.Tensor) and mask.dtype is torch.bool else mask


def moe_balance(d: Dims, seq_len: int, logits, topk_idx, mask, counts, tokens, probs, loss, ws, stream=None):
    """mask: uint8 or bool [T], or None."""
    S, f32, i32 = _sequences(d, seq_len), torch.float32, torch.int32
    _launch("moe_balance", stream, (ctypes.byref(d), seq_len),
            ((logits, "logits", f32, d.T * d.E), (topk_idx, "topk_idx", i32, d.T * d.K),
             (_mask(mask), "mask", torch.uint8, d.T), (counts, "counts", i32, S * d.E), (tokens, "tokens", i32, S + 2),
             (probs, "probs", f32, S * d.E), (loss, "loss", f32, 2), (ws, "ws", torch.uint8, 0)),
            (_numel(ws),))


def moe_balance_bwd(d: Dims, seq_len: int, logits, mask, counts, tokens, dloss, dtopk_w, topk_w, topk_idx, dlogits,
                    stream=None):
    S, f32, i32 = _sequences(d, seq_len), torch.float32, torch.int32
    _launch("moe_balance_bwd", stream, (ctypes.byref(d), seq_len),
            ((logits, "logits", f32, d.T * d.E), (_mask(mask), "mask", torch.uint8, d.T),
             (counts, "counts", i32, S * d.E), (tokens, "tokens", i32, S + 2), (dloss, "dloss", f32, 2),
             (dtopk_w, "dtopk_w", f32, d.T * d.K), (topk_w, "topk_w", f32, d.T * d.K),
             (topk_idx, "topk_idx", i32, d.T * d.K), (dlogits, "dlogits", f32, d.T * d.E)), ())


# ---------------------------------------------------------------- update by Newton-Schulz products

EXACT = 16   # MOE_EXACT
NEWTON_COEF = ((3.4445, -4.7750, 2.0315),) * 5
_NEWTON_MAX_STEPS = 16


class Newton(ctypes.Structure):
    """moe_newton: a, b, c of each step."""
    _fields_ = [("steps", ctypes.c_int32), ("coef", (ctypes.c_float * 3) * _NEWTON_MAX_STEPS)]

    def __init__(self, coef=NEWTON_COEF):
        super().__init__()
        if not 1 <= len(coef) <= _NEWTON_MAX_STEPS:
            raise ValueError(f"1 to {_NEWTON_MAX_STEPS} steps (got {len(coef)})")
        self.steps = len(coef)
        for k, abc in enumerate(coef):
            a, b, c = abc
            self.coef[k][0], self.coef[k][1], self.coef[k][2] = a, b, c


class MuonParams(ctypes.Structure):
    """moe_muon_params."""
    _fields_ = [("lr", ctypes.c_float), ("momentum", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("scale", ctypes.c_float), ("nesterov", ctypes.c_int32)]


_SIGS.update({
    "moe_balance_workspace_bytes": (ctypes.c_size_t, [_D, ctypes.c_int]),
    "moe_balance": (ctypes.c_int, [_D, ctypes.c_int] + [_P] * 8 + [ctypes.c_size_t, _P]),
    "moe_balance_bwd": (ctypes.c_int, [_D, ctypes.c_int] + [_P] * 10),
    "moe_muon_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 4),
    "moe_orthogonalize": (ctypes.c_int, [ctypes.c_int] * 4 + [ctypes.POINTER(Newton)] + [_P] * 3 + [ctypes.c_size_t, _P]),
    "moe_muon": (ctypes.c_int, [ctypes.c_int] * 4 + [ctypes.POINTER(Newton), ctypes.POINTER(MuonParams)] + [_P] * 6 +
                 [ctypes.c_size_t, _P]),
})


def moe_muon_workspace_bytes(G: int, R: int, C: int, dtype: int) -> int:
    return int(load().moe_muon_workspace_bytes(G, R, C, dtype)) if all(map(_fits_int32, (G, R, C))) else 0


def _check_stack(G, R, C):
    for name, v in (("G", G), ("R", R), ("C", C)):
        if not _fits_int32(v):
            raise ValueError(f"{name} must fit into 32 bits (got {v})")


def _newton(coef):
    return None if coef is None else ctypes.byref(Newton(coef))


def moe_orthogonalize(G: int, R: int, C: int, g, out, ws, coef=None, stream=None, exact=False):
    """g [G, R, C] float32 -> out [G, R, C], float32 or bf16.  bf16 stands for products of 11-bit factors, too,
    unless exact (EXACT in the workspace's dtype).  coef: (a, b, c) of each step, or None: NEWTON_COEF."""
    _check_stack(G, R, C)
    code, dt = _stack_dtype(out, "out")
    if exact:
        code |= EXACT
    n = G * R * C
    _launch("moe_orthogonalize", stream, (G, R, C, code, _newton(coef)),
            ((g, "g", torch.float32, n), (out, "out", dt, n), (ws, "ws", torch.uint8, 0)),
            (_numel(ws),))


def _stack_dtype(t, name):
    if t is None:
        return F32, None                     # the call reports the NULL
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor or None")
    for code, dt in _TORCH_DTYPE.items():
        if t.dtype is dt:
            return code, dt
    raise TypeError(f"{name} must be {torch.float32} or {torch.bfloat16} (got {t.dtype})")


def moe_muon(G: int, R: int, C: int, grad, mom, master, w, ws, *, lr, momentum=0.95, weight_decay=0.0, scale=1.0,
             nesterov=True, coef=None, stream=None, exact=False):
    """One step on a stack of weights, in place: mom and master [G, R, C] float32, w their bf16 copy or
    None (float32 weights: the products are as exact as float32's; with w, only if exact, with EXACT in the
    workspace's dtype).  lr: a number, or a float32 tensor of one element on the GPU."""
    _check_stack(G, R, C)
    if w is not None and not isinstance(w, torch.Tensor):
        raise TypeError("w must be a torch.Tensor or None")
    n, f32 = G * R * C, torch.float32
    on_device = isinstance(lr, torch.Tensor)
    p = MuonParams(0.0 if on_device else lr, momentum, weight_decay, scale, int(bool(nesterov)))
    _launch("moe_muon", stream, (G, R, C, (F32 if w is None else BF16) | (EXACT if exact else 0), _newton(coef),
                                ctypes.byref(p)),
            ((lr if on_device else None, "lr", f32, 1), (grad, "grad", f32, n), (mom, "mom", f32, n),
             (master, "master", f32, n), (w, "w", torch.bfloat16, n), (ws, "ws", torch.uint8, 0)),
            (_numel(ws),))
