"""Thin ctypes binding of libspear (the C ABI declared in include/spear.h).

Argument marshalling only: tensors are passed as device pointers together with
torch's current HIP stream; every step of the layer runs in the library's
kernels.  The library is opened on first use; if it has not been built the
call raises (there is no fallback path).
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspear.so")

SPEAR_OK = 0
CODES_S4 = 0
CODES_U4 = 1
OUT_BF16 = 0
OUT_F32 = 1
PATH_AUTO = 0
PATH_DECODE = 1
PATH_PREFILL = 2
PATH_DECODE_2PASS = 3
PATH_PREFILL_LARGE = 4
MAX_RANK = 256
MAX_GATE_HIDDEN = 64
ABI_VERSION = 2
ACT_NONE = 0
ACT_RELU = 1
ACT_SILU = 2
ACT_GELU = 3
ACT_GELU_TANH = 4
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
MAX_EXPERTS = 512
MAX_TOPK = 32
MAX_GROUPS = 64
KV4_COUNTER_BYTES = 163840
ROPE_HALF = 0
ROPE_PAIRS = 1
ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_BASE = 2
ROPE_PARTS = 3
E_NULL = -1
E_SHAPE = -2
E_ARG = -4

EXPORTS = ("spear_pack_w4", "spear_gate", "spear_w4_linear_workspace_size",
           "spear_workspace_init", "spear_w4_linear", "spear_w4_linear_path",
           "spear_w4_linear_noalloc", "spear_w4_linear_semifused", "spear_w4_linear_epilogue",
           "spear_route_workspace_size", "spear_route", "spear_w4_experts_workspace_size",
           "spear_w4_experts", "spear_kv4_plan", "spear_rope_frequencies", "spear_rope",
           "spear_rope_kv4_write", "spear_kv4_read", "spear_kv4_attention_workspace_size",
           "spear_kv4_attention",
           "spear_set_wait_limit", "spear_workspace_timeouts", "spear_stream_read",
           "spear_slo_predict", "spear_slo_pick_chunk", "spear_status_string",
           "spear_abi_version")


class SpearError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: status {status} ({msg})")
        self.status = status


class _W4(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class _EC(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("w_gate", ctypes.c_void_p),
                ("b", ctypes.c_float), ("tau", ctypes.c_float), ("hard", ctypes.c_int32),
                ("r", ctypes.c_int32), ("g_out", ctypes.c_void_p), ("idx_out", ctypes.c_void_p),
                ("n_active_out", ctypes.c_void_p), ("gate_h", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("gate_w1", ctypes.c_void_p),
                ("gate_c1", ctypes.c_void_p), ("gate_w2", ctypes.c_void_p),
                ("gate_c2", ctypes.c_void_p)]


class _Epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("act", ctypes.c_int32),
                ("glu", ctypes.c_int32)]


class _Router(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("E", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("score", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_best", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Experts(ctypes.Structure):
    _fields_ = [("up", ctypes.c_void_p), ("up_scales", ctypes.c_void_p),
                ("up_zeros", ctypes.c_void_p), ("up_bias", ctypes.c_void_p),
                ("down", ctypes.c_void_p), ("down_scales", ctypes.c_void_p),
                ("down_zeros", ctypes.c_void_p), ("down_bias", ctypes.c_void_p),
                ("K", ctypes.c_int64), ("I", ctypes.c_int64), ("N", ctypes.c_int64),
                ("E", ctypes.c_int32), ("act", ctypes.c_int32), ("glu", ctypes.c_int32)]


class _KV4(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("heads", ctypes.c_int32), ("D", ctypes.c_int32),
                ("P", ctypes.c_int32)]


class _Step(ctypes.Structure):
    _fields_ = [("q_start", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("n_left", ctypes.c_void_p), ("status", ctypes.c_void_p)]


class _Rotation(ctypes.Structure):
    _fields_ = [("freqs", ctypes.c_void_p), ("scale", ctypes.c_double), ("rot", ctypes.c_int32),
                ("layout", ctypes.c_int32)]


class _LUT(ctypes.Structure):
    _fields_ = [("npoints", ctypes.c_int32), ("tokens", ctypes.c_void_p),
                ("nkinds", ctypes.c_int32), ("us", ctypes.c_void_p), ("count", ctypes.c_void_p),
                ("overhead_us", ctypes.c_float)]


_lib = None


def load():
    """Open libspear.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libspear.so not found at {LIB_PATH}; build it with "
                           "quantized_gemm_w4a16_amd.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.spear_pack_w4.argtypes = [P, i32, i64, i64, P, P, P]
    lib.spear_gate.argtypes = [P, i64, i64, P, ctypes.c_float, ctypes.c_float, i32, P, P, P, P]
    lib.spear_w4_linear_workspace_size.argtypes = [i64, i64, i64, i32]
    lib.spear_w4_linear_workspace_size.restype = ctypes.c_size_t
    lib.spear_workspace_init.argtypes = [P, ctypes.c_size_t, P]
    lin = [P, i64, ctypes.POINTER(_W4), ctypes.POINTER(_EC), P, i32, P, ctypes.c_size_t]
    lib.spear_w4_linear.argtypes = lin + [P]
    lib.spear_w4_linear_path.argtypes = lin + [i32, P]
    lib.spear_w4_linear_noalloc.argtypes = [P, i64, ctypes.POINTER(_W4), ctypes.POINTER(_EC), P,
                                            i32, i32, P]
    lib.spear_w4_linear_semifused.argtypes = [P, i64, ctypes.POINTER(_W4), ctypes.POINTER(_EC), P,
                                              P, ctypes.c_size_t, P, P, P, P]
    # (structs as pointers to their bytes)
    lib.spear_w4_linear_epilogue.argtypes = [P, i64, P, P, P, P, i32, P, ctypes.c_size_t, i32, P]
    lib.spear_route_workspace_size.argtypes = [i64, i32]
    lib.spear_route_workspace_size.restype = ctypes.c_size_t
    lib.spear_route.argtypes = [P, i64, i64, P, P, P, P, ctypes.c_size_t, P]
    lib.spear_w4_experts_workspace_size.argtypes = [i64, i32, i32, i64, i64]
    lib.spear_w4_experts_workspace_size.restype = ctypes.c_size_t
    lib.spear_w4_experts.argtypes = [P, i64, P, P, P, i32, P, P, P, ctypes.c_size_t, P]
    f64 = ctypes.c_double
    lib.spear_kv4_plan.argtypes = [P, P, i32, P, i64, P, i64, P, i64, i32, P, P]
    lib.spear_rope_frequencies.argtypes = [i32, f64, i32, f64, f64, f64, f64, P]
    lib.spear_rope.argtypes = [P, i64, i64, i32, i32, P, P, P, i64, P]
    lib.spear_rope_kv4_write.argtypes = [P, i64, P, i64, P, i64, i64, i32, P, P, P, P, P, i64, P]
    lib.spear_kv4_read.argtypes = [P, P, i64, P, P, P]
    lib.spear_kv4_attention_workspace_size.argtypes = [i64, i32, i64, i32, i32, i32, i64, i32]
    lib.spear_kv4_attention_workspace_size.restype = ctypes.c_size_t
    lib.spear_kv4_attention.argtypes = [P, i64, i64, i32, P, P, i64, P, P, i32, i64, ctypes.c_float,
                                        i32, P, P, P, ctypes.c_size_t, P]
    lib.spear_set_wait_limit.argtypes = [ctypes.c_uint32]
    lib.spear_set_wait_limit.restype = None
    lib.spear_workspace_timeouts.argtypes = [P, ctypes.POINTER(i32), P]
    lib.spear_stream_read.argtypes = [P, ctypes.c_size_t, P, P]
    lib.spear_slo_predict.argtypes = [ctypes.POINTER(_LUT), i32, ctypes.POINTER(ctypes.c_float)]
    lib.spear_slo_pick_chunk.argtypes = [ctypes.POINTER(_LUT), i32, i32, i32, ctypes.c_float,
                                         ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_float)]
    lib.spear_status_string.argtypes = [i32]
    lib.spear_status_string.restype = ctypes.c_char_p
    lib.spear_abi_version.restype = i32
    for name in ("spear_pack_w4", "spear_gate", "spear_workspace_init", "spear_w4_linear",
                 "spear_w4_linear_path", "spear_w4_linear_noalloc", "spear_w4_linear_semifused",
                 "spear_w4_linear_epilogue", "spear_route", "spear_w4_experts",
                 "spear_kv4_plan", "spear_rope_frequencies", "spear_rope", "spear_rope_kv4_write",
                 "spear_kv4_read", "spear_kv4_attention", "spear_workspace_timeouts",
                 "spear_stream_read", "spear_slo_predict", "spear_slo_pick_chunk"):
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def _check(fn: str, st: int):
    if st != SPEAR_OK:
        raise SpearError(fn, st, load().spear_status_string(st).decode())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


@dataclass
class W4:
    """Packed weights on the device: packed [N][K/2] uint8, scales [N] fp32,
    zeros [N] uint8 or None (zero point 8)."""
    packed: torch.Tensor
    scales: torch.Tensor
    zeros: Optional[torch.Tensor]
    N: int
    K: int

    def _c(self):
        return _W4(_ptr(self.packed), _ptr(self.scales), _ptr(self.zeros), self.N, self.K)


@dataclass
class EC:
    """Error compensator on the device: A [r][K], B [N][r], w_gate [K] as bf16
    (torch.bfloat16 or int16 bit tensors), gate bias b, threshold tau, hard flag.
    Optional outputs g_out [M] fp32, idx_out [M] int32, n_active_out [1] int32.
    Optional vector gate (fp32): gate_w1 [h][r], gate_c1 [h], gate_w2 [r][h],
    gate_c2 [r] and its scale alpha."""
    A: torch.Tensor
    B: torch.Tensor
    w_gate: torch.Tensor
    b: float = 0.0
    tau: float = 0.0
    hard: int = 0
    g_out: Optional[torch.Tensor] = None
    idx_out: Optional[torch.Tensor] = None
    n_active_out: Optional[torch.Tensor] = None
    gate_w1: Optional[torch.Tensor] = None
    gate_c1: Optional[torch.Tensor] = None
    gate_w2: Optional[torch.Tensor] = None
    gate_c2: Optional[torch.Tensor] = None
    alpha: float = 1.0

    @property
    def r(self) -> int:
        return int(self.A.shape[0])

    @property
    def gate_h(self) -> int:
        return 0 if self.gate_w1 is None else int(self.gate_w1.shape[0])

    def _packed(self) -> bytes:
        return _PACK_EC(_at(self.A), _at(self.B), _at(self.w_gate), self.b, self.tau, self.hard,
                        self.r, _at(self.g_out), _at(self.idx_out), _at(self.n_active_out),
                        self.gate_h, self.alpha, _at(self.gate_w1), _at(self.gate_c1),
                        _at(self.gate_w2), _at(self.gate_c2))

    def _c(self):
        return _EC(_ptr(self.A), _ptr(self.B), _ptr(self.w_gate), float(self.b), float(self.tau),
                   int(self.hard), self.r, _ptr(self.g_out), _ptr(self.idx_out),
                   _ptr(self.n_active_out), self.gate_h, float(self.alpha), _ptr(self.gate_w1),
                   _ptr(self.gate_c1), _ptr(self.gate_w2), _ptr(self.gate_c2))


def spear_abi_version() -> int:
    return int(load().spear_abi_version())


def spear_status_string(st: int) -> str:
    return load().spear_status_string(st).decode()


def spear_pack_w4(codes: torch.Tensor, kind: int, packed: Optional[torch.Tensor] = None,
                  bad_codes: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    N, K = codes.shape
    if packed is None:
        packed = torch.empty((N, K // 2), dtype=torch.uint8, device=codes.device)
    _check("spear_pack_w4", load().spear_pack_w4(_ptr(codes), kind, N, K, _ptr(packed),
                                                 _ptr(bad_codes), _stream(stream)))
    return packed


def spear_gate(x: torch.Tensor, w_gate: torch.Tensor, b: float, tau: float, hard: int,
               g=None, idx=None, n_active=None, stream=None):
    M, K = x.shape
    dev = x.device
    g = torch.empty(M, dtype=torch.float32, device=dev) if g is None else g
    idx = torch.empty(max(M, 1), dtype=torch.int32, device=dev) if idx is None else idx
    n_active = torch.empty(1, dtype=torch.int32, device=dev) if n_active is None else n_active
    _check("spear_gate", load().spear_gate(_ptr(x), M, K, _ptr(w_gate), float(b), float(tau),
                                           int(hard), _ptr(g), _ptr(idx), _ptr(n_active),
                                           _stream(stream)))
    return g, idx, n_active


def spear_w4_linear_workspace_size(M: int, N: int, K: int, r: int) -> int:
    return int(load().spear_w4_linear_workspace_size(M, N, K, r))


def spear_workspace_init(ws: torch.Tensor, stream=None):
    _check("spear_workspace_init", load().spear_workspace_init(_ptr(ws), ws.numel(),
                                                               _stream(stream)))


def new_workspace(M: int, N: int, K: int, r: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace tensor of the required size (torch allocation)."""
    n = max(spear_w4_linear_workspace_size(M, N, K, r), 256)
    return torch.zeros(n, dtype=torch.uint8, device=device)


def spear_w4_linear(x: torch.Tensor, w: W4, ec: Optional[EC] = None,
                    y: Optional[torch.Tensor] = None, out_dtype: int = OUT_F32,
                    workspace: Optional[torch.Tensor] = None, path: int = PATH_AUTO,
                    stream=None) -> torch.Tensor:
    M = int(x.shape[0])
    if y is None:
        dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
        y = torch.empty((M, w.N), dtype=dt, device=x.device)
    if workspace is None:
        workspace = new_workspace(M, w.N, w.K, ec.r if ec is not None else 0, x.device)
    wc = w._c()
    ecc = ec._c() if ec is not None else None
    st = load().spear_w4_linear_path(_ptr(x), M, ctypes.byref(wc),
                                     ctypes.byref(ecc) if ecc is not None else None,
                                     _ptr(y), out_dtype, _ptr(workspace), workspace.numel(),
                                     path, _stream(stream))
    _check("spear_w4_linear", st)
    return y


class SemiFused:
    """The second stream and the two events of the semi-fused prefill (torch
    objects; the events are recorded once so that their HIP handles exist)."""

    def __init__(self, device="cuda"):
        self.aux = torch.cuda.Stream(device=device)
        self.ev_fork = torch.cuda.Event()
        self.ev_join = torch.cuda.Event()
        self.ev_fork.record(self.aux)
        self.ev_join.record(self.aux)
        self.aux.synchronize()


def spear_w4_linear_semifused(x: torch.Tensor, w: W4, ec: Optional[EC], sf: SemiFused,
                              y: Optional[torch.Tensor] = None,
                              workspace: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """The prefill layer with the EC as a separate kernel on sf.aux (fp32 y)."""
    M = int(x.shape[0])
    if y is None:
        y = torch.empty((M, w.N), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = new_workspace(M, w.N, w.K, ec.r if ec is not None else 0, x.device)
    wc = w._c()
    ecc = ec._c() if ec is not None else None
    st = load().spear_w4_linear_semifused(_ptr(x), M, ctypes.byref(wc),
                                          ctypes.byref(ecc) if ecc is not None else None,
                                          _ptr(y), _ptr(workspace), workspace.numel(),
                                          _stream(stream), sf.aux.cuda_stream,
                                          sf.ev_fork.cuda_event, sf.ev_join.cuda_event)
    _check("spear_w4_linear_semifused", st)
    return y


NOALLOC_MAX_WORKSPACE = 48 << 20


def spear_w4_linear_noalloc(x: torch.Tensor, w: W4, ec: Optional[EC] = None,
                            y: Optional[torch.Tensor] = None, out_dtype: int = OUT_F32,
                            path: int = PATH_AUTO, stream=None) -> torch.Tensor:
    """The layer through the allocation-free entry point (the library's own
    scratch stands in for the workspace).  y must be given by callers that
    cannot allocate; it is allocated here only for convenience when None."""
    M = int(x.shape[0])
    if y is None:
        dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
        y = torch.empty((M, w.N), dtype=dt, device=x.device)
    wc = w._c()
    ecc = ec._c() if ec is not None else None
    st = load().spear_w4_linear_noalloc(_ptr(x), M, ctypes.byref(wc),
                                        ctypes.byref(ecc) if ecc is not None else None,
                                        _ptr(y), out_dtype, path, _stream(stream))
    _check("spear_w4_linear_noalloc", st)
    return y


def _bad(fn: str, status: int, what: str):
    raise SpearError(fn, status, what)


def _want(fn: str, name: str, t, dtypes, shape, device):
    """A tensor argument: its element type, shape, device, and no gaps between
    its elements (the library takes bare pointers and cannot see any of it)."""
    if t.dtype in dtypes and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype not in dtypes:
        _bad(fn, E_ARG, f"{name} has type {t.dtype}")
    if t.shape != shape:
        _bad(fn, E_SHAPE, f"{name} has shape {tuple(t.shape)}, not {shape}")
    if t.device != device:
        _bad(fn, E_ARG, f"{name} is on {t.device}, not {device}")
    _bad(fn, E_ARG, f"{name} is not contiguous")


def _want_workspace(fn: str, t, device):
    if t.dtype != torch.uint8 or t.device != device or not t.is_contiguous():
        _bad(fn, E_ARG, f"workspace has to be a contiguous uint8 tensor on {device}")


def _want_flat(fn: str, name: str, t, dtypes, n: int, device):
    """The same for a tensor that is taken by its number of elements."""
    if t.dtype in dtypes and t.numel() == n and t.device == device and t.is_contiguous():
        return
    if t.numel() != n:
        _bad(fn, E_SHAPE, f"{name} has {t.numel()} elements, not {n}")
    _want(fn, name, t, dtypes, t.shape, device)


def _want_layer(fn: str, w: W4, ec: Optional[EC], M: int, device):
    """The weights and the compensator of a layer call."""
    N, K = w.N, w.K
    _want_flat(fn, "packed", w.packed, _U8, N * K // 2, device)
    _want_flat(fn, "scales", w.scales, _F32, N, device)
    if w.zeros is not None:
        _want_flat(fn, "zeros", w.zeros, _U8, N, device)
    if ec is None:
        return
    r = ec.r
    _want_flat(fn, "A", ec.A, _BF16, r * K, device)
    _want_flat(fn, "B", ec.B, _BF16, N * r, device)
    _want_flat(fn, "w_gate", ec.w_gate, _BF16, K, device)
    for name, dtypes, n in (("g_out", _F32, M), ("idx_out", _I32, M), ("n_active_out", _I32, 1)):
        t = getattr(ec, name)
        if t is not None and not (t.dtype in dtypes and t.numel() >= n and t.device == device and
                                  t.is_contiguous()):
            _want_flat(fn, name, t, dtypes, n, device)
    if ec.gate_w1 is not None:
        h = ec.gate_h
        for name, n in (("gate_w1", h * r), ("gate_c1", h), ("gate_w2", r * h), ("gate_c2", r)):
            t = getattr(ec, name)
            if t is None:
                _bad(fn, E_NULL, f"{name} is missing")
            _want_flat(fn, name, t, _F32, n, device)


_BF16 = (torch.bfloat16, torch.int16)     # raw bit tensors are taken too
_F32 = (torch.float32,)
_I32 = (torch.int32,)
_I64 = (torch.int64,)
_U8 = (torch.uint8,)


class _On:
    """The device and stream of one call: the arguments' device is current, and
    what the call allocates belongs to its stream."""

    def __init__(self, device, stream):
        self.contexts = [torch.cuda.device(device)]
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                # the null stream has no external handle
                stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                          else torch.cuda.default_stream(device))
            self.contexts.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _on(fn: str, device, stream, call):
    """call(stream handle) with the device and stream current.  Small layers take
    10 us on the GPU, so nothing is switched that already is as it should be."""
    index = device.index                                  # None on the CPU
    if stream is None and index is not None and index == _current_device():
        return call(_current_stream(index))
    if device.type != "cuda":
        _bad(fn, E_ARG, f"tensors are on {device}, not on a GPU")
    with _On(device, stream):
        return call(_current_stream(device.index))


def _public_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# torch's own raw queries, where it has them (0.1 us for 1.2, 0.05 for 0.25)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

# The C structs as packed bytes, a fifth of the time of filling ctypes
# structures field by field.
_PACK_W4 = struct.Struct("@PPPqq").pack
_PACK_EC = struct.Struct("@PPPffiiPPPifPPPP").pack
_PACK_EPILOGUE = struct.Struct("@PPii").pack


def _at(t) -> int:
    return 0 if t is None else t.data_ptr()


@dataclass
class Epilogue:
    """What follows the layer: bias [N] fp32, act (ACT_*), glu (channels 2i and
    2i + 1 of the weights are gate and up of output channel i), residual [M][N]
    ([M][N/2] with glu) of the output's type, added last; it may be y itself."""
    bias: Optional[torch.Tensor] = None
    act: int = ACT_NONE
    glu: bool = False
    residual: Optional[torch.Tensor] = None


def spear_w4_linear_epilogue(x: torch.Tensor, w: W4, ep: Epilogue, ec: Optional[EC] = None,
                             y: Optional[torch.Tensor] = None, out_dtype: int = OUT_F32,
                             workspace: Optional[torch.Tensor] = None, path: int = PATH_AUTO,
                             stream=None) -> torch.Tensor:
    """The layer with bias, activation (plain or gated pair) and residual in
    its kernels' epilogue: y [M][N], or [M][N/2] with ep.glu."""
    fn = "spear_w4_linear_epilogue"
    dev = x.device
    M, NO = x.shape[0], w.N // 2 if ep.glu else w.N
    dt = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
    _want(fn, "x", x, _BF16, (M, w.K), dev)
    if ep.bias is not None:
        _want(fn, "bias", ep.bias, _F32, (w.N,), dev)
    if ep.residual is not None:
        _want(fn, "residual", ep.residual, (dt,), (M, NO), dev)
    if y is not None:
        _want(fn, "y", y, (dt,), (M, NO), dev)
    if workspace is not None:
        _want_workspace(fn, workspace, dev)
    _want_layer(fn, w, ec, M, dev)

    def call(s):
        nonlocal y, workspace
        if y is None:
            y = torch.empty((M, NO), dtype=dt, device=dev)
        if workspace is None:
            workspace = new_workspace(M, w.N, w.K, ec.r if ec is not None else 0, dev)
        return load().spear_w4_linear_epilogue(
            x.data_ptr(), M, _PACK_W4(_at(w.packed), _at(w.scales), _at(w.zeros), w.N, w.K),
            None if ec is None else ec._packed(),
            _PACK_EPILOGUE(_at(ep.bias), _at(ep.residual), ep.act, ep.glu),
            y.data_ptr(), out_dtype, workspace.data_ptr(), workspace.numel(), path, s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return y


class Router:
    """Router of a mixture of experts: w [E][K] bf16, bias [E] fp32 (for the
    choice alone) or None; topk experts a token out of the topk_group best of
    n_group groups (a group counts the sum of its group_best best choices).
    Made once with the model; the tensors are kept, their contents may change."""

    def __init__(self, w: torch.Tensor, topk: int, score: int = SCORE_SOFTMAX,
                 bias: Optional[torch.Tensor] = None, n_group: int = 1, topk_group: int = 1,
                 group_best: int = 2, renorm: bool = True, scale: float = 1.0):
        E, K = (int(v) for v in w.shape)
        _want("Router", "w", w, _BF16, (E, K), w.device)
        if bias is not None:
            _want("Router", "bias", bias, _F32, (E,), w.device)
        self.w, self.bias, self.E, self.K, self.topk = w, bias, E, K, int(topk)
        self._s = bytes(_Router(_ptr(w), _ptr(bias), E, int(topk), int(score), int(n_group),
                                int(topk_group), int(group_best), int(bool(renorm)), float(scale)))


def spear_route_workspace_size(M: int, E: int) -> int:
    return int(load().spear_route_workspace_size(M, E))


def new_route_workspace(M: int, router: Router) -> torch.Tensor:
    """A workspace for spear_route over up to M tokens (torch allocation)."""
    return torch.empty(max(spear_route_workspace_size(M, router.E), 256), dtype=torch.uint8,
                       device=router.w.device)


def spear_route(x: torch.Tensor, router: Router, weights: Optional[torch.Tensor] = None,
                ids: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None):
    """-> (weights [M][topk] fp32, ids [M][topk] int32, best first, -1 where no
    expert is left)."""
    fn = "spear_route"
    dev = x.device
    M = x.shape[0]
    shape = (M, router.topk)
    _want(fn, "x", x, _BF16, (M, router.K), router.w.device)
    if weights is not None:
        _want(fn, "weights", weights, _F32, shape, dev)
    if ids is not None:
        _want(fn, "ids", ids, _I32, shape, dev)
    if workspace is not None:
        _want_workspace(fn, workspace, dev)

    def call(s):
        nonlocal weights, ids, workspace
        if weights is None:
            weights = torch.empty(shape, dtype=torch.float32, device=dev)
        if ids is None:
            ids = torch.empty(shape, dtype=torch.int32, device=dev)
        if workspace is None:
            workspace = new_route_workspace(M, router)
        return load().spear_route(x.data_ptr(), M, router.K, router._s, weights.data_ptr(),
                                  ids.data_ptr(), workspace.data_ptr(), workspace.numel(), s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return weights, ids


class Experts:
    """The experts' two 4-bit layers, the expert index outermost: up [E][NU][K/2]
    packed codes with scales and zeros [E][NU], down [E][N][I/2] with [E][N]
    (zeros None: zero point 8), optional fp32 biases of the same shapes; NU = 2 I
    with glu (rows 2i and 2i + 1 are gate and up of inner channel i), else I.
    Made once with the model; the tensors are kept, their contents may change."""

    def __init__(self, up, up_scales, up_zeros, down, down_scales, down_zeros, up_bias=None,
                 down_bias=None, act: int = ACT_SILU, glu: bool = True):
        fn = "Experts"
        E, NU, K = int(up.shape[0]), int(up.shape[1]), 2 * int(up.shape[2])
        N, I = int(down.shape[1]), 2 * int(down.shape[2])
        dev = up.device
        if NU != (2 * I if glu else I):
            _bad(fn, E_SHAPE, f"up has {NU} rows for {I} inner channels (glu={bool(glu)})")
        _want(fn, "up", up, _U8, (E, NU, K // 2), dev)
        _want(fn, "down", down, _U8, (E, N, I // 2), dev)
        for name, t, dt, n in (("up_scales", up_scales, _F32, NU), ("up_zeros", up_zeros, _U8, NU),
                               ("up_bias", up_bias, _F32, NU),
                               ("down_scales", down_scales, _F32, N),
                               ("down_zeros", down_zeros, _U8, N),
                               ("down_bias", down_bias, _F32, N)):
            if t is not None:
                _want(fn, name, t, dt, (E, n), dev)
        self.tensors = (up, up_scales, up_zeros, up_bias, down, down_scales, down_zeros, down_bias)
        self.E, self.K, self.I, self.N, self.device = E, K, I, N, dev
        self._s = bytes(_Experts(*(_ptr(t) for t in self.tensors), K, I, N, E, int(act),
                                 int(bool(glu))))


def spear_w4_experts_workspace_size(M: int, topk: int, E: int, I: int, N: int) -> int:
    return int(load().spear_w4_experts_workspace_size(M, topk, E, I, N))


def new_experts_workspace(M: int, topk: int, experts: Experts) -> torch.Tensor:
    """A workspace for spear_w4_experts over up to M tokens (torch allocation)."""
    n = spear_w4_experts_workspace_size(M, topk, experts.E, experts.I, experts.N)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=experts.device)


def spear_w4_experts(x: torch.Tensor, experts: Experts, ids: torch.Tensor, weights: torch.Tensor,
                     residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [M][N] bf16 = residual + the sum over a token's slots of weight times
    expert; ids outside [0, E) add nothing."""
    fn = "spear_w4_experts"
    dev = x.device
    M, topk, N = x.shape[0], ids.shape[1], experts.N
    _want(fn, "x", x, _BF16, (M, experts.K), experts.device)
    _want(fn, "ids", ids, _I32, (M, topk), dev)
    _want(fn, "weights", weights, _F32, (M, topk), dev)
    if residual is not None:
        _want(fn, "residual", residual, _BF16, (M, N), dev)
    if y is not None:
        _want(fn, "y", y, _BF16, (M, N), dev)
    if workspace is not None:
        _want_workspace(fn, workspace, dev)

    def call(s):
        nonlocal y, workspace
        if y is None:
            y = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        if workspace is None:
            workspace = new_experts_workspace(M, topk, experts)
        return load().spear_w4_experts(x.data_ptr(), M, experts._s, ids.data_ptr(),
                                       weights.data_ptr(), topk, _at(residual), y.data_ptr(),
                                       workspace.data_ptr(), workspace.numel(), s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return y


class KV4:
    """A cache of keys and values in 4 bits: codes [pages][heads][P][D/2] and scales
    [pages][heads][D/32][P], uint8, for k and v (the layout is spear.h's).  Made
    once; the tensors are kept, spear_rope_kv4_write fills them."""

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        fn = "KV4"
        if k_codes.dim() != 4:
            _bad(fn, E_SHAPE, f"k_codes has {k_codes.dim()} dimensions, not 4")
        pages, heads, P, half = (int(v) for v in k_codes.shape)
        dev, D = k_codes.device, 2 * half
        for name, t, shape in (("k_codes", k_codes, (pages, heads, P, half)),
                               ("v_codes", v_codes, (pages, heads, P, half)),
                               ("k_scales", k_scales, (pages, heads, D // 32, P)),
                               ("v_scales", v_scales, (pages, heads, D // 32, P))):
            _want(fn, name, t, _U8, shape, dev)
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.pages, self.heads, self.D, self.P, self.device = pages, heads, D, P, dev
        self._s = bytes(_KV4(_ptr(k_codes), _ptr(k_scales), _ptr(v_codes), _ptr(v_scales), pages,
                             heads, D, P))


def new_kv4(pages: int, heads: int, D: int, P: int, device="cuda") -> KV4:
    """An empty cache (torch allocation; its contents are undefined)."""
    def u8(*shape):
        return torch.empty(shape, dtype=torch.uint8, device=device)
    return KV4(u8(pages, heads, P, D // 2), u8(pages, heads, D // 32, P),
               u8(pages, heads, P, D // 2), u8(pages, heads, D // 32, P))


class KV4Plan:
    """What spear_kv4_plan fills: q_start [B + 1], kv_len [B], positions [T] int32,
    slots [T] int64, n_left [1], status [2] int32."""

    def __init__(self, q_start, kv_len, positions, slots, n_left, status):
        fn = "KV4Plan"
        B, T, dev = kv_len.numel(), positions.numel(), kv_len.device
        for name, t, dtypes, n in (("q_start", q_start, _I32, B + 1), ("kv_len", kv_len, _I32, B),
                                   ("positions", positions, _I32, T), ("slots", slots, _I64, T),
                                   ("n_left", n_left, _I32, 1), ("status", status, _I32, 2)):
            _want(fn, name, t, dtypes, (n,), dev)
        self.q_start, self.kv_len, self.positions, self.slots = q_start, kv_len, positions, slots
        self.n_left, self.status, self.B, self.T, self.device = n_left, status, B, T, dev
        self._s = bytes(_Step(*(_ptr(t) for t in (q_start, kv_len, positions, slots, n_left, status))))


def new_kv4_plan(B: int, T: int, device="cuda") -> KV4Plan:
    """The tensors of a plan for B requests and T rows (torch allocation)."""
    def i32(n):
        return torch.empty(n, dtype=torch.int32, device=device)
    return KV4Plan(i32(B + 1), i32(B), i32(T), torch.empty(T, dtype=torch.int64, device=device),
                   i32(1), i32(2))


def spear_kv4_plan(cached: torch.Tensor, fresh: torch.Tensor, table: torch.Tensor,
                   free_pages: torch.Tensor, n_free: torch.Tensor, T: int, P: int,
                   plan: Optional[KV4Plan] = None, stream=None) -> KV4Plan:
    """Block table (updated in place) and slot map of a step whose requests have
    cached [B] tokens in the cache and bring fresh [B] ones, in T rows."""
    fn = "spear_kv4_plan"
    dev, B = cached.device, cached.numel()
    if table.dim() != 2:
        _bad(fn, E_SHAPE, f"table has {table.dim()} dimensions, not 2")
    _want_int32(fn, "P", P)
    width = int(table.shape[1])
    _want(fn, "cached", cached, _I32, (B,), dev)
    _want(fn, "fresh", fresh, _I32, (B,), dev)
    _want(fn, "table", table, _I32, (B, width), dev)
    _want(fn, "free_pages", free_pages, _I32, (free_pages.numel(),), dev)
    _want(fn, "n_free", n_free, _I32, (1,), dev)
    if plan is not None and (plan.B != B or plan.T != T):
        _bad(fn, E_SHAPE, f"the plan is one for {plan.B} requests and {plan.T} rows, not {B} and {T}")
    if plan is not None and plan.device != dev:
        _bad(fn, E_ARG, f"the plan is on {plan.device}, not {dev}")

    def call(s):
        nonlocal plan
        if plan is None:
            plan = new_kv4_plan(B, T, dev)
        return load().spear_kv4_plan(cached.data_ptr(), fresh.data_ptr(), B, table.data_ptr(), width,
                                     free_pages.data_ptr(), free_pages.numel(), n_free.data_ptr(), T,
                                     P, plan._s, s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return plan


def spear_rope_frequencies(rot: int, base: float = 10000.0, kind: int = ROPE_PLAIN,
                           factor: float = 1.0, original: float = 1.0, low: float = 1.0,
                           high: float = 32.0) -> torch.Tensor:
    """The rot / 2 frequencies of a rotation, fp64 on the host; kind (ROPE_PLAIN,
    _LINEAR, _BASE, _PARTS) says how positions are stretched by factor."""
    _want_int32("spear_rope_frequencies", "rot", rot)
    f = torch.empty(max(rot // 2, 1), dtype=torch.float64)
    _check("spear_rope_frequencies",
           load().spear_rope_frequencies(rot, base, kind, factor, original, low, high, _ptr(f)))
    return f


class Rope:
    """Rotary positions: freqs [rot/2] fp64 on the device (the angle of one
    position), layout ROPE_HALF or ROPE_PAIRS, scale the factor of the rotated
    channels (for frequencies by parts, usually 0.1 ln(factor) + 1)."""

    def __init__(self, freqs: torch.Tensor, layout: int = ROPE_HALF, scale: float = 1.0):
        _want("Rope", "freqs", freqs, (torch.float64,), (freqs.numel(),), freqs.device)
        self.freqs, self.layout, self.scale, self.rot = freqs, int(layout), float(scale), 2 * freqs.numel()
        self._s = bytes(_Rotation(_ptr(freqs), self.scale, self.rot, self.layout))


def _want_int32(fn: str, name: str, n: int):
    """ctypes cuts a larger number to 32 bits."""
    if not -0x80000000 <= n <= 0x7FFFFFFF:
        _bad(fn, E_SHAPE, f"{name} is {n}")


def _want_rows(fn: str, name: str, t, shape, device) -> int:
    """A [T][H][D] bf16 tensor whose rows may lie apart (a part of a wider row);
    -> elements from row to row."""
    T, H, D = shape
    if t.shape == shape and t.dtype in _BF16 and t.device == device:
        row, head, channel = t.stride()
        if channel == 1 and (head == D or H == 1):
            return row if T > 1 else H * D
    if t.dtype not in _BF16:
        _bad(fn, E_ARG, f"{name} has type {t.dtype}")
    if t.shape != shape:
        _bad(fn, E_SHAPE, f"{name} has shape {tuple(t.shape)}, not {shape}")
    if t.device != device:
        _bad(fn, E_ARG, f"{name} is on {t.device}, not {device}")
    _bad(fn, E_ARG, f"{name} has gaps within a row")


def spear_rope(x: torch.Tensor, positions: torch.Tensor, rope: Rope,
               y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x [T][H][D] bf16 (rows may lie apart) with every head rotated to its row's
    position; y may be x itself."""
    fn = "spear_rope"
    dev = x.device
    shape = x.shape
    if len(shape) != 3:
        _bad(fn, E_SHAPE, f"x has {len(shape)} dimensions, not 3")
    T, H, D = shape
    xs = _want_rows(fn, "x", x, shape, dev)
    _want(fn, "positions", positions, _I32, (T,), dev)
    ys = H * D if y is None else _want_rows(fn, "y", y, shape, dev)
    if rope.freqs.device != dev:
        _bad(fn, E_ARG, f"the rotation is on {rope.freqs.device}, not {dev}")

    def call(s):
        nonlocal y
        if y is None:
            y = torch.empty(shape, dtype=x.dtype, device=dev)
        return load().spear_rope(x.data_ptr(), xs, T, H, D, positions.data_ptr(), rope._s,
                                 y.data_ptr(), ys, s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return y


def spear_rope_kv4_write(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         positions: Optional[torch.Tensor], slots: torch.Tensor,
                         rope: Optional[Rope], kv: KV4, q_out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """-> q [T][Hq][D] rotated (q_out may be q itself); k, rotated, and v [T][heads][D]
    go into their slots of the cache.  q, k and v may be parts of one row; rope
    None rotates nothing."""
    fn = "spear_rope_kv4_write"
    dev = q.device
    if q.dim() != 3:
        _bad(fn, E_SHAPE, f"q has {q.dim()} dimensions, not 3")
    T, Hq = int(q.shape[0]), int(q.shape[1])
    shape, row = (T, Hq, kv.D), (T, kv.heads, kv.D)
    qs = _want_rows(fn, "q", q, shape, kv.device)
    ks = _want_rows(fn, "k", k, row, dev)
    vs = _want_rows(fn, "v", v, row, dev)
    _want(fn, "slots", slots, _I64, (T,), dev)
    if rope is not None:
        if positions is None:
            _bad(fn, E_NULL, "positions is missing")
        _want(fn, "positions", positions, _I32, (T,), dev)
        if rope.freqs.device != dev:
            _bad(fn, E_ARG, f"the rotation is on {rope.freqs.device}, not {dev}")
    ys = Hq * kv.D if q_out is None else _want_rows(fn, "q_out", q_out, shape, dev)

    def call(s):
        nonlocal q_out
        if q_out is None:
            q_out = torch.empty(shape, dtype=q.dtype, device=dev)
        return load().spear_rope_kv4_write(
            q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, Hq,
            None if rope is None else positions.data_ptr(), slots.data_ptr(),
            None if rope is None else rope._s, kv._s, q_out.data_ptr(), ys, s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return q_out


def spear_kv4_read(kv: KV4, slots: torch.Tensor, k: Optional[torch.Tensor] = None,
                   v: Optional[torch.Tensor] = None, stream=None, parts: str = "kv"):
    """-> (k, v) [T][heads][D] bf16: the cache's rows, exact (zeros for a slot
    outside the cache); parts "k" or "v" reads that one alone and gives None for
    the other."""
    fn = "spear_kv4_read"
    dev = kv.device
    if parts not in ("kv", "k", "v") or (k is not None and "k" not in parts) or (v is not None and "v" not in parts):
        _bad(fn, E_ARG, f"parts is {parts!r}")
    shape = T, _, _ = (slots.numel(), kv.heads, kv.D)
    _want(fn, "slots", slots, _I64, (T,), dev)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _want(fn, name, t, _BF16, shape, dev)

    def call(s):
        nonlocal k, v
        if k is None and "k" in parts:
            k = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        if v is None and "v" in parts:
            v = torch.empty(shape, dtype=torch.bfloat16, device=dev)
        return load().spear_kv4_read(kv._s, slots.data_ptr(), T, _at(k), _at(v), s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return k, v


def spear_kv4_attention_workspace_size(T: int, B: int, max_fresh: int, Hq: int, heads: int, D: int,
                                       width: int, P: int) -> int:
    return int(load().spear_kv4_attention_workspace_size(T, B, max_fresh, Hq, heads, D, width, P))


def new_kv4_workspace(T: int, B: int, max_fresh: int, Hq: int, kv: KV4, width: int) -> torch.Tensor:
    """A workspace for spear_kv4_attention over T rows of B requests, none with more
    than max_fresh of them, and a table of that width, its counters zeroed (torch
    allocation)."""
    n = spear_kv4_attention_workspace_size(T, B, max_fresh, Hq, kv.heads, kv.D, width, kv.P)
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device=kv.device)
    ws[:KV4_COUNTER_BYTES].zero_()
    return ws


def spear_kv4_attention(q: torch.Tensor, kv: KV4, table: torch.Tensor, q_start: torch.Tensor,
                        kv_len: torch.Tensor, max_fresh: int, scale: Optional[float] = None,
                        window: int = 0, y: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of the step's rows q [T][Hq][D] bf16 over the cache -> y [T][Hq][D]
    bf16; lse [T][Hq] fp32 is filled if given.  scale None: 1 / sqrt(D).  Rows
    behind the last request are left as they are."""
    fn = "spear_kv4_attention"
    dev, B = kv.device, kv_len.numel()
    if q.dim() != 3:
        _bad(fn, E_SHAPE, f"q has {q.dim()} dimensions, not 3")
    if table.dim() != 2:
        _bad(fn, E_SHAPE, f"table has {table.dim()} dimensions, not 2")
    _want_int32(fn, "window", window)
    T, Hq, width = int(q.shape[0]), int(q.shape[1]), int(table.shape[1])
    shape = (T, Hq, kv.D)
    qs = _want_rows(fn, "q", q, shape, dev)
    _want(fn, "table", table, _I32, (B, width), dev)
    _want(fn, "q_start", q_start, _I32, (B + 1,), dev)
    _want(fn, "kv_len", kv_len, _I32, (B,), dev)
    if y is not None:
        _want(fn, "y", y, _BF16, shape, dev)
    if lse is not None:
        _want(fn, "lse", lse, _F32, (T, Hq), dev)
    if workspace is not None:
        _want_workspace(fn, workspace, dev)

    def call(s):
        nonlocal y, workspace
        if y is None:
            y = torch.empty(shape, dtype=q.dtype, device=dev)
        if workspace is None:
            workspace = new_kv4_workspace(T, B, max_fresh, Hq, kv, width)
        return load().spear_kv4_attention(
            q.data_ptr(), qs, T, Hq, kv._s, table.data_ptr(), width, q_start.data_ptr(),
            kv_len.data_ptr(), B, max_fresh, kv.D ** -0.5 if scale is None else scale, window,
            y.data_ptr(), _at(lse), workspace.data_ptr(), workspace.numel(), s)

    st = _on(fn, dev, stream, call)
    if st != SPEAR_OK:
        _check(fn, st)
    return y


def spear_set_wait_limit(rounds: int):
    load().spear_set_wait_limit(int(rounds))


def spear_workspace_timeouts(ws: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int32(0)
    _check("spear_workspace_timeouts", load().spear_workspace_timeouts(_ptr(ws), ctypes.byref(out),
                                                                       _stream(stream)))
    return int(out.value)


def spear_stream_read(buf: torch.Tensor, sink: torch.Tensor, nbytes: Optional[int] = None,
                      stream=None):
    """Measurement helper: read every byte of buf once (the plain read floor)."""
    n = buf.numel() * buf.element_size() if nbytes is None else nbytes
    _check("spear_stream_read", load().spear_stream_read(_ptr(buf), n, _ptr(sink),
                                                         _stream(stream)))


class SloLut:
    """Kernel-latency table for the chunk picker (host memory): tokens [P]
    ascending, us [kinds][P] microseconds per call, count [kinds] calls per
    step, overhead_us per step."""

    def __init__(self, tokens, us, count, overhead_us=0.0):
        import numpy as np
        self.tokens = np.ascontiguousarray(tokens, dtype=np.int32)
        self.us = np.ascontiguousarray(us, dtype=np.float32)
        self.count = np.ascontiguousarray(count, dtype=np.int32)
        assert self.us.shape == (self.count.shape[0], self.tokens.shape[0])
        self._c = _LUT(self.tokens.shape[0], self.tokens.ctypes.data, self.count.shape[0],
                       self.us.ctypes.data, self.count.ctypes.data, float(overhead_us))

    def predict(self, tokens: int) -> float:
        out = ctypes.c_float(0)
        _check("spear_slo_predict", load().spear_slo_predict(ctypes.byref(self._c), int(tokens),
                                                             ctypes.byref(out)))
        return float(out.value)

    def pick_chunk(self, n_decode: int, pending: int, slo_us: float, align: int = 1):
        c, p = ctypes.c_int32(0), ctypes.c_float(0)
        _check("spear_slo_pick_chunk", load().spear_slo_pick_chunk(
            ctypes.byref(self._c), int(n_decode), int(pending), int(align), float(slo_us),
            ctypes.byref(c), ctypes.byref(p)))
        return int(c.value), float(p.value)
