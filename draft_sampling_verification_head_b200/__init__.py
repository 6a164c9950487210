"""Thin Python binding of libspecdec.so (include/specdec.h).

Argument marshalling only: every step of the method runs in the library's
CUDA kernels.  PyTorch provides device memory and the current stream.  The
library must have been built (``build.py``); importing this module on a
machine without it raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes
import os
from contextlib import nullcontext
from dataclasses import dataclass, fields

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libspecdec.so")

SPEC_OK, SPEC_ERR_INVALID_ARG, SPEC_ERR_UNSUPPORTED, SPEC_ERR_CUDA = 0, -1, -2, -3
SPEC_ERR_TIMEOUT, SPEC_ERR_WORKSPACE, SPEC_ERR_TOKEN_RANGE = -4, -5, -6
SPEC_F32, SPEC_BF16 = 0, 1
SPEC_FLAG_FMA_BIAS = 1
SPEC_FLAG_TRACE = 2
SPEC_WORKSPACE_MIN = 256
SPEC_SCAN_CHUNK = 16

# (name, restype, argtypes) of every exported symbol declared in include/*.h
_P = ctypes.c_void_p
_SIGS = {
    "spec_workspace_size": (ctypes.c_size_t, [_P]),
    "spec_workspace_init": (ctypes.c_int, [_P, ctypes.c_size_t, _P]),
    "spec_markov_bias": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P]),
    "spec_markov_bias_sample": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_verify_block": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_verify_block_kb": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_cycle": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_cycle_kb": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_decode_loop": (ctypes.c_int, [_P, ctypes.c_int32, _P, _P, _P, ctypes.c_float, _P, _P, _P,
                                         _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_cycle_rnn": (ctypes.c_int, [_P] * 14),
    "spec_sync_status": (ctypes.c_int, [_P, _P]),
    "spec_cycle_noalloc": (ctypes.c_int, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_l2_persist": (ctypes.c_int, [_P, ctypes.c_size_t, _P]),
    "spec_schedule_verify_len": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, _P,
                                                 ctypes.c_int32, _P, _P]),
    "spec_embed_workspace_size": (ctypes.c_size_t, [_P]),
    "spec_embed": (ctypes.c_int, [_P] * 6),
    "spec_embed_grad": (ctypes.c_int, [_P] * 6),
    "spec_scan_workspace_size": (ctypes.c_size_t, [_P]),
    "spec_gated_scan": (ctypes.c_int, [_P] * 10),
    "spec_gated_scan_grad": (ctypes.c_int, [_P] * 13),
    "spec_w4_workspace_size": (ctypes.c_size_t, [_P]),
    "spec_bias_w4": (ctypes.c_int, [_P] * 9),
    "spec_w4_quantize": (ctypes.c_int, [_P, _P, ctypes.c_int32, _P, _P, _P]),
    "spec_verify_probs": (ctypes.c_int, [_P] * 13),
    "spec_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "spec_last_launch_count": (ctypes.c_int32, []),
    "spec_debug_scan_polls": (ctypes.c_int, [ctypes.c_int64]),
    "spec_debug_philox": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P]),
    "spec_debug_curand_philox": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P]),
}


class SpecParams(ctypes.Structure):
    """Mirror of spec_params."""
    _fields_ = [("B", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
                ("r", ctypes.c_int32), ("dtype", ctypes.c_int32), ("draft_dtype", ctypes.c_int32),
                ("temperature", ctypes.c_float), ("greedy", ctypes.c_int32),
                ("seed", ctypes.c_uint64), ("cycle", ctypes.c_uint64),
                ("spin_limit", ctypes.c_uint64), ("flags", ctypes.c_uint32),
                ("row_offset", ctypes.c_uint32)]


class SpecEmbedParams(ctypes.Structure):
    """Mirror of spec_embed_params."""
    _fields_ = [("n", ctypes.c_int32), ("V", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("row_dtype", ctypes.c_int32),
                ("accumulate", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("table_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64)]


class SpecScanParams(ctypes.Structure):
    """Mirror of spec_scan_params."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("D", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate_stride", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("h_stride", ctypes.c_int64)]


class SpecW4Params(ctypes.Structure):
    """Mirror of spec_w4_params."""
    _fields_ = [("B", ctypes.c_int32), ("r", ctypes.c_int32), ("V", ctypes.c_int32),
                ("group", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32), ("base_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("x_rows", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("x_stride", ctypes.c_int64),
                ("base_stride", ctypes.c_int64), ("out_stride", ctypes.c_int64)]


class SpecProbsParams(ctypes.Structure):
    """Mirror of spec_probs_params."""
    _fields_ = [("B", ctypes.c_int32), ("K", ctypes.c_int32), ("V", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("draft_dtype", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("target_stride", ctypes.c_int64),
                ("draft_stride", ctypes.c_int64)]


_lib = None


def lib():
    """Load libspecdec.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run draft_sampling_verification_head_b200/build.py")
        h = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(h, name)
            f.restype = res
            f.argtypes = args
        _lib = h
    return _lib


class SpecError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


def status_string(code: int) -> str:
    return lib().spec_status_string(code).decode()


@dataclass
class Params:
    B: int
    K: int
    V: int
    r: int
    dtype: str = "bf16"
    temperature: float = 1.0
    greedy: bool = False
    seed: int = 0
    cycle: int = 0
    spin_limit: int = 0
    flags: int = 0
    draft_dtype: str | None = None
    row_offset: int = 0  # global index of batch row 0 (Philox counter word 1)

    def c(self) -> SpecParams:
        dt = {"f32": SPEC_F32, "bf16": SPEC_BF16}
        return SpecParams(self.B, self.K, self.V, self.r, dt[self.dtype],
                          dt[self.draft_dtype or self.dtype], float(self.temperature),
                          1 if self.greedy else 0, self.seed & (2**64 - 1),
                          self.cycle & (2**64 - 1), self.spin_limit, self.flags,
                          self.row_offset)


_DT = {"f32": SPEC_F32, "bf16": SPEC_BF16}


class _Calls:
    """What the calls of one parameter object use: the C structure and its
    address, by call the (name, dtype, rows, row stride, row width) of each
    tensor and, as _run looks at them, `ready`; and by device the workspace
    sizes `need` that are known."""
    __slots__ = ("c", "at", "args", "ready", "need")

    def __init__(self, c, args):
        self.c, self.at, self.args = c, ctypes.addressof(c), args
        self.ready, self.need = {}, {}


class _Held:
    """A parameter object whose calls are prepared once: it is frozen.  The
    _Calls are made whole and published by one step, which the first of several
    threads wins, so nobody sees a part of them or another structure's address."""

    def __getattr__(self, name):  # only where the attribute is missing
        if name != "_calls":
            raise AttributeError(f"{type(self).__name__!r} object has no attribute {name!r}")
        return self.__dict__.setdefault("_calls", _Calls(self._make(), self._tensors()))

    def _size(self):
        """Workspace bytes by the library on the current device; 0 where the
        parameters are invalid (or, for the recurrence, without a GPU)."""
        return SPEC_WORKSPACE_MIN

    def c(self):
        return self._make()

    def __reduce__(self):  # copies make their own C structure
        return type(self), tuple(getattr(self, f.name) for f in fields(self))


@dataclass(frozen=True)
class EmbedParams(_Held):
    """Sizes of embed / embed_grad (spec_embed_params)."""
    n: int
    V: int
    D: int
    dtype: str = "bf16"
    row_dtype: str = "bf16"
    scale: float = 1.0
    accumulate: bool = False
    table_stride: int = 0
    row_stride: int = 0

    def _make(self):
        return SpecEmbedParams(self.n, self.V, self.D, _DT[self.dtype], _DT[self.row_dtype],
                               1 if self.accumulate else 0, float(self.scale), 0,
                               self.table_stride, self.row_stride)

    def _size(self):
        return int(lib().spec_embed_workspace_size(self._calls.at))

    def _tensors(self):
        table = (self.dtype, self.V, self.table_stride or self.D, self.D)
        rows = (self.row_dtype, self.n, self.row_stride or self.D, self.D)
        ids = ("ids", "i32", 1, self.n, self.n)
        return {"embed": (("table", *table), ids, ("rows", *rows)),
                "embed_grad": (ids, ("drows", *rows), ("dtable", *table))}


@dataclass(frozen=True)
class ScanParams(_Held):
    """Sizes of gated_scan / gated_scan_grad (spec_scan_params)."""
    B: int
    T: int
    D: int
    dtype: str = "bf16"
    gate_stride: int = 0
    x_stride: int = 0
    h_stride: int = 0

    def _make(self):
        return SpecScanParams(self.B, self.T, self.D, _DT[self.dtype], self.gate_stride,
                              self.x_stride, self.h_stride)

    def _size(self):
        return int(lib().spec_scan_workspace_size(self._calls.at))

    def _tensors(self):
        n, D = self.B * self.T, self.D
        gate = (self.dtype, n, self.gate_stride or D, D)
        x = (self.dtype, n, self.x_stride or D, D)
        h = (self.dtype, n, self.h_stride or D, D)
        state = ("f32", self.B, D, D)
        lens = ("len", "i32", 1, self.B, self.B)
        states = ("states", "f32", self.B * -(-self.T // SPEC_SCAN_CHUNK), D, D)
        return {"scan": (("gate", *gate), ("x", *x), ("h0", *state), lens, ("h", *h),
                         ("h_last", *state), states),
                "scan_grad": (("gate", *gate), ("x", *x), ("h0", *state), lens, states,
                              ("dh", *h), ("dh_last", *state), ("dgate", *gate), ("dx", *x),
                              ("dh0", *state))}


@dataclass(frozen=True)
class W4Params(_Held):
    """Sizes of bias_w4 / w4_quantize (spec_w4_params)."""
    B: int
    r: int
    V: int
    group: int = 128
    dtype: str = "bf16"
    scale_dtype: str = "bf16"
    base_dtype: str = "bf16"
    out_dtype: str = "f32"
    x_rows: int = 0
    x_stride: int = 0
    base_stride: int = 0
    out_stride: int = 0

    def _make(self):
        return SpecW4Params(self.B, self.r, self.V, self.group, _DT[self.dtype],
                            _DT[self.scale_dtype], _DT[self.base_dtype], _DT[self.out_dtype],
                            self.x_rows, 0, self.x_stride, self.base_stride, self.out_stride)

    def _size(self):
        return int(lib().spec_w4_workspace_size(self._calls.at))

    def _tensors(self):
        codes, groups = -(-self.r // 128) * 64, self.r // max(self.group, 1)
        rest = (("wq", "u8", self.V, codes, codes),
                ("wscale", self.scale_dtype, self.V, groups, groups),
                ("base", self.base_dtype, self.B, self.base_stride or self.V, self.V),
                ("out", self.out_dtype, self.B, self.out_stride or self.V, self.V))
        prev = ("prev", "i32", 1, self.B, self.B)
        x = self.x_stride or self.r
        return {"rows": (("x", self.dtype, self.B, x, self.r), prev, *rest),
                "lookup": (("x", self.dtype, self.x_rows, x, self.r), prev, *rest)}


@dataclass(frozen=True)
class ProbsParams(_Held):
    """Sizes of verify_probs (spec_probs_params)."""
    B: int
    K: int
    V: int
    dtype: str = "f32"
    draft_dtype: str = "f32"
    target_stride: int = 0
    draft_stride: int = 0

    def _make(self):
        return SpecProbsParams(self.B, self.K, self.V, _DT[self.dtype], _DT[self.draft_dtype], 0,
                               self.target_stride, self.draft_stride)

    def _tensors(self):
        B, K, V = self.B, self.K, self.V
        return {"verify": (("target", self.dtype, B * (K + 1), self.target_stride or V, V),
                           ("draft_probs", self.draft_dtype, B * K, self.draft_stride or V, V),
                           ("draft", "i32", B, K, K), ("u_accept", "f32", B, K, K),
                           ("u_draw", "f32", 1, B, B), ("verify_len", "i32", 1, B, B),
                           ("out", "i32", B, K + 1, K + 1), ("tau", "i32", 1, B, B),
                           ("p_draft", "f32", B, K, K), ("q_draft", "f32", B, K, K))}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, what):
    if code != SPEC_OK:
        raise SpecError(code, what)


def workspace_size(p) -> int:
    """Bytes of workspace for the calls these parameters (of any kind) belong to,
    on the current device."""
    if isinstance(p, _Held):
        return p._size()
    return int(lib().spec_workspace_size(ctypes.byref(p.c())))


def make_workspace(p, device="cuda"):
    """Allocate and zero a workspace for these parameters (torch memory)."""
    import torch
    d = torch.device(device)
    named = d.type == "cuda" and d.index is not None
    with torch.cuda.device(d) if named else nullcontext():  # sized for it, zeroed on its stream
        n = workspace_size(p)
        if n == 0:
            raise SpecError(SPEC_ERR_INVALID_ARG, "spec_workspace_size")
        ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
        off = (-ws.data_ptr()) % 256
        ws = ws[off:off + n]
        _check(lib().spec_workspace_init(_ptr(ws), n, _stream(None)), "spec_workspace_init")
    return ws


def workspace_init(ws, stream=None):
    _check(lib().spec_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "spec_workspace_init")


def markov_bias(p: Params, U, W, prev, bias, ws, stream=None):
    _check(lib().spec_markov_bias(ctypes.byref(p.c()), _ptr(U), _ptr(W), _ptr(prev), _ptr(bias),
                                  _ptr(ws), _stream(stream)), "spec_markov_bias")


def markov_bias_sample(p: Params, base, U, W, last_token, draft, q_draft, biased_out, ws,
                       stream=None):
    _check(lib().spec_markov_bias_sample(ctypes.byref(p.c()), _ptr(base), _ptr(U), _ptr(W),
                                         _ptr(last_token), _ptr(draft), _ptr(q_draft),
                                         _ptr(biased_out), _ptr(ws), _stream(stream)),
           "spec_markov_bias_sample")


def verify_block(p: Params, target, draft_logits, draft, out, tau, p_draft, q_draft, ws,
                 stream=None):
    _check(lib().spec_verify_block(ctypes.byref(p.c()), _ptr(target), _ptr(draft_logits),
                                   _ptr(draft), _ptr(out), _ptr(tau), _ptr(p_draft),
                                   _ptr(q_draft), _ptr(ws), _stream(stream)), "spec_verify_block")


def verify_block_kb(p: Params, target, draft_logits, draft, verify_len, out, tau, p_draft, q_draft,
                    ws, stream=None):
    """spec_verify_block_kb: verification with a verify length K_b per row."""
    _check(lib().spec_verify_block_kb(ctypes.byref(p.c()), _ptr(target), _ptr(draft_logits),
                                      _ptr(draft), _ptr(verify_len), _ptr(out), _ptr(tau),
                                      _ptr(p_draft), _ptr(q_draft), _ptr(ws), _stream(stream)),
           "spec_verify_block_kb")


def cycle(p: Params, base, target, U, W, last_token, draft, out, tau, p_draft, q_draft, ws,
          stream=None):
    _check(lib().spec_cycle(ctypes.byref(p.c()), _ptr(base), _ptr(target), _ptr(U), _ptr(W),
                            _ptr(last_token), _ptr(draft), _ptr(out), _ptr(tau), _ptr(p_draft),
                            _ptr(q_draft), _ptr(ws), _stream(stream)), "spec_cycle")


def cycle_kb(p: Params, base, target, U, W, last_token, verify_len, draft, out, tau, p_draft,
             q_draft, ws, stream=None):
    """spec_cycle_kb: one cycle with a verify length K_b per row (int32 [B], 1..K)."""
    _check(lib().spec_cycle_kb(ctypes.byref(p.c()), _ptr(base), _ptr(target), _ptr(U), _ptr(W),
                               _ptr(last_token), _ptr(verify_len), _ptr(draft), _ptr(out),
                               _ptr(tau), _ptr(p_draft), _ptr(q_draft), _ptr(ws),
                               _stream(stream)), "spec_cycle_kb")


def decode_loop(p: Params, n_cycles, base, target, U, W, last_token, draft, out, tau, p_draft,
                q_draft, next_token, ws, conf=None, conf_threshold=0.0, verify_len=None,
                stream=None):
    """spec_decode_loop: n_cycles chained cycles in one launch; inputs and
    outputs carry a leading cycle axis, next_token [B] the last cycle's last
    emitted tokens."""
    _check(lib().spec_decode_loop(ctypes.byref(p.c()), int(n_cycles), _ptr(base), _ptr(target),
                                  _ptr(conf), float(conf_threshold), _ptr(verify_len), _ptr(U),
                                  _ptr(W), _ptr(last_token), _ptr(draft), _ptr(out), _ptr(tau),
                                  _ptr(p_draft), _ptr(q_draft), _ptr(next_token), _ptr(ws),
                                  _stream(stream)), "spec_decode_loop")


def cycle_rnn(p: Params, base, target, U, W, Wh, last_token, draft, out, tau, p_draft, q_draft, ws,
              stream=None):
    """spec_cycle_rnn: one cycle with the RNN sequential head (Wh [r, r] bf16)."""
    _check(lib().spec_cycle_rnn(ctypes.byref(p.c()), _ptr(base), _ptr(target), _ptr(U), _ptr(W),
                                _ptr(Wh), _ptr(last_token), _ptr(draft), _ptr(out), _ptr(tau),
                                _ptr(p_draft), _ptr(q_draft), _ptr(ws), _stream(stream)),
           "spec_cycle_rnn")


def cycle_noalloc(p: Params, base, target, U, W, last_token, draft, out, tau, p_draft, q_draft,
                  status_out=None, stream=None):
    """spec_cycle on the library's built-in scratch array (no workspace)."""
    _check(lib().spec_cycle_noalloc(ctypes.byref(p.c()), _ptr(base), _ptr(target), _ptr(U),
                                    _ptr(W), _ptr(last_token), _ptr(draft), _ptr(out), _ptr(tau),
                                    _ptr(p_draft), _ptr(q_draft), _ptr(status_out),
                                    _stream(stream)), "spec_cycle_noalloc")


def sync_status(ws, stream=None) -> int:
    return int(lib().spec_sync_status(_ptr(ws), _stream(stream)))


def l2_persist(t, nbytes=None, stream=None):
    """Keep tensor `t` (e.g. the Markov factor W) resident in L2 for kernels
    launched on the stream; t=None clears the window."""
    ptr = None if t is None else ctypes.c_void_p(t.data_ptr())
    n = 0 if t is None else (t.numel() * t.element_size() if nbytes is None else nbytes)
    _check(lib().spec_l2_persist(ptr, n, _stream(stream)), "spec_l2_persist")


def schedule_verify_len(conf, sps):
    """Verify length per request from confidence scores conf [B, K] and the
    steps-per-second table sps [n] (host arrays).  Returns (verify_len [B]
    int32, expected tokens per step, expected tokens per second)."""
    import numpy as np
    c = np.ascontiguousarray(conf, dtype=np.float32)
    s = np.ascontiguousarray(sps, dtype=np.float64)
    if c.ndim != 2 or s.ndim != 1:
        raise ValueError("conf must be [B, K] and sps one-dimensional")
    kb = np.empty(c.shape[0], np.int32)
    ex = np.zeros(2, np.float64)
    _check(lib().spec_schedule_verify_len(c.ctypes.data, c.shape[0], c.shape[1], s.ctypes.data,
                                          s.shape[0], kb.ctypes.data, ex.ctypes.data),
           "spec_schedule_verify_len")
    return kb, float(ex[0]), float(ex[1])


_TORCH = None  # what the operators' calls use of torch, looked up once


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        # the device and the stream's handle without further Python, where torch offers it
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda d: torch.cuda.current_stream(d).cuda_stream)
        torch.cuda.init()
        _TORCH = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device), raw,
                  {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32,
                   "u8": torch.uint8})
    return _TORCH


def _check_rows(name, t, rows, stride, width):
    """A tensor's rows must lie where the call looks for them: `stride` elements
    apart, one after the other over all leading axes.  A flat tensor, or whole
    storage with longer rows, will do if it holds them."""
    need = 0 if rows <= 0 else (rows - 1) * stride + width
    last = t.storage_offset() + need
    if t.untyped_storage().nbytes() < last * t.element_size():
        raise ValueError(f"{name} holds too few elements, expected {rows} rows of {width}")
    if need == 0:
        return
    if t.dim() == 0 or t.stride(-1) != 1 and t.size(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if t.dim() == 1:
        if t.numel() < need:
            raise ValueError(f"{name} holds {t.numel()} elements, expected {need}")
        return
    if t.size(-1) < width or t.numel() // t.size(-1) < rows:
        raise ValueError(f"{name} is {tuple(t.shape)}, expected {rows} rows of {width}")
    apart = stride  # what one step along the axis, from the last but one outwards, moves
    for k in range(t.dim() - 2, -1, -1):
        if t.size(k) != 1 and t.stride(k) != apart:
            raise ValueError(f"{name}: its rows are not {stride} elements apart")
        apart *= t.size(k)


_STATUS_ONLY = frozenset(("embed", "verify"))  # calls without scratch: any workspace will do


def _need(p, dev):
    """Workspace bytes that a call on `dev`, the current device, needs.  The
    recurrence splits its steps by the device's size, so each has its own; a 0
    (no device, bad parameters: the library says which) is asked for again."""
    need = p._size()
    if need > 0:
        p._calls.need[dev] = need
    return need


def _typed(held, call):
    """The tensors of a call as _run looks at them: (torch dtype, row stride,
    elements of all rows), and what _check_rows wants."""
    types = (_TORCH or _torch())[2]
    args = tuple((types[dt], stride, rows * stride, name, dt, rows, width)
                 for name, dt, rows, stride, width in held.args[call])
    held.ready[call] = args
    return args


def _run(fn, p, call, tensors, ws, stream):
    """One operator's call, after the checks that the C side cannot make.
    Tensors, workspace and stream must belong to the current device."""
    current, raw, _ = _TORCH or _torch()
    held = p._calls
    dev = current()
    if stream is None:
        st = raw(dev)
    elif stream.device_index == dev:
        st = stream.cuda_stream
    else:
        raise ValueError("the stream belongs to another device than the current one")
    ptr = []
    for t, (dtype, stride, total, name, dt, rows, width) in zip(tensors, held.ready.get(call)
                                                                or _typed(held, call)):
        if t is None:
            ptr.append(None)
            continue
        if t.dtype is not dtype:
            raise ValueError(f"{name} is {t.dtype}, expected {dt}")
        if t.get_device() != dev:
            raise ValueError(f"{name} is on {t.device}, the call on cuda:{dev}")
        # dense rows, the common case, in three looks
        if not (t.is_contiguous() and t.numel() >= total and t.size(-1) == stride):
            _check_rows(name, t, rows, stride, width)
        ptr.append(t.data_ptr())
    need = SPEC_WORKSPACE_MIN if call in _STATUS_ONLY else held.need.get(dev) or _need(p, dev)
    if ws.get_device() != dev or ws.nbytes < need:
        raise SpecError(SPEC_ERR_WORKSPACE, f"{fn}: workspace too small or on another device")
    code = getattr(_lib or lib(), fn)(held.at, *ptr, ws.data_ptr(), st)
    if code != SPEC_OK:
        raise SpecError(code, fn)


def embed(p: EmbedParams, table, ids, rows, ws, stream=None):
    """spec_embed: rows[i] = scale * table[ids[i]] (ids int32; -1 gives zeros)."""
    _run("spec_embed", p, "embed", (table, ids, rows), ws, stream)


def embed_grad(p: EmbedParams, ids, drows, dtable, ws, stream=None):
    """spec_embed_grad: dtable[v] (+)= scale * sum of drows[i] with ids[i] = v."""
    _run("spec_embed_grad", p, "embed_grad", (ids, drows, dtable), ws, stream)


def gated_scan(p: ScanParams, gate, x, h0, len, h, h_last, states, ws, stream=None):
    """spec_gated_scan: h_t = f_t h_{t-1} + (1 - f_t) x_t, f = sigmoid(gate).
    h0, len, h, h_last and states may be None."""
    _run("spec_gated_scan", p, "scan", (gate, x, h0, len, h, h_last, states), ws, stream)


def gated_scan_grad(p: ScanParams, gate, x, h0, len, states, dh, dh_last, dgate, dx, dh0, ws,
                    stream=None):
    """spec_gated_scan_grad: the gradients of gate, x and h0 from dh and dh_last.
    h0, len, dh_last and dh0 may be None; states as gated_scan wrote them."""
    _run("spec_gated_scan_grad", p, "scan_grad",
         (gate, x, h0, len, states, dh, dh_last, dgate, dx, dh0), ws, stream)


def bias_w4(p: W4Params, x, prev, wq, wscale, base, out, ws, stream=None):
    """spec_bias_w4: out = base + X . W with W in 4 bits (X[b] = x[prev[b]] or
    x[b]).  prev and base may be None."""
    _run("spec_bias_w4", p, "rows" if prev is None else "lookup",
         (x, prev, wq, wscale, base, out), ws, stream)


def w4_quantize(p: W4Params, W, stream=None):
    """spec_w4_quantize: (wq, wscale) of a factor W [r, V] (float32 or bfloat16)."""
    import torch
    if W.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"W is {W.dtype}, expected float32 or bfloat16")
    if W.get_device() != torch.cuda.current_device() or not W.is_contiguous() or \
            W.numel() < p.r * p.V:
        raise ValueError("W must be a contiguous [r, V] tensor on the current device")
    if p.group < 1 or p.r % p.group:
        raise SpecError(SPEC_ERR_UNSUPPORTED, "spec_w4_quantize")
    s = stream if stream is not None else torch.cuda.current_stream()
    with torch.cuda.stream(s):  # the outputs' memory belongs to the call's stream
        wq = torch.empty(p.V, -(-p.r // 128) * 64, dtype=torch.uint8, device=W.device)
        wscale = torch.empty(p.V, p.r // p.group, device=W.device,
                             dtype=torch.bfloat16 if p.scale_dtype == "bf16" else torch.float32)
    _check(lib().spec_w4_quantize(p._calls.at, W.data_ptr(), SPEC_BF16 if W.dtype is torch.bfloat16
                                  else SPEC_F32, wq.data_ptr(), wscale.data_ptr(),
                                  s.cuda_stream), "spec_w4_quantize")
    return wq, wscale


def verify_probs(p: ProbsParams, target, draft_probs, draft, u_accept, u_draw, verify_len, out,
                 tau, p_draft, q_draft, ws, stream=None):
    """spec_verify_probs: verification from probabilities and given uniforms.
    verify_len, p_draft and q_draft may be None."""
    _run("spec_verify_probs", p, "verify",
         (target, draft_probs, draft, u_accept, u_draw, verify_len, out, tau, p_draft, q_draft),
         ws, stream)


def last_launch_count() -> int:
    return int(lib().spec_last_launch_count())


def debug_philox(ctr, key, out, stream=None):
    _check(lib().spec_debug_philox(_ptr(ctr), _ptr(key), _ptr(out), ctr.shape[0],
                                   _stream(stream)), "spec_debug_philox")


def debug_curand_philox(ctr, key, out, stream=None):
    _check(lib().spec_debug_curand_philox(_ptr(ctr), _ptr(key), _ptr(out), ctr.shape[0],
                                          _stream(stream)), "spec_debug_curand_philox")


def alloc_outputs(p: Params, device="cuda", n_cycles=None):
    """Output tensors for one cycle, or with a leading axis of n_cycles."""
    import torch
    lead = () if n_cycles is None else (int(n_cycles),)
    return dict(draft=torch.full(lead + (p.B, p.K), -7, dtype=torch.int32, device=device),
                out=torch.full(lead + (p.B, p.K + 1), -7, dtype=torch.int32, device=device),
                tau=torch.zeros(lead + (p.B,), dtype=torch.int32, device=device),
                p_draft=torch.full(lead + (p.B, p.K), -1.0, dtype=torch.float32, device=device),
                q_draft=torch.full(lead + (p.B, p.K), -1.0, dtype=torch.float32, device=device))
