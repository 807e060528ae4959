"""Thin ctypes binding of libqgemm.so (the C ABI in include/qgemm.h).

Argument marshalling only: every step of the computation runs in the CUDA library.  The
functions mirror the C names; torch tensors stand in for device pointers and torch's
current stream is passed as `stream`.  The library is loaded on first use; if it is
missing or fails to load, the call raises -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

Q8_0, NVFP4, MXFP4, FP8 = 0, 1, 2, 3
FORMATS = {"q8_0": Q8_0, "nvfp4": NVFP4, "mxfp4": MXFP4, "fp8": FP8}
Y_F32, Y_BF16 = 0, 1
BLOCK = {Q8_0: 32, NVFP4: 16, MXFP4: 32, FP8: 16}  # K granularity (FP8: no block scales)
TENSOR_SCALE = (NVFP4, FP8)

OK = 0
STATUS = {
    0: "QGEMM_OK", 1: "QGEMM_ERR_FORMAT", 2: "QGEMM_ERR_SHAPE", 3: "QGEMM_ERR_K_BLOCK",
    4: "QGEMM_ERR_NULL", 5: "QGEMM_ERR_ALIGN", 6: "QGEMM_ERR_WORKSPACE", 7: "QGEMM_ERR_CUDA",
    8: "QGEMM_ERR_DEVICE", 9: "QGEMM_ERR_DEVICE_TIMEOUT", 10: "QGEMM_ERR_DEVICE_ARG",
}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqgemm.so")
_lib = None
_lock = threading.Lock()

# (name, restype, argtypes) of every exported entry point
_I64, _SZ, _VP, _I = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
SIGNATURES = [
    ("qgemm_packed_size", _I, [_I, _I64, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    ("qgemm_packed_geometry", _I, [_I, _I64, _I64, ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                                   ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    ("qgemm_row_pitches", _I, [_I, _I64, ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    ("qgemm_repack_rowmajor", _I, [_I, _I64, _I64, _VP, _I64, _VP, _I64, _VP, _VP, _VP]),
    ("qgemm_pack", _I, [_I, _VP, _I64, _I64, _VP, _VP, _VP, _VP]),
    ("qgemm_workspace_size", _I, [_I, _I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    ("qgemm_run", _I, [_I, _VP, _I64, _I64, _VP, _VP, _VP, _I64, _VP, _I, _VP, _SZ, _VP]),
    ("qgemm_run_noalloc", _I, [_I, _VP, _I64, _I64, _VP, _VP, _VP, _I64, _VP, _I, _VP]),
    ("qgemm_ffn_workspace_size", _I, [_I, _I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    ("qgemm_ffn_gate_up", _I, [_I, _VP, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP, _VP,
                               _SZ, _VP]),
    ("qgemm_moe_workspace_size", _I, [_I, _I64, _I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    ("qgemm_moe_run", _I, [_I, _VP, _I64, _I64, _I, _VP, _I64, _VP, _VP, _VP, _I64, _VP, _I, _VP,
                           _SZ, _VP]),
    ("qgemm_moe_gate_up", _I, [_I, _VP, _I64, _I64, _I, _VP, _I64, _VP, _VP, _VP, _VP, _VP, _VP,
                               _I64, _VP, _VP, _SZ, _VP]),
    ("qgemm_bs_split_size", _I, [_I, _I64, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ),
                                 ctypes.POINTER(_SZ)]),
    ("qgemm_bs_split_x", _I, [_I, _VP, _I64, _I64, _VP, _VP, _VP, _VP]),
    ("qgemm_bs_workspace_size", _I, [_I, _I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    ("qgemm_bs_run", _I, [_I, _VP, _I64, _I64, _VP, _VP, _VP, _I64, _VP, _I, _VP, _SZ, _VP]),
    ("qgemm_bs_ffn_workspace_size", _I, [_I, _I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    ("qgemm_bs_ffn_gate_up", _I, [_I, _VP, _I64, _I64, _VP, _VP, _VP, _VP, _VP, _VP, _I64, _VP,
                                  _VP, _SZ, _VP]),
    ("qgemm_moe_dispatch", _I, [_VP, _I, _I64, _I64, _VP, _I, _I, _VP, _VP, _VP, _VP]),
    ("qgemm_moe_dispatch_grad", _I, [_VP, _I, _I64, _I64, _VP, _I, _VP, _I, _VP]),
    ("qgemm_moe_combine", _I, [_VP, _I, _I64, _I64, _VP, _VP, _I, _VP, _I, _VP]),
    ("qgemm_moe_combine_grad", _I, [_VP, _I, _VP, _I, _I64, _I64, _VP, _VP, _I, _VP, _VP, _VP]),
    ("qgemm_i8_packed_size", _I, [_I64, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    ("qgemm_i8_pack", _I, [_VP, _I64, _I64, _VP, _VP, _VP]),
    ("qgemm_i8_repack_rowmajor", _I, [_I64, _I64, _VP, _I64, _VP, _VP]),
    ("qgemm_i8_quant_x", _I, [_VP, _I64, _I64, _VP, _VP, _VP]),
    ("qgemm_i8_workspace_size", _I, [_I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    ("qgemm_i8_run", _I, [_VP, _I64, _I64, _VP, _VP, _I64, _VP, _I, _VP, _SZ, _VP]),
    ("qgemm_i8_moe_workspace_size", _I, [_I64, _I64, _I64, ctypes.POINTER(_SZ)]),
    ("qgemm_i8_moe_run", _I, [_VP, _I64, _I64, _I, _VP, _I64, _VP, _VP, _I64, _VP, _I, _VP, _SZ,
                              _VP]),
    ("qgemm_i8_moe_gate_up", _I, [_VP, _I64, _I64, _I, _VP, _I64, _VP, _VP, _VP, _VP, _I64, _VP,
                                  _VP, _SZ, _VP]),
    ("qgemm_split_k", _I, [_I, _I64, _I64, ctypes.POINTER(_I)]),
    ("qgemm_device_status", _I, [_I]),
    ("qgemm_profile_events", _I, [_VP, _VP]),
    ("qgemm_status_str", ctypes.c_char_p, [_I]),
    ("qgemm_last_cuda_error", ctypes.c_char_p, []),
]


class QgemmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        lib = _lib
        detail = lib.qgemm_status_str(status).decode() if lib else ""
        cuda = lib.qgemm_last_cuda_error().decode() if (lib and status == 7) else ""
        super().__init__("%s: %s (%s)%s" % (where, STATUS.get(status, status), detail,
                                            (" -- " + cuda) if cuda else ""))


def lib():
    """The loaded library (raises if libqgemm.so is missing: build it first)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libqgemm.so not found at %s; run "
                                   "`python -m block_quantized_weight_qgemm_b200.build`" % LIB_PATH)
            handle = ctypes.CDLL(LIB_PATH)
            for name, res, args in SIGNATURES:
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
    return _lib


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def _check(status: int, where: str):
    if status != OK:
        raise QgemmError(status, where)


def _ptr(t):
    """Device address of a tensor (None for a missing or empty one)."""
    return None if (t is None or t.numel() == 0) else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ---- sizes -----------------------------------------------------------------------------

def packed_size(fmt, N: int, K: int):
    cb, sb = _SZ(), _SZ()
    _check(lib().qgemm_packed_size(_fmt(fmt), N, K, ctypes.byref(cb), ctypes.byref(sb)),
           "qgemm_packed_size")
    return cb.value, sb.value


def packed_geometry(fmt, N: int, K: int):
    """(row tiles T, chunks C, elements per chunk CK, scale bytes per row per chunk SB)."""
    t, c, ck, sb = _I64(), _I64(), _I(), _I()
    _check(lib().qgemm_packed_geometry(_fmt(fmt), N, K, ctypes.byref(t), ctypes.byref(c),
                                       ctypes.byref(ck), ctypes.byref(sb)), "qgemm_packed_geometry")
    return t.value, c.value, ck.value, sb.value


def row_pitches(fmt, K: int):
    cp, sp = _I64(), _I64()
    _check(lib().qgemm_row_pitches(_fmt(fmt), K, ctypes.byref(cp), ctypes.byref(sp)),
           "qgemm_row_pitches")
    return cp.value, sp.value


def workspace_size(fmt, N: int, K: int, B: int) -> int:
    b = _SZ()
    _check(lib().qgemm_workspace_size(_fmt(fmt), N, K, B, ctypes.byref(b)), "qgemm_workspace_size")
    return b.value


def ffn_workspace_size(fmt, N: int, K: int, M: int) -> int:
    b = _SZ()
    _check(lib().qgemm_ffn_workspace_size(_fmt(fmt), N, K, M, ctypes.byref(b)),
           "qgemm_ffn_workspace_size")
    return b.value


def split_k(fmt, N: int, K: int) -> int:
    s = _I()
    _check(lib().qgemm_split_k(_fmt(fmt), N, K, ctypes.byref(s)), "qgemm_split_k")
    return s.value


def device_status(reset: bool = True) -> int:
    return lib().qgemm_device_status(1 if reset else 0)


def profile_events(begin=None, end=None):
    """Record torch.cuda.Event `begin` / `end` around the next GEMM kernel launches."""
    lib().qgemm_profile_events(ctypes.c_void_p(begin.cuda_event) if begin is not None else None,
                               ctypes.c_void_p(end.cuda_event) if end is not None else None)


# ---- packed weights ---------------------------------------------------------------------

class PackedWeight:
    """Device buffers of one packed [N, K] matrix (codes, block scales -- empty for FP8 --
    and the fp32 tensor scale of NVFP4 and FP8)."""

    def __init__(self, fmt, N: int, K: int, device=None):
        self.fmt = _fmt(fmt)
        self.N, self.K = N, K
        device = device or torch.device("cuda", torch.cuda.current_device())
        cb, sb = packed_size(self.fmt, N, K)
        self.codes = torch.empty(cb, dtype=torch.uint8, device=device)   # tile-major layout
        self.scales = torch.empty(sb, dtype=torch.uint8, device=device)
        self.tensor_scale = (torch.empty(1, dtype=torch.float32, device=device)
                             if self.fmt in TENSOR_SCALE else None)

    @property
    def nbytes(self) -> int:
        """Algorithmic bytes a GEMM reads for this matrix (codes + scales, no row padding)."""
        code = self.N * (self.K if self.fmt in (Q8_0, FP8) else self.K // 2)
        if self.fmt == FP8:
            scale = 0
        else:
            scale = self.N * (2 * self.K // 32 if self.fmt == Q8_0 else self.K // BLOCK[self.fmt])
        return code + scale


def pack(fmt, W: torch.Tensor, stream=None, out: PackedWeight | None = None) -> PackedWeight:
    """qgemm_pack: W fp32 [N, K] on the device -> PackedWeight."""
    assert W.is_cuda and W.dtype == torch.float32 and W.is_contiguous()
    N, K = W.shape
    pw = out or PackedWeight(fmt, N, K, W.device)
    _check(lib().qgemm_pack(pw.fmt, _ptr(W), N, K, _ptr(pw.codes), _ptr(pw.scales),
                            _ptr(pw.tensor_scale), None, _stream(stream)), "qgemm_pack")
    return pw


def repack_rowmajor(fmt, codes_rm: torch.Tensor, scales_rm: torch.Tensor, N: int, K: int,
                    stream=None, out: PackedWeight | None = None) -> PackedWeight:
    """qgemm_repack_rowmajor: row-major interchange layout [N, pitch] -> PackedWeight."""
    assert codes_rm.is_cuda and scales_rm.is_cuda and codes_rm.dim() == 2 and scales_rm.dim() == 2
    pw = out or PackedWeight(fmt, N, K, codes_rm.device)
    spitch = scales_rm.stride(0) if scales_rm.numel() else 0
    _check(lib().qgemm_repack_rowmajor(pw.fmt, N, K, _ptr(codes_rm), codes_rm.stride(0),
                                       _ptr(scales_rm), spitch, _ptr(pw.codes),
                                       _ptr(pw.scales), _stream(stream)), "qgemm_repack_rowmajor")
    return pw


def run(x: torch.Tensor, pw: PackedWeight, y: torch.Tensor | None = None, y_dtype=torch.float32,
        workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qgemm_run: x bf16 [B, K] (device) -> y [B, N] (fp32 or bf16)."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 2
    B, K = x.shape
    assert K == pw.K
    if y is None:
        y = torch.empty((B, pw.N), dtype=y_dtype, device=x.device)
    ydt = Y_BF16 if y.dtype == torch.bfloat16 else Y_F32
    if workspace is None:
        nbytes = workspace_size(pw.fmt, pw.N, K, B)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_run(pw.fmt, _ptr(x), B, K, _ptr(pw.codes), _ptr(pw.scales),
                           _ptr(pw.tensor_scale), pw.N, _ptr(y), ydt, _ptr(workspace),
                           workspace.numel(), _stream(stream)), "qgemm_run")
    return y


def bs_split_size(fmt, M: int, K: int) -> tuple[int, int, int]:
    """qgemm_bs_split_size: (code bytes, scale bytes, exponent bytes) of the split of x for
    weight format fmt (MXFP4, NVFP4 or FP8)."""
    c, sc, e = _SZ(), _SZ(), _SZ()
    _check(lib().qgemm_bs_split_size(_fmt(fmt), M, K, ctypes.byref(c), ctypes.byref(sc),
                                     ctypes.byref(e)), "qgemm_bs_split_size")
    return c.value, sc.value, e.value


def bs_split_x(x: torch.Tensor, fmt="mxfp4", stream=None):
    """qgemm_bs_split_x: x bf16 [M, K] -> (codes u8, scales u8, x_exp int32) in the layout of
    include/qgemm.h (three E2M1 terms per row for MXFP4 / NVFP4, two E4M3 terms for FP8, with the
    MMA's block scales)."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 2
    M, K = x.shape
    nc, ns, ne = bs_split_size(fmt, M, K)
    codes = torch.empty(nc, dtype=torch.uint8, device=x.device)
    scales = torch.empty(ns, dtype=torch.uint8, device=x.device)
    x_exp = torch.empty(ne // 4, dtype=torch.int32, device=x.device)
    _check(lib().qgemm_bs_split_x(_fmt(fmt), _ptr(x), M, K, _ptr(codes), _ptr(scales),
                                  _ptr(x_exp), _stream(stream)), "qgemm_bs_split_x")
    return codes, scales, x_exp


def bs_workspace_size(fmt: int, N: int, K: int, M: int) -> int:
    n = _SZ()
    _check(lib().qgemm_bs_workspace_size(fmt, N, K, M, ctypes.byref(n)), "qgemm_bs_workspace_size")
    return n.value


def bs_run(x: torch.Tensor, pw: PackedWeight, y: torch.Tensor | None = None, y_dtype=torch.float32,
           workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qgemm_bs_run: the block-scaled path (MXFP4, NVFP4 or FP8 weights): x bf16 [M, K] -> y [M, N]."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 2
    M, K = x.shape
    assert K == pw.K
    if y is None:
        y = torch.empty((M, pw.N), dtype=y_dtype, device=x.device)
    ydt = Y_BF16 if y.dtype == torch.bfloat16 else Y_F32
    if workspace is None:
        nbytes = bs_workspace_size(pw.fmt, pw.N, K, M)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_bs_run(pw.fmt, _ptr(x), M, K, _ptr(pw.codes), _ptr(pw.scales),
                              _ptr(pw.tensor_scale), pw.N, _ptr(y), ydt, _ptr(workspace),
                              workspace.numel(), _stream(stream)), "qgemm_bs_run")
    return y


def bs_ffn_workspace_size(fmt, N: int, K: int, M: int) -> int:
    n = _SZ()
    _check(lib().qgemm_bs_ffn_workspace_size(_fmt(fmt), N, K, M, ctypes.byref(n)),
           "qgemm_bs_ffn_workspace_size")
    return n.value


def bs_ffn_gate_up(x: torch.Tensor, wg: PackedWeight, wu: PackedWeight, h: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qgemm_bs_ffn_gate_up: h = bf16(SiLU(x Wg^T) * (x Wu^T)) on the block-scaled path."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()
    M, K = x.shape
    assert wg.fmt == wu.fmt and wg.N == wu.N and wg.K == wu.K == K
    if h is None:
        h = torch.empty((M, wg.N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(bs_ffn_workspace_size(wg.fmt, wg.N, K, M), 16),
                                dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_bs_ffn_gate_up(wg.fmt, _ptr(x), M, K, _ptr(wg.codes), _ptr(wg.scales),
                                      _ptr(wg.tensor_scale), _ptr(wu.codes), _ptr(wu.scales),
                                      _ptr(wu.tensor_scale), wg.N, _ptr(h), _ptr(workspace),
                                      workspace.numel(), _stream(stream)), "qgemm_bs_ffn_gate_up")
    return h


def ffn_gate_up(x: torch.Tensor, wg: PackedWeight, wu: PackedWeight, h: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qgemm_ffn_gate_up: h = bf16(SiLU(x Wg^T) * (x Wu^T)), x bf16 [M, K] -> h bf16 [M, N]."""
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()
    M, K = x.shape
    assert wg.fmt == wu.fmt and wg.N == wu.N and wg.K == wu.K == K
    if h is None:
        h = torch.empty((M, wg.N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        nbytes = ffn_workspace_size(wg.fmt, wg.N, K, M)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_ffn_gate_up(wg.fmt, _ptr(x), M, K, _ptr(wg.codes), _ptr(wg.scales),
                                   _ptr(wg.tensor_scale), _ptr(wu.codes), _ptr(wu.scales),
                                   _ptr(wu.tensor_scale), wg.N, _ptr(h), _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "qgemm_ffn_gate_up")
    return h


# ---- routed mixture-of-experts --------------------------------------------------------

def moe_workspace_size(fmt, N: int, K: int, M: int, max_rows: int) -> int:
    b = _SZ()
    _check(lib().qgemm_moe_workspace_size(_fmt(fmt), N, K, M, max_rows, ctypes.byref(b)),
           "qgemm_moe_workspace_size")
    return b.value


class ExpertTable:
    """Device pointer tables of a list of packed experts (one PackedWeight each, same format
    and shape): codes, scales (absent for FP8) and tensor scales (NVFP4, FP8)."""

    def __init__(self, experts):
        assert experts and all(e.fmt == experts[0].fmt and e.N == experts[0].N and
                               e.K == experts[0].K for e in experts)
        self.fmt, self.N, self.K, self.E = experts[0].fmt, experts[0].N, experts[0].K, len(experts)
        dev = experts[0].codes.device

        def table(ts):
            return torch.tensor([t.data_ptr() for t in ts], dtype=torch.int64, device=dev)
        self.codes = table([e.codes for e in experts])
        self.scales = table([e.scales for e in experts]) if experts[0].scales.numel() else None
        self.ts = (table([e.tensor_scale for e in experts])
                   if experts[0].tensor_scale is not None else None)
        self.experts = experts  # keeps the buffers alive


def _moe_common(x, offsets, tab):
    assert x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous() and x.dim() == 2
    assert offsets.is_cuda and offsets.dtype == torch.int32 and offsets.numel() == tab.E + 1
    assert x.shape[1] == tab.K


def moe_run(x: torch.Tensor, offsets: torch.Tensor, tab: ExpertTable, max_rows: int,
            y: torch.Tensor | None = None, y_dtype=torch.float32, workspace=None, stream=None):
    """qgemm_moe_run: rows of x grouped by expert (int32 offsets[E+1] on the device)."""
    _moe_common(x, offsets, tab)
    M, K = x.shape
    if y is None:
        y = torch.empty((M, tab.N), dtype=y_dtype, device=x.device)
    ydt = Y_BF16 if y.dtype == torch.bfloat16 else Y_F32
    if workspace is None:
        nbytes = moe_workspace_size(tab.fmt, tab.N, K, M, max_rows)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_moe_run(tab.fmt, _ptr(x), M, K, tab.E, _ptr(offsets), max_rows,
                               _ptr(tab.codes), _ptr(tab.scales), _ptr(tab.ts), tab.N, _ptr(y), ydt,
                               _ptr(workspace), workspace.numel(), _stream(stream)), "qgemm_moe_run")
    return y


def moe_gate_up(x: torch.Tensor, offsets: torch.Tensor, gate: ExpertTable, up: ExpertTable,
                max_rows: int, h: torch.Tensor | None = None, workspace=None, stream=None):
    """qgemm_moe_gate_up: h = bf16(SiLU(x Wg_e^T) * (x Wu_e^T)) per routed row."""
    _moe_common(x, offsets, gate)
    assert gate.fmt == up.fmt and gate.N == up.N and gate.K == up.K and gate.E == up.E
    M, K = x.shape
    if h is None:
        h = torch.empty((M, gate.N), dtype=torch.bfloat16, device=x.device)
    if workspace is None:
        nbytes = moe_workspace_size(gate.fmt, gate.N, K, M, max_rows)
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_moe_gate_up(gate.fmt, _ptr(x), M, K, gate.E, _ptr(offsets), max_rows,
                                   _ptr(gate.codes), _ptr(gate.scales), _ptr(gate.ts),
                                   _ptr(up.codes), _ptr(up.scales), _ptr(up.ts), gate.N, _ptr(h),
                                   _ptr(workspace), workspace.numel(), _stream(stream)),
           "qgemm_moe_gate_up")
    return h


# ---- routed tokens: sorted by expert, and back --------------------------------------------
#
# These calls take a few microseconds on the device, so the marshalling is kept lean: integer
# addresses, one pass of checks, sizes remembered per shape.  A call on another device than the
# current one is made again with that device current (the library launches on the current device), one
# with a stream of its own with that stream current, so that what it allocates belongs to that stream.
#
# Like every call of this binding they are unknown to autograd: results carry no graph, whether or not
# the inputs require gradients.  A training step calls the gradients itself (from an autograd.Function of
# its own, say); those of the experts' products between combine and dispatch are its own as well.

_ROW_DTYPES = {torch.float32: Y_F32, torch.bfloat16: Y_BF16}

# torch's own accessors behind torch.cuda.current_device() and current_stream(), without the stream
# object (3 us); the device is initialised once a tensor lies on it.  A torch without them (built for
# the host alone) imports this module all the same, and has the public calls.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    def _raw_stream(i):
        return torch.cuda.current_stream(i).cuda_stream
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _device(*tensors) -> int:
    """The CUDA device of the tensors of a call, which all lie there and are contiguous."""
    i = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != i or not t.is_contiguous():
            raise AssertionError("the tensors of a call are contiguous and on one device")
    assert i >= 0, "the tensors of a call are on a CUDA device"
    return i


def _row_dtype(t) -> int:
    d = _ROW_DTYPES.get(t.dtype)
    assert d is not None, "rows are bf16 or fp32"
    return d


def _scratch(nbytes: int, like):
    """Device bytes for one call."""
    return like.new_empty(max(nbytes, 16), dtype=torch.uint8)


def _on(stream, t, call, *args, **kwargs):
    """`call` with `stream`, of t's device, as the current stream."""
    assert stream.device == t.device, "the stream and the tensors of a call are on one device"
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def _new(M, N, dtype, like):
    # (given its strides, torch makes a tensor in 1.5 us, without in 2.0 to 2.3)
    return torch.empty_strided((M, N), (N, 1), dtype=dtype, device=like.device)


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def moe_dispatch(x: torch.Tensor, experts: torch.Tensor, E: int, xs: torch.Tensor | None = None,
                 offsets: torch.Tensor | None = None, rows: torch.Tensor | None = None, stream=None):
    """qgemm_moe_dispatch: tokens x [T, H] (bf16 or fp32) and their experts int32 [T, k] (outside
    [0, E): none) -> (xs [T*k, H] sorted by expert, offsets int32 [E+1], rows int32 [T, k])."""
    if stream is not None:
        return _on(stream, x, moe_dispatch, x, experts, E, xs, offsets, rows)
    T, H = x.shape
    T2, k = experts.shape
    assert T2 == T and experts.dtype == torch.int32
    if xs is None:
        xs = _new(T * k, H, x.dtype, x)
    else:
        assert xs.dtype == x.dtype and xs.shape == (T * k, H)
    if offsets is None:
        offsets = experts.new_empty(E + 1)
    else:
        assert offsets.dtype == torch.int32 and offsets.numel() == E + 1
    if rows is None:
        rows = torch.empty_like(experts)
    else:
        assert rows.dtype == torch.int32 and rows.shape == experts.shape
    i = _device(x, experts, xs, offsets, rows)
    if i != _current_device():
        with torch.cuda.device(i):
            return moe_dispatch(x, experts, E, xs, offsets, rows)
    _check((_lib or lib()).qgemm_moe_dispatch(
        x.data_ptr(), _row_dtype(x), T, H, experts.data_ptr(), k, E, offsets.data_ptr(), rows.data_ptr(),
        xs.data_ptr(), _raw_stream(i)), "qgemm_moe_dispatch")
    return xs, offsets, rows


def _routed(a, rows):
    """(T, k, H) of sorted rows a [T*k, H] and their map [T, k]."""
    T, k = rows.shape
    S, H = a.shape
    assert S == T * k and rows.dtype == torch.int32
    return T, k, H


def _out(out, M, N, dtype, like):
    if out is None:
        return _new(M, N, dtype, like)
    assert out.shape == (M, N)
    return out


def moe_dispatch_grad(dxs: torch.Tensor, rows: torch.Tensor, dx: torch.Tensor | None = None,
                      dx_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """qgemm_moe_dispatch_grad: dx[t] = sum_j dxs[rows[t, j]], the gradient of moe_dispatch's x given that of
    its xs (which the caller takes from the experts' backward)."""
    if stream is not None:
        return _on(stream, dxs, moe_dispatch_grad, dxs, rows, dx, dx_dtype)
    T, k, H = _routed(dxs, rows)
    dx = _out(dx, T, H, dx_dtype, dxs)
    i = _device(dxs, rows, dx)
    if i != _current_device():
        with torch.cuda.device(i):
            return moe_dispatch_grad(dxs, rows, dx)
    _check((_lib or lib()).qgemm_moe_dispatch_grad(
        dxs.data_ptr(), _row_dtype(dxs), T, H, rows.data_ptr(), k, dx.data_ptr(), _row_dtype(dx),
        _raw_stream(i)), "qgemm_moe_dispatch_grad")
    return dx


def moe_combine(ys: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor,
                y: torch.Tensor | None = None, y_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """qgemm_moe_combine: y[t] = sum_j weights[t, j] * ys[rows[t, j]], weights fp32 [T, k]."""
    if stream is not None:
        return _on(stream, ys, moe_combine, ys, rows, weights, y, y_dtype)
    T, k, H = _routed(ys, rows)
    assert weights.dtype == torch.float32 and weights.shape == rows.shape
    y = _out(y, T, H, y_dtype, ys)
    i = _device(ys, rows, weights, y)
    if i != _current_device():
        with torch.cuda.device(i):
            return moe_combine(ys, rows, weights, y)
    _check((_lib or lib()).qgemm_moe_combine(
        ys.data_ptr(), _row_dtype(ys), T, H, rows.data_ptr(), weights.data_ptr(), k, y.data_ptr(), _row_dtype(y),
        _raw_stream(i)), "qgemm_moe_combine")
    return y


def moe_combine_grad(dy: torch.Tensor, ys: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor,
                     dys: torch.Tensor | None = None, dw: torch.Tensor | None = None, stream=None):
    """qgemm_moe_combine_grad: the gradients (dys [T*k, H] in ys's type, dw fp32 [T, k]) of
    moe_combine, given dy [T, H]."""
    if stream is not None:
        return _on(stream, dy, moe_combine_grad, dy, ys, rows, weights, dys, dw)
    T, k, H = _routed(ys, rows)
    assert weights.dtype == torch.float32 and weights.shape == rows.shape and dy.shape == (T, H)
    if dys is None:
        dys = torch.empty_like(ys)
    else:
        assert dys.dtype == ys.dtype and dys.shape == ys.shape
    if dw is None:
        dw = torch.empty_like(weights)
    else:
        assert dw.dtype == torch.float32 and dw.shape == rows.shape
    i = _device(dy, ys, rows, weights, dys, dw)
    if i != _current_device():
        with torch.cuda.device(i):
            return moe_combine_grad(dy, ys, rows, weights, dys, dw)
    _check((_lib or lib()).qgemm_moe_combine_grad(
        dy.data_ptr(), _row_dtype(dy), ys.data_ptr(), _row_dtype(ys), T, H, rows.data_ptr(), weights.data_ptr(), k,
        dys.data_ptr(), dw.data_ptr(), _raw_stream(i)),
        "qgemm_moe_combine_grad")
    return dys, dw


# ---- int8 weights and activations ---------------------------------------------------------

def i8_packed_size(N: int, K: int):
    cb, sb = _SZ(), _SZ()
    _check(lib().qgemm_i8_packed_size(N, K, ctypes.byref(cb), ctypes.byref(sb)), "qgemm_i8_packed_size")
    return cb.value, sb.value


class I8Weight:
    """Device buffers of one int8 [N, K] matrix: tile-major codes, fp32 scales [N]."""

    def __init__(self, N: int, K: int, device=None):
        self.N, self.K = N, K
        device = device or torch.device("cuda", torch.cuda.current_device())
        self.codes = torch.empty(i8_packed_size(N, K)[0], dtype=torch.uint8, device=device)
        self.scales = torch.empty(N, dtype=torch.float32, device=device)

    @property
    def nbytes(self) -> int:
        """Algorithmic bytes a GEMM reads for this matrix (codes + scales, no padding)."""
        return self.N * self.K + 4 * self.N


def i8_pack(W: torch.Tensor, out: I8Weight | None = None, stream=None) -> I8Weight:
    """qgemm_i8_pack: W fp32 [N, K] on the device -> I8Weight."""
    if stream is not None:
        return _on(stream, W, i8_pack, W, out)
    N, K = W.shape
    assert W.dtype == torch.float32
    w = out or I8Weight(N, K, W.device)
    assert (w.N, w.K) == (N, K)
    i = _device(W, w.codes, w.scales)
    if i != _current_device():
        with torch.cuda.device(i):
            return i8_pack(W, w)
    _check(lib().qgemm_i8_pack(W.data_ptr(), N, K, w.codes.data_ptr(), w.scales.data_ptr(),
                               _raw_stream(i)), "qgemm_i8_pack")
    return w


def i8_repack_rowmajor(codes_rm: torch.Tensor, scales: torch.Tensor, out: I8Weight | None = None,
                       stream=None) -> I8Weight:
    """qgemm_i8_repack_rowmajor: a checkpoint's int8 codes [N, K] (rows may be strided) and fp32
    scales [N] -> I8Weight.  Both are copied; with `out`, into its buffers, which tables and captured
    graphs may hold the addresses of."""
    if stream is not None:
        return _on(stream, codes_rm, i8_repack_rowmajor, codes_rm, scales, out)
    N, K = codes_rm.shape
    assert codes_rm.dtype == torch.int8 and (codes_rm.stride(1) == 1 or K == 1)
    assert scales.dtype == torch.float32 and scales.shape == (N,)
    w = out or I8Weight(N, K, codes_rm.device)
    assert (w.N, w.K) == (N, K) and codes_rm.get_device() == scales.get_device()
    i = _device(w.codes, w.scales, scales)
    if i != _current_device():
        with torch.cuda.device(i):
            return i8_repack_rowmajor(codes_rm, scales, w)
    _check(lib().qgemm_i8_repack_rowmajor(N, K, codes_rm.data_ptr(), codes_rm.stride(0) if N > 1 else K,
                                          w.codes.data_ptr(),
                                          _raw_stream(i)),
           "qgemm_i8_repack_rowmajor")
    with torch.inference_mode():  # (plain bytes, whatever mode or graph either tensor was made in)
        w.scales.copy_(scales)
    return w


def i8_quant_x(x: torch.Tensor, codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
               stream=None):
    """qgemm_i8_quant_x: x bf16 [M, K] -> (codes int8 [M, K], scales fp32 [M])."""
    if stream is not None:
        return _on(stream, x, i8_quant_x, x, codes, scales)
    M, K = x.shape
    assert x.dtype == torch.bfloat16
    if codes is None:
        codes = _new(M, K, torch.int8, x)
    else:
        assert codes.dtype == torch.int8 and codes.shape == (M, K)
    if scales is None:
        scales = x.new_empty(M, dtype=torch.float32)
    else:
        assert scales.dtype == torch.float32 and scales.shape == (M,)
    i = _device(x, codes, scales)
    if i != _current_device():
        with torch.cuda.device(i):
            return i8_quant_x(x, codes, scales)
    _check((_lib or lib()).qgemm_i8_quant_x(x.data_ptr(), M, K, codes.data_ptr(), scales.data_ptr(),
                                            _raw_stream(i)),
           "qgemm_i8_quant_x")
    return codes, scales


@functools.lru_cache(maxsize=256)
def i8_workspace_size(N: int, K: int, M: int) -> int:
    """Bytes of workspace that is enough for every i8_run of at most M rows."""
    b = _SZ()
    _check(lib().qgemm_i8_workspace_size(N, K, M, ctypes.byref(b)), "qgemm_i8_workspace_size")
    return b.value


def i8_run(x: torch.Tensor, w: I8Weight, y: torch.Tensor | None = None, y_dtype=torch.float32,
           workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """qgemm_i8_run: x bf16 [M, K], quantised per row on the fly -> y [M, N] (fp32 or bf16)."""
    if stream is not None:
        return _on(stream, x, i8_run, x, w, y, y_dtype, workspace)
    M, K = x.shape
    N, codes, scales = w.N, w.codes, w.scales
    assert x.dtype == torch.bfloat16 and K == w.K
    y = _out(y, M, N, y_dtype, x)
    ws, nbytes = None, 0
    if workspace is not None:
        ws, nbytes = workspace.data_ptr(), _nbytes(workspace)
    else:
        nbytes = i8_workspace_size(N, K, M)
        if nbytes:
            workspace = _scratch(nbytes, x)
            ws = workspace.data_ptr()
    i = _device(x, codes, scales, y, x if workspace is None else workspace)
    if i != _current_device():
        with torch.cuda.device(i):
            return i8_run(x, w, y, workspace=workspace)
    _check((_lib or lib()).qgemm_i8_run(
        x.data_ptr(), M, K, codes.data_ptr(), scales.data_ptr(), N, y.data_ptr(), _row_dtype(y), ws, nbytes,
        _raw_stream(i)), "qgemm_i8_run")
    return y


class I8ExpertTable:
    """Device pointer tables of a list of int8 experts (one I8Weight each, same shape)."""

    def __init__(self, experts):
        assert experts and all((e.N, e.K) == (experts[0].N, experts[0].K) and
                               e.codes.device == experts[0].codes.device for e in experts)
        self.N, self.K, self.E = experts[0].N, experts[0].K, len(experts)
        dev = experts[0].codes.device
        self.codes = torch.tensor([e.codes.data_ptr() for e in experts], dtype=torch.int64, device=dev)
        self.scales = torch.tensor([e.scales.data_ptr() for e in experts], dtype=torch.int64, device=dev)
        self.experts = experts
        self.buffers = [(e.codes, e.scales) for e in experts]  # the addresses' tensors, kept alive


@functools.lru_cache(maxsize=256)
def i8_moe_workspace_size(N: int, K: int, M: int) -> int:
    """Bytes of workspace that is enough for every routed call of at most M rows."""
    b = _SZ()
    _check(lib().qgemm_i8_moe_workspace_size(N, K, M, ctypes.byref(b)), "qgemm_i8_moe_workspace_size")
    return b.value


def _i8_moe(x, offsets, tab, workspace):
    """(M, K, workspace) of a routed int8 call."""
    M, K = x.shape
    assert x.dtype == torch.bfloat16 and K == tab.K
    assert offsets.dtype == torch.int32 and offsets.numel() == tab.E + 1
    if workspace is None:
        workspace = _scratch(i8_moe_workspace_size(tab.N, K, M), x)
    return M, K, workspace


def i8_moe_run(x: torch.Tensor, offsets: torch.Tensor, tab: I8ExpertTable, max_rows: int,
               y: torch.Tensor | None = None, y_dtype=torch.float32, workspace=None, stream=None):
    """qgemm_i8_moe_run: rows of x grouped by expert (int32 offsets[E+1] on the device)."""
    if stream is not None:
        return _on(stream, x, i8_moe_run, x, offsets, tab, max_rows, y, y_dtype, workspace)
    M, K, workspace = _i8_moe(x, offsets, tab, workspace)
    y = _out(y, M, tab.N, y_dtype, x)
    i = _device(x, offsets, tab.codes, y, workspace)
    if i != _current_device():
        with torch.cuda.device(i):
            return i8_moe_run(x, offsets, tab, max_rows, y, workspace=workspace)
    _check((_lib or lib()).qgemm_i8_moe_run(
        x.data_ptr(), M, K, tab.E, offsets.data_ptr(), max_rows, tab.codes.data_ptr(), tab.scales.data_ptr(), tab.N,
        y.data_ptr(), _row_dtype(y), workspace.data_ptr(), _nbytes(workspace),
        _raw_stream(i)), "qgemm_i8_moe_run")
    return y


def i8_moe_gate_up(x: torch.Tensor, offsets: torch.Tensor, gate: I8ExpertTable, up: I8ExpertTable,
                   max_rows: int, h: torch.Tensor | None = None, workspace=None, stream=None):
    """qgemm_i8_moe_gate_up: h = bf16(SiLU(g) * u) per routed row."""
    if stream is not None:
        return _on(stream, x, i8_moe_gate_up, x, offsets, gate, up, max_rows, h, workspace)
    M, K, workspace = _i8_moe(x, offsets, gate, workspace)
    assert (gate.N, gate.K, gate.E) == (up.N, up.K, up.E)
    h = _out(h, M, gate.N, torch.bfloat16, x)
    assert h.dtype == torch.bfloat16
    i = _device(x, offsets, gate.codes, up.codes, h, workspace)
    if i != _current_device():
        with torch.cuda.device(i):
            return i8_moe_gate_up(x, offsets, gate, up, max_rows, h, workspace)
    _check((_lib or lib()).qgemm_i8_moe_gate_up(
        x.data_ptr(), M, K, gate.E, offsets.data_ptr(), max_rows, gate.codes.data_ptr(), gate.scales.data_ptr(),
        up.codes.data_ptr(), up.scales.data_ptr(), gate.N, h.data_ptr(), workspace.data_ptr(), _nbytes(workspace),
        _raw_stream(i)), "qgemm_i8_moe_gate_up")
    return h
