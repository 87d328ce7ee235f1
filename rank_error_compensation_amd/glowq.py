"""Thin ctypes binding of libglowq (include/glowq.h).

Argument marshalling only: every step of the path runs in the library's HIP kernels.  torch is
used for device memory and the current stream (plumbing); tensors are passed as raw pointers.
There is no fallback: if the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libglowq.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_SHAPE = -2
ERR_ALIGN = -3
ERR_UNSUPPORTED = -4
ERR_WORKSPACE = -5
ERR_HIP = -6
ERR_RANGE = -7
ERR_HANDOFF = -8
ERR_ROUTING = -9
MOE_SHARE_EXPERT = 0
MOE_SHARE_ALL = 1
FMT_INT4_G128 = 0
FMT_MXFP4 = 1
FMT_MXFP6_E2M3 = 2
FMT_MXFP6_E3M2 = 3
FMT_INT8_CHANNEL = 4
FMT_FP8_BLOCK = 5
FORMATS = {"int4": FMT_INT4_G128, "mxfp4": FMT_MXFP4, "mxfp6_e2m3": FMT_MXFP6_E2M3, "mxfp6_e3m2": FMT_MXFP6_E3M2}

DTYPE_F32 = 0
DTYPE_F16 = 1
SCORES = {"softmax": 0, "sigmoid": 1}
UNIT_GROUP = 0
UNIT_SOLO = 1
MAX_MODULES = 8

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t


class QWeightC(ctypes.Structure):
    _fields_ = [("q", _vp), ("sz", _vp), ("n_out", _i64), ("k_in", _i64), ("format", _i32), ("reserved", _i32)]


class MoeModuleC(ctypes.Structure):
    _fields_ = [("q", _vp), ("sz", _vp), ("a", _vp), ("y", _vp), ("n_out", _i64), ("k_in", _i64)]


class UnitC(ctypes.Structure):
    _fields_ = [("kind", _i32), ("m", _i32), ("x", _vp), ("T", _i64), ("d", _i64),
                ("w", ctypes.POINTER(QWeightC)), ("b", _vp), ("a", ctypes.POINTER(_vp)),
                ("r", _i32), ("restore", _i32), ("y", ctypes.POINTER(_vp))]


EXPORTS = {
    "glowq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "glowq_version": (ctypes.c_int, []),
    "glowq_q_bytes": (_sz, [_i64, _i64]),
    "glowq_sz_bytes": (_sz, [_i64, _i64]),
    "glowq_repack": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "glowq_mx_q_bytes": (_sz, [_i32, _i64, _i64]),
    "glowq_repack_mx": (ctypes.c_int, [_i32, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "glowq_dequant": (ctypes.c_int, [ctypes.POINTER(QWeightC), _vp, _i32, _vp]),
    "glowq_workspace_bytes": (_sz, [_i64, _i32, _i32]),
    "glowq_workspace_init": (ctypes.c_int, [_vp, _sz, _vp]),
    "glowq_workspace_status": (ctypes.c_int, [_vp, _sz, _vp]),
    "glowq_group_forward": (ctypes.c_int, [_vp, _i64, _i64, _i32, ctypes.POINTER(QWeightC), _vp,
                                           ctypes.POINTER(_vp), _i32, _i32, _vp, _sz,
                                           ctypes.POINTER(_vp), _vp]),
    "glowq_static_scratch_bytes": (_sz, []),
    "glowq_group_forward_static": (ctypes.c_int, [_vp, _i64, _i64, _i32, ctypes.POINTER(QWeightC), _vp,
                                                  ctypes.POINTER(_vp), _i32, _i32, ctypes.POINTER(_vp), _vp]),
    "glowq_w4a8_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "glowq_mx8_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "glowq_group_forward_w4a8": (ctypes.c_int, [_vp, _i64, _i64, _i32, ctypes.POINTER(QWeightC), _vp,
                                                ctypes.POINTER(_vp), _i32, _i32, _vp, _sz, ctypes.POINTER(_vp), _vp]),
    "glowq_group_forward_mx8": (ctypes.c_int, [_vp, _i64, _i64, _i32, ctypes.POINTER(QWeightC), _vp,
                                                ctypes.POINTER(_vp), _i32, _i32, _vp, _sz, ctypes.POINTER(_vp), _vp]),
    "glowq_w8_q_bytes": (_sz, [_i64, _i64]),
    "glowq_w8_sz_bytes": (_sz, [_i64]),
    "glowq_repack_w8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "glowq_w8a8_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    # host arrays as addresses (packed bytes or ctypes arrays)
    "glowq_group_forward_w8a8": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _sz, _vp, _vp]),
    "glowq_fp8_q_bytes": (_sz, [_i64, _i64]),
    "glowq_fp8_sz_bytes": (_sz, [_i64, _i64]),
    "glowq_repack_fp8": (ctypes.c_int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "glowq_fp8_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "glowq_group_forward_fp8": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _i32, _i32, _vp, _sz, _vp, _vp]),
    "glowq_moe_fp8_workspace_bytes": (_sz, [_i64, _i64, _i64, _i32, _i32]),
    "glowq_moe_forward_fp8": (ctypes.c_int, [_vp, _i64, _i64, _i32, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _i64, _vp,
                                             _sz, _vp]),
    "glowq_moe_sort_workspace_bytes": (_sz, [_i64, _i64, _i32]),
    "glowq_moe_sort": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "glowq_moe_dispatch": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _sz, _vp]),
    "glowq_moe_combine": (ctypes.c_int, [_vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _sz, _vp]),
    "glowq_moe_combine_backward": (ctypes.c_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp,
                                                  _sz, _vp]),
    "glowq_moe_combine_backward_whole": (ctypes.c_int, [_vp, _vp, _i64, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _vp, _vp,
                                                        _vp, _sz, _vp]),
    "glowq_moe_route": (ctypes.c_int, [_vp, _i64, _i32, _i64, _i32, _i32, _vp, _i32, _i32, _i32, _i32, ctypes.c_float, _vp,
                                       _vp, _vp, _sz, _vp]),
    "glowq_moe_route_backward": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _i64, _i32, _i32, _i32, ctypes.c_float, _vp, _vp,
                                                _sz, _vp]),
    "glowq_layer_norm": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, ctypes.c_float, _i32, _vp, _vp, _vp, _vp]),
    "glowq_layer_norm_workspace_bytes": (_sz, [_i64, _i64]),
    "glowq_layer_norm_backward": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "glowq_swiglu": (ctypes.c_int, [_vp, _vp, _i64, _i32, _vp, _vp]),
    "glowq_swiglu_backward": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, _vp, _vp, _vp]),
    "glowq_moe_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32]),
    "glowq_moe_forward": (ctypes.c_int, [_vp, _i64, _i64, _i32, _i32, ctypes.POINTER(MoeModuleC), _vp, _i32, _i32,
                                         _i32, _vp, _vp, _i64, _vp, _sz, _vp]),
    "glowq_solo_forward": (ctypes.c_int, [_vp, _i64, _i64, ctypes.POINTER(QWeightC), _vp, _vp, _i32,
                                          _i32, _vp, _sz, _vp, _vp]),
    "glowq_layerwise_forward": (ctypes.c_int, [_vp, _i64, _i64, _i32, ctypes.POINTER(QWeightC),
                                               ctypes.POINTER(_vp), ctypes.POINTER(_vp), _i32, _i32,
                                               _vp, _sz, ctypes.POINTER(_vp), _vp]),
    "glowq_path_forward": (ctypes.c_int, [ctypes.POINTER(UnitC), _i32, _vp, _sz, _vp]),
    "glowq_ner_workspace_bytes": (_sz, [_i64]),
    "glowq_ner_sums": (ctypes.c_int, [_vp, ctypes.POINTER(QWeightC), _vp, _sz, _vp, _vp]),
    "glowq_ner_sums_batch": (ctypes.c_int, [_i32, ctypes.POINTER(_vp), ctypes.POINTER(QWeightC), _vp, _sz,
                                            _vp, _vp]),
    "glowq_restore_topk": (ctypes.c_int, [_vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "glowq_restore_select": (ctypes.c_int, [_vp, _i32, _i32, _i32, ctypes.c_double, _vp, _vp, _vp]),
    "glowq_second_moment_workspace_bytes": (_sz, [_i64, _i64]),
    "glowq_second_moment": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _sz, _vp]),
    "glowq_solve_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32]),
    "glowq_solve_factors": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz,
                                           _vp]),
    "glowq_ec_score_workspace_bytes": (_sz, [_i64, _i64]),
    "glowq_ec_score": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _i32, _vp, _vp, _sz, _vp]),
}

_lib = None


def lib():
    """Load libglowq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build the HIP library first "
                               "(python -m rank_error_compensation_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


class GlowQError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {lib().glowq_status_string(status).decode()} ({status})")


def check(status: int, what: str) -> None:
    if status != OK:
        raise GlowQError(status, what)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _require(cond: bool, status: int, what: str) -> None:
    if not cond:
        raise GlowQError(status, what)


_DTYPES = {torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}


def _same_place(what: str, first: torch.Tensor, *others) -> None:
    """Dense GPU tensors of one device (None allowed among the others)."""
    dev = first.get_device() if first.is_cuda else -1
    if dev < 0 or not first.is_contiguous():
        raise GlowQError(ERR_INVALID_ARG, f"{what}: dense GPU tensors")
    for t in others:
        if t is not None and (t.get_device() != dev or not t.is_contiguous()):
            raise GlowQError(ERR_INVALID_ARG, f"{what}: dense tensors on one device")


def _elsewhere(t: torch.Tensor, stream):
    """None where the call can go to the current stream of the current device; else the context that
    makes the tensors' device, or the given stream, current -- so that what the call allocates belongs
    to the stream that uses it."""
    if stream is not None:
        _require(stream.device == t.device, ERR_INVALID_ARG, "stream of another device than the tensors")
        return torch.cuda.stream(stream)
    return torch.cuda.device(t.device) if t.get_device() != torch.cuda.current_device() else None


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(t: torch.Tensor) -> int:
    """Handle of the current stream of the tensor's device."""
    dev = t.get_device()
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


# --------------------------------------------------------------------------- weights
@dataclass
class QWeight:
    """One module (INT4-g128 or MX) in the library's device layout."""
    q: torch.Tensor     # uint8, glowq_q_bytes (MX: glowq_mx_q_bytes)
    sz: torch.Tensor    # uint8, glowq_sz_bytes
    n_out: int
    k_in: int
    fmt: int = FMT_INT4_G128

    def c(self) -> QWeightC:
        return QWeightC(self.q.data_ptr(), self.sz.data_ptr(), self.n_out, self.k_in, self.fmt, 0)

    @staticmethod
    def from_mx(fmt, codes: torch.Tensor, scales: torch.Tensor, device=None, stream=None) -> "QWeight":
        """Repack MX codes (uint8 [n_out][k_in], one code per byte) and E8M0 scales (uint8
        [n_out][k_in/32]) into the device layout (glowq_repack_mx; synchronises the stream)."""
        device = device or torch.device("cuda")
        f = FORMATS[fmt] if isinstance(fmt, str) else int(fmt)
        n_out, k_in = codes.shape
        c = codes.to(device=device, dtype=torch.uint8).contiguous()
        s = scales.to(device=device, dtype=torch.uint8).contiguous()
        L = lib()
        qb, zb = L.glowq_mx_q_bytes(f, n_out, k_in), L.glowq_sz_bytes(n_out, k_in)
        if qb == 0 or zb == 0:
            raise GlowQError(ERR_SHAPE, "glowq_mx_q_bytes")
        q_dev = torch.empty(qb, dtype=torch.uint8, device=device)
        sz_dev = torch.empty(zb, dtype=torch.uint8, device=device)
        flag = torch.empty(1, dtype=torch.int32, device=device)
        check(L.glowq_repack_mx(f, _ptr(c), _ptr(s), n_out, k_in, _ptr(q_dev), _ptr(sz_dev), _ptr(flag),
                                _stream(stream)), "glowq_repack_mx")
        return QWeight(q_dev, sz_dev, int(n_out), int(k_in), f)

    @staticmethod
    def from_canonical(q_packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor,
                       device=None, stream=None) -> "QWeight":
        """Repack canonical (q_packed int32 [n_out][k_in/8], scales/zeros fp16 [n_out][k_in/128])
        into the device layout (glowq_repack; synchronises the stream)."""
        device = device or torch.device("cuda")
        n_out, kw = q_packed.shape
        k_in = kw * 8
        qc = q_packed.to(device).contiguous()
        s = scales.to(device=device, dtype=torch.float16).contiguous()
        z = zeros.to(device=device, dtype=torch.float16).contiguous()
        L = lib()
        qb, zb = L.glowq_q_bytes(n_out, k_in), L.glowq_sz_bytes(n_out, k_in)
        if qb == 0 or zb == 0:
            raise GlowQError(ERR_SHAPE, "glowq_q_bytes")
        q_dev = torch.empty(qb, dtype=torch.uint8, device=device)
        sz_dev = torch.empty(zb, dtype=torch.uint8, device=device)
        flag = torch.empty(1, dtype=torch.int32, device=device)
        check(L.glowq_repack(_ptr(qc), _ptr(s), _ptr(z), n_out, k_in, _ptr(q_dev), _ptr(sz_dev),
                             _ptr(flag), _stream(stream)), "glowq_repack")
        return QWeight(q_dev, sz_dev, int(n_out), int(k_in))

    @staticmethod
    def from_int8(codes: torch.Tensor, scales: torch.Tensor, device=None, stream=None) -> "QWeight":
        """Repack 8-bit integer codes (int8 [n_out][k_in]) and per-row scales (fp32 [n_out]) into the
        device layout of group_forward_w8a8 (glowq_repack_w8; synchronises the stream)."""
        device = torch.device("cuda" if device is None else device)
        _require(codes.dim() == 2 and codes.dtype == torch.int8 and scales.dtype == torch.float32, ERR_INVALID_ARG,
                 "from_int8: int8 codes [n_out][k_in], fp32 scales [n_out]")
        _require(tuple(scales.shape) == (codes.shape[0],), ERR_SHAPE, "from_int8: one scale per row")
        n_out, k_in = (int(n) for n in codes.shape)
        L = lib()
        qb, zb = L.glowq_w8_q_bytes(n_out, k_in), L.glowq_w8_sz_bytes(n_out)
        if qb == 0 or zb == 0:
            raise GlowQError(ERR_SHAPE, "glowq_w8_q_bytes")
        _require(device.type == "cuda", ERR_INVALID_ARG, "from_int8: a GPU device")
        _require(stream is None or device.index is None or stream.device == device, ERR_INVALID_ARG,
                 "from_int8: stream of another device")
        # copies, allocations and the repack all on the one stream
        with torch.cuda.device(device) if stream is None else torch.cuda.stream(stream):
            c, s = codes.to(device).contiguous(), scales.to(device).contiguous()
            q_dev = torch.empty(qb, dtype=torch.uint8, device=c.device)
            sz_dev = torch.empty(zb, dtype=torch.uint8, device=c.device)
            flag = torch.empty(1, dtype=torch.int32, device=c.device)
            check(L.glowq_repack_w8(_ptr(c), _ptr(s), n_out, k_in, _ptr(q_dev), _ptr(sz_dev), _ptr(flag),
                                    _stream(stream)), "glowq_repack_w8")
        return QWeight(q_dev, sz_dev, n_out, k_in, FMT_INT8_CHANNEL)

    @staticmethod
    def from_fp8(codes: torch.Tensor, scales: torch.Tensor, device=None, stream=None) -> "QWeight":
        """Repack e4m3 codes (torch.float8_e4m3fn, or their bytes as uint8, [n_out][k_in]) and the scales of their
        128 x 128 blocks (fp32 [ceil(n_out / 128)][k_in / 128]) into the device layout of group_forward_fp8
        (glowq_repack_fp8; synchronises the stream)."""
        device = torch.device("cuda" if device is None else device)
        _require(codes.dim() == 2 and codes.dtype in (torch.float8_e4m3fn, torch.uint8) and scales.dtype == torch.float32,
                 ERR_INVALID_ARG, "from_fp8: e4m3 codes [n_out][k_in], fp32 scales [ceil(n_out / 128)][k_in / 128]")
        n_out, k_in = (int(n) for n in codes.shape)
        L = lib()
        qb, zb = L.glowq_fp8_q_bytes(n_out, k_in), L.glowq_fp8_sz_bytes(n_out, k_in)
        if qb == 0 or zb == 0:
            raise GlowQError(ERR_SHAPE, "glowq_fp8_q_bytes")
        _require(tuple(scales.shape) == (-(-n_out // 128), k_in // 128), ERR_SHAPE, "from_fp8: one scale per 128 x 128 block")
        _require(device.type == "cuda", ERR_INVALID_ARG, "from_fp8: a GPU device")
        _require(stream is None or device.index is None or stream.device == device, ERR_INVALID_ARG,
                 "from_fp8: stream of another device")
        # copies, allocations and the repack all on the one stream
        with torch.cuda.device(device) if stream is None else torch.cuda.stream(stream):
            c, s = codes.to(device).contiguous(), scales.to(device).contiguous()
            q_dev = torch.empty(qb, dtype=torch.uint8, device=c.device)
            sz_dev = torch.empty(zb, dtype=torch.uint8, device=c.device)
            flag = torch.empty(1, dtype=torch.int32, device=c.device)
            check(L.glowq_repack_fp8(_ptr(c), _ptr(s), n_out, k_in, _ptr(q_dev), _ptr(sz_dev), _ptr(flag),
                                     _stream(stream)), "glowq_repack_fp8")
        return QWeight(q_dev, sz_dev, n_out, k_in, FMT_FP8_BLOCK)

    @staticmethod
    def from_workload(qw, device=None, stream=None) -> "QWeight":
        if getattr(qw, "fmt", "int4") != "int4":
            return QWeight.from_mx(qw.fmt, qw.codes, qw.scales, device, stream)
        return QWeight.from_canonical(qw.q_packed, qw.s, qw.z, device, stream)


def dequant(w: QWeight, dtype=torch.float32, stream=None) -> torch.Tensor:
    out = torch.empty(w.n_out, w.k_in, dtype=dtype, device=w.q.device)
    code = DTYPE_F32 if dtype == torch.float32 else DTYPE_F16
    wc = w.c()
    check(lib().glowq_dequant(ctypes.byref(wc), _ptr(out), code, _stream(stream)), "glowq_dequant")
    return out


# --------------------------------------------------------------------------- restore selection
def ner_sums(w: torch.Tensor, qw: QWeight, out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp64 [2]: ||W - W_hat||_F^2 and ||W||_F^2 of one module (glowq_ner_sums); `out` may be a
    16-byte aligned fp64 view of two elements."""
    w = w.contiguous()
    if out is None:
        out = torch.empty(2, dtype=torch.float64, device=w.device)
    if workspace is None:
        workspace = torch.empty(int(lib().glowq_ner_workspace_bytes(qw.n_out)), dtype=torch.uint8,
                                device=w.device)
    wc = qw.c()
    check(lib().glowq_ner_sums(_ptr(w), ctypes.byref(wc), _ptr(workspace), workspace.numel(), _ptr(out),
                               _stream(stream)), "glowq_ner_sums")
    return out


def ner_workspace_bytes_batch(n_outs: Sequence[int]) -> int:
    return int(sum(lib().glowq_ner_workspace_bytes(n) for n in n_outs))


def ner_sums_batch(ws_and_qws: Sequence, out: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp64 [n][2] pairs of glowq_ner_sums for (fp16 W, QWeight) pairs, in one batch call."""
    items = [(w.contiguous(), qw) for w, qw in ws_and_qws]
    dev = items[0][0].device
    if out is None:
        out = torch.empty(len(items), 2, dtype=torch.float64, device=dev)
    if workspace is None:
        workspace = torch.empty(ner_workspace_bytes_batch([qw.n_out for _, qw in items]), dtype=torch.uint8,
                                device=dev)
    wp = _arr(_vp, [w.data_ptr() for w, _ in items])
    wc = _arr(QWeightC, [qw.c() for _, qw in items])
    check(lib().glowq_ner_sums_batch(len(items), wp, wc, _ptr(workspace), workspace.numel(), _ptr(out),
                                     _stream(stream)), "glowq_ner_sums_batch")
    return out


def restore_select(sums: torch.Tensor, k: int, rel_tol: float, stream=None):
    """glowq_restore_select: (scores fp64 [n_units], mask int32 [n_units]) with the layer-order
    fallback for scores within rel_tol steps of the best."""
    sums = sums.contiguous()
    n_units, n_per = int(sums.shape[0]), int(sums.shape[1])
    scores = torch.empty(n_units, dtype=torch.float64, device=sums.device)
    mask = torch.empty(n_units, dtype=torch.int32, device=sums.device)
    check(lib().glowq_restore_select(_ptr(sums), n_units, n_per, k, float(rel_tol), _ptr(scores), _ptr(mask),
                                     _stream(stream)), "glowq_restore_select")
    return scores, mask


def restore_topk(sums: torch.Tensor, k: int, stream=None):
    """sums fp64 [n_units][n_per_unit][2] -> (scores fp64 [n_units], mask int32 [n_units])."""
    sums = sums.contiguous()
    n_units, n_per = int(sums.shape[0]), int(sums.shape[1])
    scores = torch.empty(n_units, dtype=torch.float64, device=sums.device)
    mask = torch.empty(n_units, dtype=torch.int32, device=sums.device)
    check(lib().glowq_restore_topk(_ptr(sums), n_units, n_per, k, _ptr(scores), _ptr(mask),
                                   _stream(stream)), "glowq_restore_topk")
    return scores, mask


# --------------------------------------------------------------------------- offline factor solve
def second_moment(x: torch.Tensor, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp32 [d][d] Sigma_x = X^T X / N of fp16 calibration activations x [N][d]."""
    x = x.contiguous()
    N, d = int(x.shape[0]), int(x.shape[1])
    if out is None:
        out = torch.empty(d, d, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(int(lib().glowq_second_moment_workspace_bytes(N, d)), dtype=torch.uint8,
                                device=x.device)
    check(lib().glowq_second_moment(_ptr(x), N, d, _ptr(out), _ptr(workspace), workspace.numel(),
                                    _stream(stream)), "glowq_second_moment")
    return out


def solve_factors(e: torch.Tensor, sigma: torch.Tensor, omega: torch.Tensor, r: int, q: int = 0,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """fp64 stacked errors e [m][d], Sigma_x [d][d], test matrix omega [d][k] -> (A [m][r],
    B [r][d], S [r]) (glowq_solve_factors; synchronises the stream)."""
    e, sigma, omega = e.contiguous(), sigma.contiguous(), omega.contiguous()
    m, d = int(e.shape[0]), int(e.shape[1])
    k = int(omega.shape[1])
    A = torch.empty(m, r, dtype=torch.float64, device=e.device)
    B = torch.empty(r, d, dtype=torch.float64, device=e.device)
    S = torch.empty(r, dtype=torch.float64, device=e.device)
    if workspace is None:
        workspace = torch.empty(int(lib().glowq_solve_workspace_bytes(m, d, k, r)), dtype=torch.uint8, device=e.device)
    check(lib().glowq_solve_factors(_ptr(e), m, d, _ptr(sigma), _ptr(omega), r, k, q, _ptr(A), _ptr(B), _ptr(S),
                                    _ptr(workspace), workspace.numel(), _stream(stream)), "glowq_solve_factors")
    return A, B, S


def ec_score(e: torch.Tensor, sigma: torch.Tensor, s: Optional[torch.Tensor], r: int,
             workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """fp64 [3]: ||E_cat L||_F^2, sum of the first r squared singular values s, and g_ec, their
    ratio (glowq_ec_score)."""
    e, sigma = e.contiguous(), sigma.contiguous()
    m, d = int(e.shape[0]), int(e.shape[1])
    out = torch.empty(3, dtype=torch.float64, device=e.device)
    if workspace is None:
        workspace = torch.empty(int(lib().glowq_ec_score_workspace_bytes(m, d)), dtype=torch.uint8, device=e.device)
    s = s.contiguous() if s is not None else None
    check(lib().glowq_ec_score(_ptr(e), m, d, _ptr(sigma), _ptr(s), r, _ptr(out), _ptr(workspace), workspace.numel(),
                               _stream(stream)), "glowq_ec_score")
    return out


# --------------------------------------------------------------------------- forward
def workspace_bytes(T: int, r: int, n_proj: int = 1) -> int:
    return int(lib().glowq_workspace_bytes(T, r, n_proj))


def init_workspace(ws: torch.Tensor, stream=None) -> torch.Tensor:
    """Zero-fill a workspace with the library's fill kernel (glowq_workspace_init)."""
    check(lib().glowq_workspace_init(_ptr(ws), ws.numel(), _stream(stream)), "glowq_workspace_init")
    return ws


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    """glowq_workspace_status: synchronises, returns OK, ERR_HANDOFF or ERR_ROUTING and clears the word."""
    st = int(lib().glowq_workspace_status(_ptr(ws), ws.numel(), _stream(stream)))
    if st not in (OK, ERR_HANDOFF, ERR_ROUTING):
        check(st, "glowq_workspace_status")
    return st


def make_workspace(T: int, r: int, n_proj: int = 1, device=None, min_bytes: int = 0) -> Optional[torch.Tensor]:
    n = max(workspace_bytes(T, r, n_proj), min_bytes)
    if n == 0:
        return None
    ws = torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))
    return init_workspace(ws)


def _arr(kind, items):
    return (kind * max(1, len(items)))(*items)


def _outs(x: torch.Tensor, weights: Sequence[QWeight], y):
    if y is None:
        y = [torch.empty(x.shape[0], w.n_out, dtype=torch.float16, device=x.device) for w in weights]
    return y


def group_forward(x: torch.Tensor, weights: Sequence[QWeight], b: Optional[torch.Tensor],
                  a: Sequence[torch.Tensor], r: int, restore: bool = True,
                  workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                  stream=None) -> List[torch.Tensor]:
    m = len(weights)
    y = _outs(x, weights, y)
    if workspace is None and restore and r > 0:
        workspace = make_workspace(x.shape[0], r, 1, x.device)
    wc = _arr(QWeightC, [w.c() for w in weights])
    ac = _arr(_vp, [t.data_ptr() for t in a]) if a else None
    yc = _arr(_vp, [t.data_ptr() for t in y])
    ws_n = 0 if workspace is None else workspace.numel()
    check(lib().glowq_group_forward(_ptr(x), x.shape[0], x.shape[1], m, wc, _ptr(b), ac, r,
                                    int(bool(restore)), _ptr(workspace), ws_n, yc, _stream(stream)),
          "glowq_group_forward")
    return y


def group_forward_static(x: torch.Tensor, weights: Sequence[QWeight], b: Optional[torch.Tensor],
                         a: Sequence[torch.Tensor], r: int, restore: bool = True,
                         y: Optional[List[torch.Tensor]] = None, stream=None) -> List[torch.Tensor]:
    """glowq_group_forward_static: no workspace argument; the library's per-device scratch."""
    m = len(weights)
    y = _outs(x, weights, y)
    wc = _arr(QWeightC, [w.c() for w in weights])
    ac = _arr(_vp, [t.data_ptr() for t in a]) if a else None
    yc = _arr(_vp, [t.data_ptr() for t in y])
    check(lib().glowq_group_forward_static(_ptr(x), x.shape[0], x.shape[1], m, wc, _ptr(b), ac, r,
                                           int(bool(restore)), yc, _stream(stream)),
          "glowq_group_forward_static")
    return y


def w4a8_workspace_bytes(T: int, d: int, r: int) -> int:
    return int(lib().glowq_w4a8_workspace_bytes(T, d, r))


def group_forward_w4a8(x: torch.Tensor, weights: Sequence[QWeight], b: Optional[torch.Tensor],
                       a: Sequence[torch.Tensor], r: int, restore: bool = True,
                       workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                       stream=None) -> List[torch.Tensor]:
    """glowq_group_forward_w4a8: per-token 8-bit activations for the quantised product, the
    correction on the fp16 activations."""
    m = len(weights)
    y = _outs(x, weights, y)
    if workspace is None and x.shape[0] > 0:
        n = w4a8_workspace_bytes(x.shape[0], x.shape[1], r if restore else 0)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
    wc = _arr(QWeightC, [w.c() for w in weights])
    ac = _arr(_vp, [t.data_ptr() for t in a]) if a else None
    yc = _arr(_vp, [t.data_ptr() for t in y])
    ws_n = 0 if workspace is None else workspace.numel()
    check(lib().glowq_group_forward_w4a8(_ptr(x), x.shape[0], x.shape[1], m, wc, _ptr(b), ac, r,
                                         int(bool(restore)), _ptr(workspace), ws_n, yc, _stream(stream)),
          "glowq_group_forward_w4a8")
    return y


def mx8_workspace_bytes(T: int, d: int, r: int) -> int:
    return int(lib().glowq_mx8_workspace_bytes(T, d, r))


def group_forward_mx8(x: torch.Tensor, weights: Sequence[QWeight], b: Optional[torch.Tensor],
                      a: Sequence[torch.Tensor], r: int, restore: bool = True,
                      workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                      stream=None) -> List[torch.Tensor]:
    """glowq_group_forward_mx8: MXFP4 weights against MXFP8 activations on the block-scaled matrix
    cores, the correction on the fp16 activations."""
    m = len(weights)
    y = _outs(x, weights, y)
    if workspace is None and x.shape[0] > 0:
        n = mx8_workspace_bytes(x.shape[0], x.shape[1], r if restore else 0)
        workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
    wc = _arr(QWeightC, [w.c() for w in weights])
    ac = _arr(_vp, [t.data_ptr() for t in a]) if a else None
    yc = _arr(_vp, [t.data_ptr() for t in y])
    ws_n = 0 if workspace is None else workspace.numel()
    check(lib().glowq_group_forward_mx8(_ptr(x), x.shape[0], x.shape[1], m, wc, _ptr(b), ac, r,
                                        int(bool(restore)), _ptr(workspace), ws_n, yc, _stream(stream)),
          "glowq_group_forward_mx8")
    return y


def w8a8_workspace_bytes(T: int, d: int, r: int) -> int:
    return int(lib().glowq_w8a8_workspace_bytes(T, d, r))


_WEIGHT = struct.Struct("QQqqii")


def group_forward_w8a8(x: torch.Tensor, weights: Sequence[QWeight], b: Optional[torch.Tensor],
                       a: Sequence[torch.Tensor], r: int, restore: bool = True,
                       workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                       stream=None) -> List[torch.Tensor]:
    """glowq_group_forward_w8a8: 8-bit integer weights (QWeight.from_int8) and activations, scales
    per output row and per token, the correction on the fp16 activations."""
    what = "group_forward_w8a8"
    a = a or ()
    _same_place(what, x, b, workspace, *a, *(y or ()))
    dev = x.get_device()
    for w in weights:
        if w.q.get_device() != dev or w.sz.get_device() != dev:
            raise GlowQError(ERR_INVALID_ARG, f"{what}: weights on the device of x")
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return group_forward_w8a8(x, weights, b, a, r, restore, workspace, y)
    if x.dim() != 2 or x.dtype != torch.float16:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: x fp16 [T][d]")
    T, d = x.shape
    m = len(weights)
    correct = bool(restore) and r > 0
    ap = None
    if correct:
        if b is None or len(a) != m or b.dtype != torch.float16:
            raise GlowQError(ERR_INVALID_ARG, f"{what}: fp16 factors, one per module")
        _require(b.shape == (r, d), ERR_SHAPE, f"{what}: b [r][d]")
        for t, w in zip(a, weights):
            if t.dtype != torch.float16 or t.shape != (w.n_out, r):
                raise GlowQError(ERR_SHAPE, f"{what}: a[i] fp16 [n_out][r]")
        ap = struct.pack(f"{m}Q", *[t.data_ptr() for t in a])
    if y is None:
        y = [x.new_empty((T, w.n_out)) for w in weights]
    else:
        _require(len(y) == m, ERR_SHAPE, f"{what}: an output per module")
        for t, w in zip(y, weights):
            _require(t.dtype == torch.float16 and t.shape == (T, w.n_out), ERR_SHAPE, f"{what}: y[i] fp16 [T][n_out]")
    if workspace is None and T > 0:
        workspace = torch.empty(max(w8a8_workspace_bytes(T, d, r if correct else 0), 256), dtype=torch.uint8,
                                device=x.device)
    wp = b"".join([_WEIGHT.pack(w.q.data_ptr(), w.sz.data_ptr(), w.n_out, w.k_in, w.fmt, 0) for w in weights])
    yp = struct.pack(f"{m}Q", *[t.data_ptr() for t in y])
    st = lib().glowq_group_forward_w8a8(x.data_ptr(), T, d, m, wp, _addr(b), ap, r, 1 if correct else 0,
                                        _addr(workspace), _bytes(workspace), yp, _current(x))
    if st != OK:
        check(st, "glowq_group_forward_w8a8")
    return y


def fp8_workspace_bytes(T: int, d: int, r: int) -> int:
    return int(lib().glowq_fp8_workspace_bytes(T, d, r))


def group_forward_fp8(x: torch.Tensor, weights: Sequence[QWeight], b: Optional[torch.Tensor],
                       a: Sequence[torch.Tensor], r: int, restore: bool = True,
                       workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                       stream=None) -> List[torch.Tensor]:
    """glowq_group_forward_fp8: e4m3 weights (QWeight.from_fp8) and activations, a scale for each block of 128, the
    correction on the fp16 activations."""
    what = "group_forward_fp8"
    a = a or ()
    _same_place(what, x, b, workspace, *a, *(y or ()))
    dev = x.get_device()
    for w in weights:
        if w.q.get_device() != dev or w.sz.get_device() != dev:
            raise GlowQError(ERR_INVALID_ARG, f"{what}: weights on the device of x")
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return group_forward_fp8(x, weights, b, a, r, restore, workspace, y)
    if x.dim() != 2 or x.dtype != torch.float16:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: x fp16 [T][d]")
    T, d = x.shape
    m = len(weights)
    correct = bool(restore) and r > 0
    ap = None
    if correct:
        if b is None or len(a) != m or b.dtype != torch.float16:
            raise GlowQError(ERR_INVALID_ARG, f"{what}: fp16 factors, one per module")
        _require(b.shape == (r, d), ERR_SHAPE, f"{what}: b [r][d]")
        for t, w in zip(a, weights):
            if t.dtype != torch.float16 or t.shape != (w.n_out, r):
                raise GlowQError(ERR_SHAPE, f"{what}: a[i] fp16 [n_out][r]")
        ap = struct.pack(f"{m}Q", *[t.data_ptr() for t in a])
    if y is None:
        y = [x.new_empty((T, w.n_out)) for w in weights]
    else:
        _require(len(y) == m, ERR_SHAPE, f"{what}: an output per module")
        for t, w in zip(y, weights):
            _require(t.dtype == torch.float16 and t.shape == (T, w.n_out), ERR_SHAPE, f"{what}: y[i] fp16 [T][n_out]")
    if workspace is None and T > 0:
        workspace = torch.empty(max(fp8_workspace_bytes(T, d, r if correct else 0), 256), dtype=torch.uint8,
                                device=x.device)
    wp = b"".join([_WEIGHT.pack(w.q.data_ptr(), w.sz.data_ptr(), w.n_out, w.k_in, w.fmt, 0) for w in weights])
    yp = struct.pack(f"{m}Q", *[t.data_ptr() for t in y])
    st = lib().glowq_group_forward_fp8(x.data_ptr(), T, d, m, wp, _addr(b), ap, r, 1 if correct else 0,
                                        _addr(workspace), _bytes(workspace), yp, _current(x))
    if st != OK:
        check(st, "glowq_group_forward_fp8")
    return y


# --------------------------------------------------------------------------- mixture of experts
@dataclass
class MoeModule:
    """One module (gate, up or down) of every expert, stacked: expert e's device layout at
    e * q_bytes / e * sz_bytes, its left factor a[e] fp16 [n_out][r].  Weights of one format and shape, INT4
    (moe_forward) or block-scaled FP8 (moe_forward_fp8): the experts' products take expert e's place from these sizes."""
    q: torch.Tensor
    sz: torch.Tensor
    a: Optional[torch.Tensor]   # fp16 [n_exp][n_out][r]
    n_out: int
    k_in: int
    fmt: int = FMT_INT4_G128

    @staticmethod
    def stack(weights: Sequence[QWeight], a: Optional[Sequence[torch.Tensor]]) -> "MoeModule":
        _require(len(weights) > 0, ERR_SHAPE, "MoeModule.stack: a weight per expert")
        for w in weights:
            _require(w.fmt == weights[0].fmt and w.fmt in (FMT_INT4_G128, FMT_FP8_BLOCK), ERR_UNSUPPORTED,
                     "MoeModule.stack: INT4 or FP8 weights")
            _require((w.n_out, w.k_in) == (weights[0].n_out, weights[0].k_in), ERR_SHAPE,
                     "MoeModule.stack: weights of one shape")
        q = torch.cat([w.q for w in weights]).contiguous()
        sz = torch.cat([w.sz for w in weights]).contiguous()
        a_st = torch.stack(list(a)).contiguous() if a is not None else None
        return MoeModule(q, sz, a_st, weights[0].n_out, weights[0].k_in, weights[0].fmt)


def moe_workspace_bytes(n_rows: int, T: int, r: int, share: int) -> int:
    return int(lib().glowq_moe_workspace_bytes(n_rows, T, r, share))


def moe_forward(x: torch.Tensor, n_exp: int, modules: Sequence[MoeModule], b: Optional[torch.Tensor], share: int,
                r: int, restore: bool, row_token: Optional[torch.Tensor], offsets: torch.Tensor, n_rows: int,
                workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                stream=None) -> List[torch.Tensor]:
    """glowq_moe_forward: outputs y_i fp16 [n_rows][n_out_i] in routed-row order."""
    for mm in modules:
        _require(mm.fmt == FMT_INT4_G128, ERR_UNSUPPORTED, "moe_forward: INT4 modules")
        blocks = n_exp * (-(-mm.n_out // 16) * (mm.k_in // 128))  # 16 x 128 weights: 1024 bytes of codes, 64 of scales
        if mm.q.nbytes < 1024 * blocks or mm.sz.nbytes < 64 * blocks:
            raise GlowQError(ERR_SHAPE, "moe_forward: INT4 modules of n_exp experts")
    if y is None:
        y = [torch.empty(n_rows, mm.n_out, dtype=torch.float16, device=x.device) for mm in modules]
    if workspace is None:
        workspace = make_workspace(1, 8, 1, x.device,
                                   min_bytes=moe_workspace_bytes(n_rows, x.shape[0], r if restore else 0, share))
    mc = _arr(MoeModuleC, [MoeModuleC(mm.q.data_ptr(), mm.sz.data_ptr(),
                                      None if mm.a is None else mm.a.data_ptr(), yy.data_ptr(), mm.n_out, mm.k_in)
                           for mm, yy in zip(modules, y)])
    check(lib().glowq_moe_forward(_ptr(x), x.shape[0], x.shape[1], n_exp, len(modules), mc, _ptr(b), share, r,
                                  int(bool(restore)), _ptr(row_token), _ptr(offsets), n_rows, _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "glowq_moe_forward")
    return y


def moe_fp8_workspace_bytes(n_rows: int, T: int, d: int, r: int, share: int) -> int:
    return int(lib().glowq_moe_fp8_workspace_bytes(n_rows, T, d, r, share))


_MOE_MODULE = struct.Struct("QQQQqq")


def moe_forward_fp8(x: torch.Tensor, n_exp: int, modules: Sequence[MoeModule], b: Optional[torch.Tensor], share: int,
                    r: int, restore: bool, row_token: Optional[torch.Tensor], offsets: torch.Tensor, n_rows: int,
                    workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                    stream=None) -> List[torch.Tensor]:
    """glowq_moe_forward_fp8: moe_forward on block-scaled FP8 modules (stacked QWeight.from_fp8), outputs y_i fp16
    [n_rows][n_out_i] in routed-row order.  workspace None: as with the routed rows below, a fresh one; the call then
    synchronises, raises ERR_ROUTING itself and cannot be captured."""
    what = "moe_forward_fp8"
    correct = bool(restore) and r > 0
    m = len(modules)
    used = [t for mm in modules for t in (mm.q, mm.sz, mm.a if correct else None)]
    _same_place(what, x, b if correct else None, row_token, offsets, workspace, *used, *(y or ()))
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return moe_forward_fp8(x, n_exp, modules, b, share, r, restore, row_token, offsets, n_rows, workspace, y)
    if x.dim() != 2 or x.dtype != torch.float16:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: x fp16 [T][d]")
    T, d = x.shape
    if offsets.dtype != torch.int32 or (row_token is not None and row_token.dtype != torch.int32):
        raise GlowQError(ERR_INVALID_ARG, f"{what}: int32 lists")
    if offsets.numel() != n_exp + 1 or (row_token is not None and row_token.numel() < n_rows):
        raise GlowQError(ERR_SHAPE, f"{what}: offsets [n_exp + 1], row_token [n_rows]")
    for mm in modules:
        _require(mm.fmt == FMT_FP8_BLOCK, ERR_UNSUPPORTED, f"{what}: FP8 modules")
        if (mm.q.nbytes < n_exp * lib().glowq_fp8_q_bytes(mm.n_out, mm.k_in)
                or mm.sz.nbytes < n_exp * lib().glowq_fp8_sz_bytes(mm.n_out, mm.k_in)):
            raise GlowQError(ERR_SHAPE, f"{what}: modules of n_exp experts")
        if correct and (mm.a is None or mm.a.dtype != torch.float16 or mm.a.shape != (n_exp, mm.n_out, r)):
            raise GlowQError(ERR_SHAPE, f"{what}: a fp16 [n_exp][n_out][r]")
    if correct and (b is None or b.dtype != torch.float16 or b.shape != ((n_exp, r, d) if share == MOE_SHARE_EXPERT else (r, d))):
        raise GlowQError(ERR_SHAPE, f"{what}: b fp16 [n_exp][r][d], or [r][d] shared by all")
    _require(n_rows >= 0, ERR_SHAPE, f"{what}: n_rows >= 0")
    if y is None:
        y = [x.new_empty((n_rows, mm.n_out)) for mm in modules]
    else:
        _require(len(y) == m, ERR_SHAPE, f"{what}: an output per module")
        for t, mm in zip(y, modules):
            _require(t.dtype == torch.float16 and t.shape == (n_rows, mm.n_out), ERR_SHAPE, f"{what}: y[i] fp16 [n_rows][n_out]")
    ws = workspace
    if ws is None:
        ws = _moe_ws(None, x, max(moe_fp8_workspace_bytes(n_rows, T, d, r if correct else 0, share), _MOE_HEADER))
    mc = b"".join([_MOE_MODULE.pack(mm.q.data_ptr(), mm.sz.data_ptr(), mm.a.data_ptr() if correct else 0, t.data_ptr(),
                                    mm.n_out, mm.k_in) for mm, t in zip(modules, y)])
    st = lib().glowq_moe_forward_fp8(x.data_ptr(), T, d, n_exp, m, mc, _addr(b) if correct else None, share, r,
                                     1 if correct else 0, _addr(row_token), offsets.data_ptr(), n_rows, ws.data_ptr(),
                                     _bytes(ws), _current(x))
    if st != OK or workspace is None:
        _moe_done(st, ws, "glowq_moe_forward_fp8")
    return y


# --------------------------------------------------------------------------- routed rows
# Calls with a workspace are asynchronous and report list entries out of range through workspace_status; without
# one they look themselves: they synchronise, raise ERR_ROUTING, and are refused under capture.
def _bytes(ws: Optional[torch.Tensor]) -> int:
    return 0 if ws is None else ws.numel() * ws.element_size()


def _moe_ws(workspace: Optional[torch.Tensor], like: torch.Tensor, n: int) -> torch.Tensor:
    """The caller's workspace, or a fresh zero-filled one, whose error word _moe_done reads.  A captured call
    has to bring its own: nothing but the program that replays it can look at the word."""
    if workspace is None:
        _require(not torch.cuda.is_current_stream_capturing(), ERR_WORKSPACE, "a captured call takes a workspace")
        workspace = init_workspace(torch.empty(n, dtype=torch.uint8, device=like.device))
    return workspace


def _moe_done(status: int, ws: torch.Tensor, what: str) -> None:
    """Raises a call's status or, after one with its own workspace, list entries out of range (synchronises
    the stream); with the caller's workspace they wait for workspace_status."""
    check(status, what)
    check(workspace_status(ws), what)


def _new(out: Optional[torch.Tensor], shape, dtype, like: torch.Tensor, what: str) -> torch.Tensor:
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    if out.dtype != dtype or out.shape != shape:
        raise GlowQError(ERR_SHAPE, f"{what}: out {list(shape)} {dtype}")
    return out


def _row_dtype(what: str, t: torch.Tensor) -> int:
    dt = _DTYPES.get(t.dtype)
    if dt is None or t.dim() != 2:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: fp16 or fp32 rows [n][d]")
    return dt


def _pairs(what: str, pair_row: torch.Tensor, weights: Optional[torch.Tensor]):
    if pair_row.dim() != 2 or pair_row.dtype != torch.int32:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: int32 lists [T][top_k]")
    if weights is not None:
        if weights.dtype != torch.float32:
            raise GlowQError(ERR_INVALID_ARG, f"{what}: fp32 weights")
        if weights.shape != pair_row.shape:
            raise GlowQError(ERR_SHAPE, f"{what}: weights [T][top_k]")
    return pair_row.shape


_MOE_HEADER = 8192


def moe_sort_workspace_bytes(T: int, top_k: int, n_exp: int) -> int:
    return int(lib().glowq_moe_sort_workspace_bytes(T, top_k, n_exp))


def moe_sort(expert_ids: torch.Tensor, n_exp: int, workspace: Optional[torch.Tensor] = None, out=None, stream=None):
    """glowq_moe_sort: expert ids int32 [T][top_k] (-1: no expert) -> (offsets int32 [n_exp + 1], row_token
    int32 [T top_k], pair_row int32 [T][top_k]); `out` may hold the three.  Here and in the calls below
    `workspace` None means a fresh one: the call then synchronises, raises ERR_ROUTING itself and cannot be
    captured."""
    T, k = _pairs("moe_sort", expert_ids, None)
    _same_place("moe_sort", expert_ids, workspace, *(out or ()))
    ctx = _elsewhere(expert_ids, stream)
    if ctx is not None:
        with ctx:
            return moe_sort(expert_ids, n_exp, workspace, out)
    if out is None:
        off, tok, pr = expert_ids.new_empty(n_exp + 1), expert_ids.new_empty(T * k), expert_ids.new_empty((T, k))
    else:
        off, tok, pr = (_new(o, s, torch.int32, expert_ids, "moe_sort") for o, s in zip(out, ((n_exp + 1,), (T * k,), (T, k))))
    ws = workspace
    if ws is None:
        ws = _moe_ws(None, expert_ids, max(moe_sort_workspace_bytes(T, k, n_exp), _MOE_HEADER))
    st = lib().glowq_moe_sort(expert_ids.data_ptr(), T, k, n_exp, off.data_ptr(), tok.data_ptr(), pr.data_ptr(),
                              ws.data_ptr(), _bytes(ws), _current(expert_ids))
    if st != OK or workspace is None:
        _moe_done(st, ws, "glowq_moe_sort")
    return off, tok, pr


def moe_dispatch(x: torch.Tensor, row_token: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """glowq_moe_dispatch: rows [n_rows][d] = x[row_token], zeros for token -1 (row_token int32 [n_rows])."""
    dt = _row_dtype("moe_dispatch", x)
    if row_token.dim() != 1 or row_token.dtype != torch.int32:
        raise GlowQError(ERR_INVALID_ARG, "moe_dispatch: int32 list [n_rows]")
    _same_place("moe_dispatch", x, row_token, workspace, out)
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return moe_dispatch(x, row_token, workspace, out)
    T, d = x.shape
    n = row_token.shape[0]
    out = _new(out, (n, d), x.dtype, x, "moe_dispatch")
    ws = _moe_ws(workspace, x, _MOE_HEADER)
    st = lib().glowq_moe_dispatch(x.data_ptr(), T, d, dt, row_token.data_ptr(), n, out.data_ptr(), ws.data_ptr(),
                                  _bytes(ws), _current(x))
    if st != OK or workspace is None:
        _moe_done(st, ws, "glowq_moe_dispatch")
    return out


def moe_combine(rows: torch.Tensor, pair_row: torch.Tensor, weights: Optional[torch.Tensor],
                add: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """glowq_moe_combine: y [T][d] = add + sum_j weights[:, j] rows[pair_row[:, j]] (weights None: ones)."""
    dt = _row_dtype("moe_combine", rows)
    T, k = _pairs("moe_combine", pair_row, weights)
    _same_place("moe_combine", rows, pair_row, weights, add, workspace, out)
    ctx = _elsewhere(rows, stream)
    if ctx is not None:
        with ctx:
            return moe_combine(rows, pair_row, weights, add, workspace, out)
    n, d = rows.shape
    if add is not None and (add.dtype != rows.dtype or add.shape != (T, d)):
        raise GlowQError(ERR_SHAPE, "moe_combine: add [T][d]")
    out = _new(out, (T, d), rows.dtype, rows, "moe_combine")
    ws = _moe_ws(workspace, rows, _MOE_HEADER)
    st = lib().glowq_moe_combine(rows.data_ptr(), n, pair_row.data_ptr(), _addr(weights), _addr(add), T, k, d, dt,
                                 out.data_ptr(), ws.data_ptr(), _bytes(ws), _current(rows))
    if st != OK or workspace is None:
        _moe_done(st, ws, "glowq_moe_combine")
    return out


def moe_dispatch_backward(d_rows: torch.Tensor, pair_row: torch.Tensor, workspace: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_dispatch: dx [T][d] = sum_j d_rows[pair_row[:, j]] (glowq_moe_combine without weights)."""
    return moe_combine(d_rows, pair_row, None, None, workspace, out, stream)


def moe_combine_backward(dy: torch.Tensor, rows: torch.Tensor, pair_row: torch.Tensor, row_token: torch.Tensor,
                         weights: Optional[torch.Tensor], workspace: Optional[torch.Tensor] = None, out=None,
                         stream=None):
    """Gradients of moe_combine: (d_rows [n_rows][d], d_weights fp32 [T][top_k]) for dy [T][d].  Every row of
    fresh memory is written: rows of token -1 and rows that no pair takes get zeros
    (glowq_moe_combine_backward_whole).  In the two tensors of `out` the latter are left as they were
    (glowq_moe_combine_backward)."""
    what = "moe_combine_backward"
    dt = _row_dtype(what, rows)
    T, k = _pairs(what, pair_row, weights)
    _same_place(what, rows, dy, pair_row, row_token, weights, workspace, *(out or ()))
    ctx = _elsewhere(rows, stream)
    if ctx is not None:
        with ctx:
            return moe_combine_backward(dy, rows, pair_row, row_token, weights, workspace, out)
    n, d = rows.shape
    if dy.dtype != rows.dtype or dy.shape != (T, d):
        raise GlowQError(ERR_SHAPE, f"{what}: dy [T][d]")
    if row_token.dtype != torch.int32 or row_token.dim() != 1:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: int32 list [n_rows]")
    _require(row_token.shape[0] == n, ERR_SHAPE, f"{what}: row_token [n_rows]")
    d_rows, d_w = out if out is not None else (None, None)
    f = lib().glowq_moe_combine_backward_whole if d_rows is None else lib().glowq_moe_combine_backward
    d_rows = _new(d_rows, (n, d), rows.dtype, rows, what)
    d_w = _new(d_w, (T, k), torch.float32, rows, what)
    ws = _moe_ws(workspace, rows, _MOE_HEADER)
    st = f(dy.data_ptr(), rows.data_ptr(), n, pair_row.data_ptr(), row_token.data_ptr(), _addr(weights), T, k, d, dt,
           d_rows.data_ptr(), d_w.data_ptr(), ws.data_ptr(), _bytes(ws), _current(rows))
    if st != OK or workspace is None:
        _moe_done(st, ws, "glowq_moe_combine_backward")
    return d_rows, d_w


# --------------------------------------------------------------------------- router
def _score(what: str, score: str) -> int:
    code = SCORES.get(score)
    if code is None:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: score one of {sorted(SCORES)}")
    return code


def moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None, n_group: int = 1,
              keep_groups: int = 1, group_best: int = 1, renorm: bool = True, scale: float = 1.0,
              workspace: Optional[torch.Tensor] = None, out=None, stream=None):
    """glowq_moe_route: router logits [T][n_exp] -> (ids int32 [T][top_k], weights fp32 [T][top_k]) as moe_sort and
    moe_combine take them; id -1 where a token's experts run out (logits of -inf are out).  bias fp32 [n_exp] decides,
    with the scores, which experts are chosen, and is in no weight.  `out` may hold the two."""
    what = "moe_route"
    dt = _row_dtype(what, logits)
    code = _score(what, score)
    _same_place(what, logits, bias, workspace, *(out or ()))
    ctx = _elsewhere(logits, stream)
    if ctx is not None:
        with ctx:
            return moe_route(logits, top_k, score, bias, n_group, keep_groups, group_best, renorm, scale, workspace, out)
    T, n_exp = logits.shape
    _require(top_k >= 1, ERR_SHAPE, f"{what}: top_k >= 1")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (n_exp,)):
        raise GlowQError(ERR_SHAPE, f"{what}: bias fp32 [n_exp]")
    ids, w = out if out is not None else (None, None)
    ids = _new(ids, (T, top_k), torch.int32, logits, what)
    w = _new(w, (T, top_k), torch.float32, logits, what)
    ws = _moe_ws(workspace, logits, _MOE_HEADER)
    st = lib().glowq_moe_route(logits.data_ptr(), T, n_exp, top_k, dt, code, _addr(bias), n_group, keep_groups, group_best,
                               1 if renorm else 0, scale, ids.data_ptr(), w.data_ptr(), ws.data_ptr(), _bytes(ws),
                               _current(logits))
    if st != OK or workspace is None:
        _moe_done(st, ws, "glowq_moe_route")
    return ids, w


def moe_route_backward(d_weights: torch.Tensor, logits: torch.Tensor, ids: torch.Tensor, score: str = "softmax",
                       renorm: bool = True, scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of moe_route's weights: d_logits [T][n_exp] for d_weights fp32 [T][top_k], the chosen ids held
    (glowq_moe_route_backward)."""
    what = "moe_route_backward"
    dt = _row_dtype(what, logits)
    code = _score(what, score)
    T, k = _pairs(what, ids, d_weights)
    _same_place(what, logits, d_weights, ids, workspace, out)
    ctx = _elsewhere(logits, stream)
    if ctx is not None:
        with ctx:
            return moe_route_backward(d_weights, logits, ids, score, renorm, scale, workspace, out)
    if logits.shape[0] != T:
        raise GlowQError(ERR_SHAPE, f"{what}: logits [T][n_exp]")
    out = _new(out, logits.shape, logits.dtype, logits, what)
    ws = _moe_ws(workspace, logits, _MOE_HEADER)
    st = lib().glowq_moe_route_backward(d_weights.data_ptr(), logits.data_ptr(), ids.data_ptr(), T, logits.shape[1], k, dt, code,
                                        1 if renorm else 0, scale, out.data_ptr(), ws.data_ptr(), _bytes(ws),
                                        _current(logits))
    if st != OK or workspace is None:
        _moe_done(st, ws, "glowq_moe_route_backward")
    return out


# --------------------------------------------------------------------------- layer norm
def _norm_rows(what: str, x: torch.Tensor, *columns) -> int:
    dt = _row_dtype(what, x)
    for t in columns:
        if t is not None and (t.dtype != x.dtype or t.shape != x.shape[1:]):
            raise GlowQError(ERR_SHAPE, f"{what}: weight and bias [d] of x's type")
    return dt


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, out=None, stream=None):
    """glowq_layer_norm: rows x [T][d] -> (y [T][d], mean fp32 [T], rstd fp32 [T]); `out` may hold the three."""
    what = "layer_norm"
    dt = _norm_rows(what, x, weight, bias)
    _same_place(what, x, weight, bias, *(out or ()))
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return layer_norm(x, weight, bias, eps, out)
    T, d = x.shape
    y, mean, rstd = out if out is not None else (None, None, None)
    y = _new(y, (T, d), x.dtype, x, what)
    mean = _new(mean, (T,), torch.float32, x, what)
    rstd = _new(rstd, (T,), torch.float32, x, what)
    st = lib().glowq_layer_norm(x.data_ptr(), _addr(weight), _addr(bias), T, d, eps, dt, y.data_ptr(), mean.data_ptr(),
                                rstd.data_ptr(), _current(x))
    if st != OK:
        check(st, "glowq_layer_norm")
    return y, mean, rstd


def layer_norm_workspace_bytes(T: int, d: int) -> int:
    return int(lib().glowq_layer_norm_workspace_bytes(T, d))


def layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                        weight: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, out=None, stream=None):
    """Gradients of layer_norm for dy [T][d]: (dx [T][d], d_weight fp32 [d], d_bias fp32 [d]); mean and rstd are the
    forward's.  `out` may hold the three."""
    what = "layer_norm_backward"
    dt = _norm_rows(what, x, weight)
    _same_place(what, x, dy, mean, rstd, weight, workspace, *(out or ()))
    ctx = _elsewhere(x, stream)
    if ctx is not None:
        with ctx:
            return layer_norm_backward(dy, x, mean, rstd, weight, workspace, out)
    T, d = x.shape
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise GlowQError(ERR_SHAPE, f"{what}: dy [T][d] of x's type")
    for t in (mean, rstd):
        if t.dtype != torch.float32 or t.shape != (T,):
            raise GlowQError(ERR_SHAPE, f"{what}: mean and rstd fp32 [T]")
    dx, dw, db = out if out is not None else (None, None, None)
    dx = _new(dx, (T, d), x.dtype, x, what)
    dw = _new(dw, (d,), torch.float32, x, what)
    db = _new(db, (d,), torch.float32, x, what)
    if workspace is None:
        workspace = torch.empty(max(layer_norm_workspace_bytes(T, d), 256), dtype=torch.uint8, device=x.device)
    st = lib().glowq_layer_norm_backward(dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _addr(weight), T, d, dt,
                                         dx.data_ptr(), dw.data_ptr(), db.data_ptr(), workspace.data_ptr(), _bytes(workspace),
                                         _current(x))
    if st != OK:
        check(st, "glowq_layer_norm_backward")
    return dx, dw, db


# --------------------------------------------------------------------------- gated activation
def _gate_dtype(what: str, first: torch.Tensor, *others) -> int:
    dt = _DTYPES.get(first.dtype)
    if dt is None:
        raise GlowQError(ERR_INVALID_ARG, f"{what}: fp16 or fp32")
    for t in others:
        if t.dtype != first.dtype or t.shape != first.shape:
            raise GlowQError(ERR_SHAPE, f"{what}: tensors of one type and shape")
    return dt


def swiglu(gate: torch.Tensor, up: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """glowq_swiglu: gate sigmoid(gate) up, elementwise."""
    dt = _gate_dtype("swiglu", gate, up)
    _same_place("swiglu", gate, up, out)
    ctx = _elsewhere(gate, stream)
    if ctx is not None:
        with ctx:
            return swiglu(gate, up, out)
    out = _new(out, gate.shape, gate.dtype, gate, "swiglu")
    st = lib().glowq_swiglu(gate.data_ptr(), up.data_ptr(), gate.numel(), dt, out.data_ptr(), _current(gate))
    if st != OK:
        check(st, "glowq_swiglu")
    return out


def swiglu_backward(dh: torch.Tensor, gate: torch.Tensor, up: torch.Tensor, out=None, stream=None):
    """glowq_swiglu_backward: (d_gate, d_up) for dh (`out` may hold the two tensors)."""
    dt = _gate_dtype("swiglu_backward", gate, up, dh)
    _same_place("swiglu_backward", gate, up, dh, *(out or ()))
    ctx = _elsewhere(gate, stream)
    if ctx is not None:
        with ctx:
            return swiglu_backward(dh, gate, up, out)
    dg, du = out if out is not None else (None, None)
    dg = _new(dg, gate.shape, gate.dtype, gate, "swiglu_backward")
    du = _new(du, gate.shape, gate.dtype, gate, "swiglu_backward")
    st = lib().glowq_swiglu_backward(dh.data_ptr(), gate.data_ptr(), up.data_ptr(), gate.numel(), dt, dg.data_ptr(),
                                     du.data_ptr(), _current(gate))
    if st != OK:
        check(st, "glowq_swiglu_backward")
    return dg, du


def solo_forward(x: torch.Tensor, w: QWeight, b: Optional[torch.Tensor], a: Optional[torch.Tensor],
                 r: int, restore: bool = True, workspace: Optional[torch.Tensor] = None,
                 y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    if y is None:
        y = torch.empty(x.shape[0], w.n_out, dtype=torch.float16, device=x.device)
    if workspace is None and restore and r > 0:
        workspace = make_workspace(x.shape[0], r, 1, x.device)
    wc = w.c()
    ws_n = 0 if workspace is None else workspace.numel()
    check(lib().glowq_solo_forward(_ptr(x), x.shape[0], x.shape[1], ctypes.byref(wc), _ptr(b), _ptr(a),
                                   r, int(bool(restore)), _ptr(workspace), ws_n, _ptr(y), _stream(stream)),
          "glowq_solo_forward")
    return y


def layerwise_forward(x: torch.Tensor, weights: Sequence[QWeight], b: Sequence[torch.Tensor],
                      a: Sequence[torch.Tensor], r: int, restore: bool = True,
                      workspace: Optional[torch.Tensor] = None, y: Optional[List[torch.Tensor]] = None,
                      stream=None) -> List[torch.Tensor]:
    m = len(weights)
    y = _outs(x, weights, y)
    if workspace is None and restore and r > 0:
        workspace = make_workspace(x.shape[0], r, m, x.device)
    wc = _arr(QWeightC, [w.c() for w in weights])
    bc = _arr(_vp, [t.data_ptr() for t in b]) if b else None
    ac = _arr(_vp, [t.data_ptr() for t in a]) if a else None
    yc = _arr(_vp, [t.data_ptr() for t in y])
    ws_n = 0 if workspace is None else workspace.numel()
    check(lib().glowq_layerwise_forward(_ptr(x), x.shape[0], x.shape[1], m, wc, bc, ac, r,
                                        int(bool(restore)), _ptr(workspace), ws_n, yc, _stream(stream)),
          "glowq_layerwise_forward")
    return y


@dataclass
class PathUnit:
    """One unit of a decoder-layer schedule (a group or a solo module) with its restore bit."""
    kind: int
    x: torch.Tensor
    weights: List[QWeight]
    b: Optional[torch.Tensor]
    a: List[torch.Tensor]
    r: int
    restore: bool
    y: List[torch.Tensor]


class PathPlan:
    """Marshalled glowq_unit array for repeated glowq_path_forward calls (keeps the ctypes
    arrays alive)."""

    def __init__(self, units: Sequence[PathUnit]):
        self.units = list(units)
        self._keep = []
        arr = (UnitC * max(1, len(self.units)))()
        for i, u in enumerate(self.units):
            wc = _arr(QWeightC, [w.c() for w in u.weights])
            ac = _arr(_vp, [t.data_ptr() for t in u.a]) if u.a else None
            yc = _arr(_vp, [t.data_ptr() for t in u.y])
            self._keep += [wc, ac, yc]
            arr[i] = UnitC(u.kind, len(u.weights), u.x.data_ptr(), u.x.shape[0], u.x.shape[1],
                           ctypes.cast(wc, ctypes.POINTER(QWeightC)),
                           None if u.b is None else u.b.data_ptr(),
                           None if ac is None else ctypes.cast(ac, ctypes.POINTER(_vp)),
                           u.r, int(bool(u.restore)), ctypes.cast(yc, ctypes.POINTER(_vp)))
        self.arr = arr
        need = max([workspace_bytes(u.x.shape[0], u.r, 1) for u in self.units if u.restore] + [0])
        dev = self.units[0].x.device if self.units else torch.device("cuda")
        self.workspace = make_workspace(1, 8, 1, dev, min_bytes=need)

    def run(self, stream=None) -> None:
        check(lib().glowq_path_forward(self.arr, len(self.units), _ptr(self.workspace),
                                       self.workspace.numel(), _stream(stream)), "glowq_path_forward")
