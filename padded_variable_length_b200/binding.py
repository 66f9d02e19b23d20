"""Thin ctypes binding of libsigattn.so (declared in include/sigattn.h).

Argument marshalling only: every step of the attention path runs in the library's
CUDA kernels.  PyTorch provides device memory and streams.  There is no fallback: if
the library is missing, importing this module raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libsigattn.so")

SIGMOID, SOFTMAX, SOFTMAX1 = 0, 1, 2
OK = 0
ERR_PLAN = -9  # SIGATTN_ERR_PLAN: a tile list failed a structural check
ERR = {-1: "INVALID", -2: "UNSUPPORTED", -3: "ALIGNMENT", -4: "SHAPE", -5: "CUDA",
       -6: "TIMEOUT", -7: "NO_DEVICE", -8: "NOMEM", -9: "PLAN"}


class SigattnError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        detail = _lib.sigattn_error_string(code).decode()
        if code in (-5, -8):
            detail += f" [{_lib.sigattn_last_cuda_error().decode()}]"
        super().__init__(f"{what}: sigattn error {code} ({ERR.get(code, '?')}): {detail}")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python -m padded_variable_length_b200.build`")

_lib = ctypes.CDLL(LIB_PATH)

_p = ctypes.c_void_p
_i32 = ctypes.c_int32
_i64 = ctypes.c_int64
_u64 = ctypes.c_uint64
_I64x3 = ctypes.c_int64 * 3


class PlanSizes(ctypes.Structure):
    _fields_ = [("B", _i32), ("Nq", _i32), ("Nk", _i32), ("QT", _i32), ("KT", _i32),
                ("nonempty", _i64), ("full", _i64), ("partial", _i64), ("grid_total", _i64),
                ("rows_nonempty", _i32), ("cols_nonempty", _i32)]


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_sig("sigattn_plan_from_lengths", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, _p, ctypes.POINTER(_p))
_sig("sigattn_plan_from_mask", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64, _i64,
     _p, ctypes.POINTER(_p))
_sig("sigattn_plan_from_cu_seqlens", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, _p, ctypes.POINTER(_p))
_sig("sigattn_plan_get_sizes", ctypes.c_int, _p, ctypes.POINTER(PlanSizes))
_sig("sigattn_plan_export", ctypes.c_int, _p, _p, _p, _p, _p, _p, _p, _p, _p)
_sig("sigattn_plan_export_work", ctypes.c_int, _p, _p, _p)
_sig("sigattn_plan_export_runs", ctypes.c_int, _p, _p, _p, ctypes.POINTER(_i64))
_sig("sigattn_plan_destroy", None, _p)
_sig("sigattn_plan_validate", ctypes.c_int, _p, _p, ctypes.POINTER(_i64))
_sig("sigattn_tile_list_check_host", ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64, _i64,
     _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _i64, ctypes.POINTER(_i64))
_sig("sigattn_bias_from_counts", ctypes.c_int, _p, _i64, _p, _p)
_sig("sigattn_fwd", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _i64, _p, _I64x3, _p, _p)
_sig("sigattn_bwd", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _i64, _p, _p,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p)
_sig("sigattn_bwd_ex", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _i64, _p, _p,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, ctypes.c_int, _p)
_sig("sigattn_bwd_noalloc", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _i64, _p,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p)
_sig("sigattn_bwd_fused_workspace_size", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
     ctypes.POINTER(ctypes.c_size_t))
_sig("sigattn_bwd_fused", ctypes.c_int, _p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_float,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _I64x3, _p, _i64, _p, _p, ctypes.c_size_t,
     _p, _I64x3, _p, _I64x3, _p, _I64x3, _p)
_qk_rot = [_p, _p, ctypes.c_int, ctypes.c_float, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.POINTER(_i32), _p,
           _p, _i64, _i64]
_sig("sigattn_qk_norm_rope", ctypes.c_int, *[ctypes.c_int] * 5, _p, *[_p, _I64x3] * 2, *_qk_rot, *[_p, _I64x3] * 2, _p)
_sig("sigattn_qk_norm_rope_bwd_workspace_size", ctypes.c_int, *[ctypes.c_int] * 3, ctypes.POINTER(ctypes.c_size_t))
_sig("sigattn_qk_norm_rope_bwd", ctypes.c_int, *[ctypes.c_int] * 5, _p, *[_p, _I64x3] * 4, *_qk_rot, *[_p, _I64x3] * 2,
     _p, _p, _p, ctypes.c_size_t, _p)
_I64x2 = ctypes.c_int64 * 2
_sig("sigattn_linear_workspace_size", ctypes.c_int, *[ctypes.c_int] * 5, ctypes.POINTER(ctypes.c_size_t))
_sig("sigattn_linear_fwd", ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int, _p, _p, _p,
     ctypes.c_float, *[_p, _I64x3] * 3, _p, _p, _I64x3, _p, _p, ctypes.c_size_t, _p)
_sig("sigattn_linear_bwd", ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int, _p, _p, _p,
     ctypes.c_float, *[_p, _I64x3] * 4, _p, _p, *[_p, _I64x3] * 3, _p, _p, ctypes.c_size_t, _p)
_sig("sigattn_linear_fwd_ex", ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int, _p, _p, _p,
     ctypes.c_float, *[_p, _I64x3] * 3, _p, _p, _I64x3, _p, ctypes.c_int, _p, ctypes.c_size_t, _p)
_sig("sigattn_linear_bwd_ex", ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64, ctypes.c_int, ctypes.c_int, _p, _p, _p,
     ctypes.c_float, *[_p, _I64x3] * 4, _p, _p, *[_p, _I64x3] * 3, _p, ctypes.c_int, _p, ctypes.c_size_t, _p)
_sig("sigattn_linear_step", ctypes.c_int, *[ctypes.c_int] * 3, _p, _p, ctypes.c_float, *[_p, _I64x2] * 3, _p, _p,
     _p, _I64x2, _p)
_sig("sigattn_get_status", ctypes.c_int, _p)
_sig("sigattn_set_wait_limit_ns", ctypes.c_int, _u64)
_sig("sigattn_selftest_wait_timeout", ctypes.c_int, _u64, _p)
_sig("sigattn_error_string", ctypes.c_char_p, ctypes.c_int)
_sig("sigattn_version", ctypes.c_int)
_sig("sigattn_last_cuda_error", ctypes.c_char_p)

lib = _lib


def _check(rc: int, what: str):
    if rc != OK:
        raise SigattnError(rc, what)


# torch's current stream of the current device as a raw handle, without building a Stream
# object on every call (the public route below is the fallback)
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        if _raw_current_stream is not None and _current_device is not None:
            return _raw_current_stream(_current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _strides(t: torch.Tensor) -> ctypes.Array:
    """(batch, token, head) element strides of a padded [B, N, H, d] tensor, or of a packed
    [T, H, d] tensor (batch stride 0: ignored by the library for packed plans)."""
    if t.dtype != torch.bfloat16 or t.stride(-1) != 1 or t.dim() not in (3, 4):
        raise ValueError("expected a bf16 [B, N, H, d] or packed [T, H, d] tensor, d contiguous")
    if t.dim() == 3:
        return _I64x3(0, t.stride(0), t.stride(1))
    return _I64x3(t.stride(0), t.stride(1), t.stride(2))


def _keep_until_run(t: torch.Tensor, stream):
    """The plan builds return before the device has read their input: when the build runs
    on another torch stream than the current one, the caching allocator is told that the
    input is in use there (on the current stream, stream order already covers it)."""
    if isinstance(stream, torch.cuda.Stream):
        t.record_stream(stream)


class Plan:
    """A tile plan (owns device buffers; destroyed with the object).  Lengths and mask
    plans are built asynchronously on the stream: the attention calls wait for the build,
    and sizes() / the exports wait for it on the host."""

    def __init__(self, handle: int, dims=None):
        self._h = ctypes.c_void_p(handle)
        self._dims = dims  # (B, Nq, Nk, packed) when known on the host at construction

    @classmethod
    def from_lengths(cls, lengths: torch.Tensor, npad: int, stream=None) -> "Plan":
        if lengths.dtype != torch.int32 or not lengths.is_cuda or not lengths.is_contiguous():
            raise ValueError("lengths must be a contiguous int32 CUDA tensor")
        h = ctypes.c_void_p()
        _keep_until_run(lengths, stream)
        _check(_lib.sigattn_plan_from_lengths(lengths.data_ptr(), lengths.numel(), int(npad),
                                              _stream(stream), ctypes.byref(h)), "plan_from_lengths")
        return cls(h.value, (lengths.numel(), int(npad), int(npad), False))

    @classmethod
    def from_cu_seqlens(cls, cu: torch.Tensor, max_seqlen: int, stream=None) -> "Plan":
        """Plan of a packed batch: sequence b is rows cu[b] .. cu[b+1] of [T, H, d] tensors."""
        if cu.dtype != torch.int32 or not cu.is_cuda or not cu.is_contiguous() or cu.dim() != 1:
            raise ValueError("cu must be a contiguous int32 CUDA tensor [B + 1]")
        h = ctypes.c_void_p()
        _check(_lib.sigattn_plan_from_cu_seqlens(cu.data_ptr(), cu.numel() - 1, int(max_seqlen),
                                                 _stream(stream), ctypes.byref(h)), "plan_from_cu_seqlens")
        return cls(h.value, (cu.numel() - 1, int(max_seqlen), int(max_seqlen), True))

    @classmethod
    def from_mask(cls, mask: torch.Tensor, stream=None) -> "Plan":
        if mask.dtype != torch.uint8 or not mask.is_cuda or mask.dim() != 3 or mask.stride(2) != 1:
            raise ValueError("mask must be a uint8 CUDA tensor [B, Nq, Nk] with Nk contiguous")
        h = ctypes.c_void_p()
        _keep_until_run(mask, stream)
        B, Nq, Nk = mask.shape
        _check(_lib.sigattn_plan_from_mask(mask.data_ptr(), B, Nq, Nk, mask.stride(0), mask.stride(1),
                                           _stream(stream), ctypes.byref(h)), "plan_from_mask")
        return cls(h.value, (B, Nq, Nk, False))

    @property
    def handle(self):
        return self._h

    def dims(self):
        """(B, Nq, Nk, packed): the batch and row extents the plan addresses.  Known on the
        host from the construction arguments, so this never waits for the build (a Plan
        wrapped around a raw handle asks sigattn_plan_get_sizes, which may).  For a packed
        plan Nq = Nk = the longest sequence."""
        if self._dims is None:
            z = self.sizes()
            self._dims = (z["B"], z["Nq"], z["Nk"], False)
        return self._dims

    def sizes(self) -> dict:
        s = PlanSizes()
        _check(_lib.sigattn_plan_get_sizes(self._h, ctypes.byref(s)), "plan_get_sizes")
        return {f: getattr(s, f) for f, _ in PlanSizes._fields_}

    def export(self) -> dict:
        z = self.sizes()
        rows, cols, nz, npart = z["B"] * z["QT"], z["B"] * z["KT"], z["nonempty"], z["partial"]
        out = {
            "row_ptr": np.zeros(rows + 1, np.int32), "col_idx": np.zeros(nz, np.int32),
            "kind": np.zeros(nz, np.uint8), "pidx": np.zeros(nz, np.int32),
            "colT_ptr": np.zeros(cols + 1, np.int32), "rowT_idx": np.zeros(nz, np.int32),
            "csc_map": np.zeros(nz, np.int32), "bits": np.zeros((npart, 512), np.uint32),
        }
        ptr = lambda a: a.ctypes.data if a.size else None
        _check(_lib.sigattn_plan_export(self._h, *(ptr(out[k]) for k in
                                                   ("row_ptr", "col_idx", "kind", "pidx", "colT_ptr",
                                                    "rowT_idx", "csc_map", "bits"))), "plan_export")
        return out

    def export_work(self):
        z = self.sizes()
        rw = np.zeros(z["B"] * z["QT"], np.int32)
        cw = np.zeros(z["B"] * z["KT"], np.int32)
        _check(_lib.sigattn_plan_export_work(self._h, rw.ctypes.data, cw.ctypes.data), "plan_export_work")
        return rw, cw

    def export_runs(self):
        """(run_ptr int32 [B*QT + 1], runs int32 [nruns, 4]): each q-tile row's maximal
        ranges of consecutive k-tiles of one kind, {first k-tile, count, kind, first entry}."""
        z = self.sizes()
        n = _i64()
        _check(_lib.sigattn_plan_export_runs(self._h, None, None, ctypes.byref(n)), "plan_export_runs")
        run_ptr = np.zeros(z["B"] * z["QT"] + 1, np.int32)
        runs = np.zeros((n.value, 4), np.int32)
        _check(_lib.sigattn_plan_export_runs(self._h, run_ptr.ctypes.data,
                                             runs.ctypes.data if runs.size else None,
                                             ctypes.byref(n)), "plan_export_runs")
        return run_ptr, runs

    def validate(self, stream=None) -> int:
        """Debug check of the plan's device arrays (sigattn_plan_validate): -1 when every
        structural property holds, else (check number << 40) | index of the first failure."""
        where = _i64()
        rc = _lib.sigattn_plan_validate(self._h, _stream(stream), ctypes.byref(where))
        if rc not in (OK, ERR_PLAN):
            _check(rc, "plan_validate")
        return where.value

    def close(self):
        if self._h is not None and self._h.value:
            _lib.sigattn_plan_destroy(self._h)
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def tile_list_check_host(t: dict, run_ptr=None, runs=None) -> int:
    """sigattn_tile_list_check_host on host arrays in the export layout (a dict with B, QT,
    KT, row_ptr, col_idx, kind, pidx, colT_ptr, rowT_idx, csc_map, bits): -1 when the list
    passes, else (check number << 40) | index of the first failure.  Needs no GPU."""
    a = {k: np.ascontiguousarray(t[k], dtype=dt) for k, dt in (
        ("row_ptr", np.int32), ("col_idx", np.int32), ("kind", np.uint8), ("pidx", np.int32),
        ("colT_ptr", np.int32), ("rowT_idx", np.int32), ("csc_map", np.int32), ("bits", np.uint32))}
    ptr = lambda x: x.ctypes.data if x is not None and x.size else None
    rp = None if run_ptr is None else np.ascontiguousarray(run_ptr, dtype=np.int32)
    ru = None if runs is None else np.ascontiguousarray(runs, dtype=np.int32).reshape(-1, 4)
    where = _i64()
    rc = _lib.sigattn_tile_list_check_host(
        int(t["B"]), int(t["QT"]), int(t["KT"]), a["col_idx"].size, a["bits"].size // 512,
        *(ptr(a[k]) for k in ("row_ptr", "col_idx", "kind", "pidx", "colT_ptr", "rowT_idx",
                              "csc_map", "bits")),
        ptr(rp), ptr(ru), 0 if ru is None else ru.shape[0], ctypes.byref(where))
    if rc not in (OK, ERR_PLAN):
        _check(rc, "tile_list_check_host")
    return where.value


def _in_order(stream, call, args: dict):
    """``call`` with these arguments and with the stream that it was given as torch's current
    one: what it allocates, zeroes or copies is then in the stream's order, as its kernels are,
    and not beside work of the current stream that still uses the same memory.  The caller's
    tensors are kept until the stream has run the call, and new ones until the current stream
    has used them."""
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)  # 0 and 1 are names of the default stream
        stream = torch.cuda.ExternalStream(handle) if handle not in (None, 0, 1) else torch.cuda.default_stream()
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        got = call(**{**args, "stream": None})
    for t in args.values():
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    for t in got if isinstance(got, tuple) else (got,):
        if t is not None:
            t.record_stream(here)
    return got


def bias_from_counts(counts: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """b = -log(n) per query row from the int32 counts n (0 where n = 0)."""
    if stream is not None:
        return _in_order(stream, bias_from_counts, locals())
    if counts.dtype != torch.int32 or not counts.is_cuda or not counts.is_contiguous():
        raise ValueError("counts must be a contiguous int32 CUDA tensor")
    if out is None:
        out = torch.empty(counts.shape, dtype=torch.float32, device=counts.device)
    _check(_lib.sigattn_bias_from_counts(counts.data_ptr(), counts.numel(), out.data_ptr(),
                                         _stream(None)), "bias_from_counts")
    return out


def _bias_args(bias):
    if bias is None:
        return None, 0
    if bias.dtype != torch.float32 or bias.stride(-1) != 1 or bias.dim() not in (1, 2):
        raise ValueError("bias must be fp32 [B, Nq] (or [T] for a packed plan) with unit row stride")
    return bias.data_ptr(), (bias.stride(0) if bias.dim() == 2 else 0)


def _shape(plan: "Plan", q: torch.Tensor):
    """(B, Nq, H, d): from a padded Q, or from the plan for a packed [T, H, d] Q."""
    if q.dim() == 4:
        return tuple(q.shape)
    B, Nq, _, _ = plan.dims()
    return B, Nq, q.shape[1], q.shape[2]


def _check_extents(plan: "Plan", q_side, k_side, bias=None, lse=None, workspace=None):
    """The library sees pointers and strides only: it addresses B x Nq (Q side) and B x Nk
    (K side) rows of every tensor, B x Nq bias values and B x H x Nq fp32 row statistics,
    with the plan's B and N.  Raise ValueError, before anything is launched, when a tensor
    is smaller than that or disagrees with Q in H or d (a larger tensor is fine: rows past
    the plan's extents are not touched).  Packed [T, H, d] tensors must all have Q's shape."""
    B, Nq, Nk, packed = plan.dims()
    q = q_side[0]
    if packed:
        if q.dim() != 3:
            raise ValueError("a packed plan takes [T, H, d] tensors")
        for t in list(q_side) + list(k_side):
            if t.dim() != 3 or tuple(t.shape) != tuple(q.shape):
                raise ValueError(f"packed tensors must all be {tuple(q.shape)}, got {tuple(t.shape)}")
        H = q.shape[1]
        if bias is not None and (bias.dim() != 1 or bias.shape[0] < q.shape[0]):
            raise ValueError(f"bias of a packed plan must be [T] with T >= {q.shape[0]}")
    else:
        if q.dim() != 4:
            raise ValueError("a padded plan takes [B, N, H, d] tensors")
        H, d = q.shape[2], q.shape[3]
        for side, n in ((q_side, Nq), (k_side, Nk)):
            for t in side:
                if (t.dim() != 4 or t.shape[0] < B or t.shape[1] < n or t.shape[2] != H
                        or t.shape[3] != d):
                    raise ValueError(f"tensor {tuple(t.shape)} does not cover the plan's "
                                     f"[{B}, {n}, {H}, {d}]")
        if bias is not None and (bias.dim() != 2 or bias.shape[0] < B or bias.shape[1] < Nq):
            raise ValueError(f"bias {tuple(bias.shape)} does not cover the plan's [{B}, {Nq}]")
    rows = B * H * Nq
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous()
                            or lse.numel() < rows):
        raise ValueError(f"lse must be a contiguous fp32 [B, H, Nq] buffer of >= {rows} values")
    if workspace is not None and workspace.numel() * workspace.element_size() < 4 * rows:
        raise ValueError(f"workspace must hold >= {rows} fp32 values")


def fwd(plan: Plan, q, k, v, bias=None, epilogue: int = SIGMOID, scale: Optional[float] = None,
        out=None, lse=None, stream=None):
    """O (and the row log-normaliser for the softmax modes) of the planned attention."""
    if stream is not None:
        return _in_order(stream, fwd, locals())
    B, Nq, H, d = _shape(plan, q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if epilogue != SIGMOID and lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check_extents(plan, (q, out), (k, v), bias, lse)
    bp, bs = _bias_args(bias)
    _check(_lib.sigattn_fwd(plan.handle, epilogue, H, d, float(scale),
                            q.data_ptr(), _strides(q), k.data_ptr(), _strides(k),
                            v.data_ptr(), _strides(v), bp, bs, out.data_ptr(), _strides(out),
                            lse.data_ptr() if lse is not None else None, _stream(None)), "fwd")
    return out, lse


BWD_PREP, BWD_DKDV, BWD_DQ, BWD_ALL = 1, 2, 4, 7


def bwd(plan: Plan, q, k, v, o, do, bias=None, epilogue: int = SIGMOID, lse=None,
        scale: Optional[float] = None, workspace=None, dq=None, dk=None, dv=None, stream=None,
        parts: int = BWD_ALL):
    """dQ, dK, dV of L = sum(dO * O) (``parts`` selects PREP / DKDV / DQ)."""
    if stream is not None:
        return _in_order(stream, bwd, locals())
    B, Nq, H, d = _shape(plan, q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if epilogue != SIGMOID and workspace is None:
        workspace = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    _check_extents(plan, [x for x in (q, o, do, dq) if x is not None], (k, v, dk, dv), bias, lse,
                   workspace)
    bp, bs = _bias_args(bias)
    o_ptr = o.data_ptr() if o is not None else None
    o_str = _strides(o) if o is not None else _I64x3(0, 0, 0)
    _check(_lib.sigattn_bwd_ex(plan.handle, epilogue, H, d, float(scale),
                               q.data_ptr(), _strides(q), k.data_ptr(), _strides(k),
                               v.data_ptr(), _strides(v), o_ptr, o_str, do.data_ptr(), _strides(do),
                               bp, bs, lse.data_ptr() if lse is not None else None,
                               workspace.data_ptr() if workspace is not None else None,
                               dq.data_ptr(), _strides(dq), dk.data_ptr(), _strides(dk),
                               dv.data_ptr(), _strides(dv), int(parts), _stream(None)), "bwd")
    return dq, dk, dv


def bwd_fused_workspace_bytes(plan: Plan, H: int, d: int, epilogue: int = SIGMOID) -> int:
    n = ctypes.c_size_t()
    _check(_lib.sigattn_bwd_fused_workspace_size(plan.handle, epilogue, H, d, ctypes.byref(n)),
           "bwd_fused_workspace_size")
    return n.value


def bwd_fused(plan: Plan, q, k, v, o, do, bias=None, epilogue: int = SIGMOID, lse=None,
              scale: Optional[float] = None, workspace=None, dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV of L = sum(dO * O) in one walk over the k-tile columns (d = 64): dQ is
    accumulated in fp32 in ``workspace`` (a 16-byte aligned CUDA buffer of at least
    bwd_fused_workspace_bytes bytes; allocated here if None) and converted at the end."""
    if stream is not None:
        return _in_order(stream, bwd_fused, locals())
    B, Nq, H, d = _shape(plan, q)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = bwd_fused_workspace_bytes(plan, H, d, epilogue)
    if workspace is None:
        workspace = torch.empty((need + 3) // 4, dtype=torch.float32, device=q.device)
    nbytes = workspace.numel() * workspace.element_size()
    _check_extents(plan, [x for x in (q, o, do, dq) if x is not None], (k, v, dk, dv), bias, lse)
    bp, bs = _bias_args(bias)
    o_ptr = o.data_ptr() if o is not None else None
    o_str = _strides(o) if o is not None else _I64x3(0, 0, 0)
    _check(_lib.sigattn_bwd_fused(plan.handle, epilogue, H, d, float(scale),
                                  q.data_ptr(), _strides(q), k.data_ptr(), _strides(k),
                                  v.data_ptr(), _strides(v), o_ptr, o_str, do.data_ptr(), _strides(do),
                                  bp, bs, lse.data_ptr() if lse is not None else None,
                                  workspace.data_ptr(), nbytes,
                                  dq.data_ptr(), _strides(dq), dk.data_ptr(), _strides(dk),
                                  dv.data_ptr(), _strides(dv), _stream(None)), "bwd_fused")
    return dq, dk, dv


# --------------------------------------------------------------------------------------
# Norm and rotation of queries and keys; linear attention
# --------------------------------------------------------------------------------------
# On a few tokens the checks here take longer than the kernels, so what follows from shapes
# and strides alone is worked out once for each combination and looked up after that.
_MEMO_ENTRIES = 4096
_layouts: dict = {}
_qk_shapes: dict = {}
_section_arrays: dict = {}


def _remember(memo: dict, key, value):
    if len(memo) >= _MEMO_ENTRIES:
        memo.clear()
    memo[key] = value
    return value


class _Layout:
    """Of a tensor's shape and strides: the strides the library takes, (batch, token, head)
    and for single tokens (batch, head), and whether entries share memory.  A dimension of
    one entry is never stepped over: 0 is passed, whatever its stride is."""
    __slots__ = ("shape", "dims", "strides", "strides2", "expanded", "dense")

    def __init__(self, shape, stride):
        if not 2 <= len(shape) <= 4:
            raise ValueError("expected a tensor of 3 or 4 dimensions")
        if stride[-1] != 1 and shape[-1] != 1:
            raise ValueError("the last dimension must be contiguous")
        s = [st if n > 1 else 0 for st, n in zip(stride, shape)][:-1]
        self.shape, self.dims = tuple(shape), len(shape)
        self.dense = list(stride) == [math.prod(shape[i + 1:]) for i in range(len(shape))]
        self.strides = _I64x3(*([0] * (3 - len(s)) + s))
        self.strides2 = _I64x2(*([0] + s)[-2:])
        self.expanded = any(st == 0 and n > 1 for st, n in zip(stride, shape))


_NO_STRIDES = _I64x3(0, 0, 0)
_Tensor, _bf16, _f32, _empty_like = torch.Tensor, torch.bfloat16, torch.float32, torch.empty_like


def _here() -> int:
    """The current device, on which the kernels run (-2, no tensor's device, without a GPU)."""
    try:
        return _current_device() if _current_device is not None else torch.cuda.current_device()
    except RuntimeError:
        return -2


def _tensor(t, name: str, dev: int, dims=(3, 4)) -> _Layout:
    """Layout of a bf16 tensor on device ``dev``, the last dimension contiguous."""
    if not isinstance(t, _Tensor) or t.dtype is not _bf16:
        raise ValueError(f"{name} must be a bf16 tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    key = (t.shape, t.stride())
    lay = _layouts.get(key) or _remember(_layouts, key, _Layout(*key))
    if lay.dims not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions")
    return lay


def _small(t, name: str, dtype, shape, dev: int) -> Optional[int]:
    """Pointer of a contiguous tensor of exactly this type and shape (None passes)."""
    if t is None:
        return None
    if not isinstance(t, _Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the current CUDA device")
    return t.data_ptr()


def _out(t: Optional[torch.Tensor], like: torch.Tensor, like_lay: _Layout, name: str, dev: int):
    """(output tensor, its layout): a new one, or the caller's after the checks it needs."""
    if t is None:
        t = _empty_like(like)
        return t, like_lay if like_lay.dense else _tensor(t, name, dev)
    lay = _tensor(t, name, dev, (like_lay.dims,))
    if lay.shape != like_lay.shape:
        raise ValueError(f"{name} must have shape {like_lay.shape}")
    if lay.expanded:
        raise ValueError(f"{name} must not be an expanded tensor")
    return t, lay


def _workspace(workspace, need: int, like: torch.Tensor, dev: int):
    """(tensor, pointer, bytes): the caller's buffer, or a new one of `need` bytes."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = like.new_empty(need, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    elif not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be contiguous and on the current CUDA device")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _qk_shape(qs, ks):
    """(B, N, Hq, Hk, d), the rows' dimensions and whether the batch is packed."""
    one = qs if qs is not None else ks
    if qs is not None and ks is not None and (qs[:-2] != ks[:-2] or qs[-1] != ks[-1]):
        raise ValueError(f"q {qs} and k {ks} must agree in all but the heads")
    B = 1 if len(one) == 3 else one[0]
    return ((B, one[-3], 0 if qs is None else qs[-2], 0 if ks is None else ks[-2], one[-1]), one[:-2], len(one) == 3)


def _qk_args(q, k, wq, wk, eps, inv_freq, positions, sections, interleaved, lengths, norm, dev):
    """The arguments that both directions of qk_norm_rope share, checked: shape arguments,
    norm and rotation arguments, the layouts of q and k."""
    if q is None and k is None:
        raise ValueError("q or k is needed")
    ql = None if q is None else _tensor(q, "q", dev)
    kl = None if k is None else _tensor(k, "k", dev)
    key = (ql, kl)
    got = _qk_shapes.get(key)
    if got is None:
        got = _remember(_qk_shapes, key, _qk_shape(ql and ql.shape, kl and kl.shape))
    head, rows, packed = got
    lp = _small(lengths, "lengths", torch.int32, head[:1], dev)
    d = head[4:]
    wqp, wkp = _small(wq, "wq", _f32, d, dev), _small(wk, "wk", _f32, d, dev)
    rot = n_sec = sa = sb = 0
    sec = ip = pp = None
    if inv_freq is not None:
        if positions is None:
            raise ValueError("a rotation needs positions")
        pairs = inv_freq.numel()
        ip = _small(inv_freq, "inv_freq", torch.float64, (pairs,), dev)
        rot = 2 * pairs
        key = None if sections is None else tuple(sections)
        sec = _section_arrays.get((pairs, key))
        if sec is None:
            counts = [int(x) for x in key] if key is not None else [pairs]
            if pairs < 1 or not counts or sum(counts) != pairs or min(counts) < 0:
                raise ValueError(f"sections must be counts that add up to {pairs}")
            sec = _remember(_section_arrays, (pairs, key), (_i32 * len(counts))(*counts))
        n_sec = len(sec)
        if not isinstance(positions, _Tensor) or positions.dtype is not torch.int32 or positions.get_device() != dev:
            raise ValueError("positions must be an int32 tensor on the current CUDA device")
        ps = positions.shape
        st = positions.stride()
        if n_sec == 1 and ps == rows:
            st = (0,) + st
        elif ps != (n_sec,) + rows:
            raise ValueError(f"positions must have shape {(n_sec,) + rows}")
        if st[-1] != 1 and ps[-1] > 1:
            raise ValueError("positions: the rows must be contiguous")
        pp = positions.data_ptr()
        sa, sb = st[0], (0 if packed else st[1])
    elif positions is not None or sections is not None:
        raise ValueError("positions and sections need inv_freq")
    return (*head, lp), (wqp, wkp, 1 if norm else 0, eps, rot, 1 if interleaved else 0, n_sec, sec, ip, pp, sa, sb), ql, kl


def _pair(t, lay):
    return (None, _NO_STRIDES) if t is None else (t.data_ptr(), lay.strides)


def qk_norm_rope(q, k=None, wq=None, wk=None, eps: float = 1e-6, inv_freq=None, positions=None, sections=None,
                 interleaved: bool = False, lengths=None, norm: bool = True, out_q=None, out_k=None, stream=None):
    """(yq, yk): every head of q and k normed by its root mean square (norm=False: not),
    weighted, and its first 2 * len(inv_freq) values rotated by the positions.  q, k bf16
    [B, N, H, d] or packed [T, H, d] (either may be None); wq, wk fp32 [d]; inv_freq fp64
    [pairs]; positions int32 [axes, B, N] resp. [axes, T] (one axis: that dimension may be
    left out); sections: pairs of each axis.  Pad rows (lengths int32 [B]) come out as 0; of a
    packed batch all rows are valid, or the first lengths[0] (int32 [1], cu_seqlens[-1:])."""
    if stream is not None:
        return _in_order(stream, qk_norm_rope, locals())
    dev = _here()
    head, rot, ql, kl = _qk_args(q, k, wq, wk, eps, inv_freq, positions, sections, interleaved, lengths, norm, dev)
    yq, yql = (None, None) if q is None else _out(out_q, q, ql, "out_q", dev)
    yk, ykl = (None, None) if k is None else _out(out_k, k, kl, "out_k", dev)
    if head[0] and head[1] and head[2] + head[3]:
        _check(_lib.sigattn_qk_norm_rope(*head, *_pair(q, ql), *_pair(k, kl), *rot, *_pair(yq, yql), *_pair(yk, ykl),
                                         _stream(None)), "qk_norm_rope")
    return yq, yk


@functools.lru_cache(maxsize=_MEMO_ENTRIES)
def qk_norm_rope_bwd_workspace_bytes(B: int, N: int, d: int) -> int:
    n = ctypes.c_size_t()
    _check(_lib.sigattn_qk_norm_rope_bwd_workspace_size(B, N, d, ctypes.byref(n)), "qk_norm_rope_bwd_workspace_size")
    return n.value


def qk_norm_rope_bwd(q, k, dyq, dyk, wq=None, wk=None, eps: float = 1e-6, inv_freq=None, positions=None,
                     sections=None, interleaved: bool = False, lengths=None, norm: bool = True, dq=None, dk=None,
                     workspace=None, stream=None):
    """(dq, dk, dwq, dwk) from the gradients dyq, dyk of qk_norm_rope's outputs; dwq, dwk are
    fp32 [d], None for a weight that is None.  Rows of a packed batch that hold no data (NaN,
    say) must be behind lengths[0], or the weights' sums take them up.  ``workspace``: a
    contiguous CUDA buffer of qk_norm_rope_bwd_workspace_bytes bytes (allocated here if None and
    needed)."""
    if stream is not None:
        return _in_order(stream, qk_norm_rope_bwd, locals())
    dev = _here()
    head, rot, ql, kl = _qk_args(q, k, wq, wk, eps, inv_freq, positions, sections, interleaved, lengths, norm, dev)
    args, outs, grads = [], [], []
    for x, lay, dy, w, dx, name in ((q, ql, dyq, wq, dq, "q"), (k, kl, dyk, wk, dk, "k")):
        if x is None:
            if dy is not None or w is not None or dx is not None:
                raise ValueError(f"gradients or weights of an absent {name}")
            args.append((None, _NO_STRIDES, None, _NO_STRIDES))
            outs.append(None)
            grads.append(None)
            continue
        dyl = _tensor(dy, "dy" + name, dev)
        if dyl.shape != lay.shape:
            raise ValueError(f"dy{name} must have shape {lay.shape}")
        dx, dxl = _out(dx, x, lay, "d" + name, dev)
        args.append((dy.data_ptr(), dyl.strides, dx.data_ptr(), dxl.strides))
        outs.append(dx)
        grads.append(None if w is None else _empty_like(w))
    gq, gk = grads
    if not (head[0] and head[1] and head[2] + head[3]):
        return outs[0], outs[1], *(None if g is None else g.zero_() for g in grads)
    need = qk_norm_rope_bwd_workspace_bytes(head[0], head[1], head[4]) if gq is not None or gk is not None else 0
    ws, wp, wn = _workspace(workspace, need, q if q is not None else k, dev)
    _check(_lib.sigattn_qk_norm_rope_bwd(*head, *_pair(q, ql), *_pair(k, kl), *args[0][:2], *args[1][:2], *rot,
                                         *args[0][2:], *args[1][2:], None if gq is None else gq.data_ptr(),
                                         None if gk is None else gk.data_ptr(), wp, wn, _stream(None)),
           "qk_norm_rope_bwd")
    return outs[0], outs[1], gq, gk


@functools.lru_cache(maxsize=_MEMO_ENTRIES)
def linear_workspace_bytes(B: int, N: int, H: int, d: int, backward: bool = False) -> int:
    n = ctypes.c_size_t()
    _check(_lib.sigattn_linear_workspace_size(B, N, H, d, 1 if backward else 0, ctypes.byref(n)), "linear_workspace_size")
    return n.value


def _linear_args(q, others, log_decay, lengths, cu_seqlens, max_seqlen, states, dev):
    """The arguments that linear_fwd and linear_bwd share, checked: shape arguments, pointers
    of the states, and pointer and strides of q and the others."""
    lay = _tensor(q, "q", dev)
    pairs = [q.data_ptr(), lay.strides]
    for t, name in others:
        x = _tensor(t, name, dev)
        if x is not lay and x.shape != lay.shape:
            raise ValueError(f"{name} must have q's shape {lay.shape}")
        pairs += (t.data_ptr(), x.strides)
    *rows, H, d = lay.shape
    lp = cp = None
    if len(rows) == 1:
        if cu_seqlens is None or max_seqlen is None or lengths is not None:
            raise ValueError("a packed batch takes cu_seqlens and max_seqlen, no lengths")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be a contiguous int32 CUDA tensor [B + 1]")
        cp = _small(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, dev)
        B, N, T = cu_seqlens.numel() - 1, int(max_seqlen), rows[0]
    else:
        if cu_seqlens is not None or max_seqlen is not None:
            raise ValueError("a padded batch takes lengths, no cu_seqlens or max_seqlen")
        (B, N), T = rows, 0
        lp = _small(lengths, "lengths", torch.int32, (B,), dev)
    gp = _small(log_decay, "log_decay", _f32, (H,), dev)
    if gp is None:
        raise ValueError("log_decay is needed")
    ptrs = [_small(s, name, _f32, (B, H, d, d), dev) for s, name in states]
    return (B, N, T, H, d, lp, cp, gp), ptrs, pairs, lay


def _hand_on(to: Optional[torch.Tensor], state: Optional[torch.Tensor]):
    """Without tokens a state stays as it is (None: 0)."""
    if to is not None and to is not state:
        to.zero_() if state is None else to.copy_(state)
    return to


def linear_fwd(q, k, v, log_decay, lengths=None, cu_seqlens=None, max_seqlen=None, state=None,
               return_state: bool = False, scale: Optional[float] = None, out=None, final_state=None,
               workspace=None, stream=None):
    """(o, final_state) of linear attention with the decay exp(log_decay[h]): S = decay S +
    k v^T, o = scale S^T q for each token in turn.  q, k, v bf16 [B, N, H, d] (with lengths) or
    packed [T, H, d] (with cu_seqlens and max_seqlen); state fp32 [B, H, d, d] is what the
    sequences start from (None: 0).  The final state is returned where return_state is set or
    a buffer for it is given, else None.  Rows of no sequence come out as 0; of a packed tensor
    given as ``out`` they stay as they are."""
    if stream is not None:
        return _in_order(stream, linear_fwd, locals())
    dev = _here()
    head, (sp, fp), pairs, lay = _linear_args(q, ((k, "k"), (v, "v")), log_decay, lengths, cu_seqlens, max_seqlen,
                                              ((state, "state"), (final_state, "final_state")), dev)
    B, N, _, H, d = head[:5]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rest = 1 if out is None else 0
    out, ol = _out(out, q, lay, "out", dev)
    if return_state and final_state is None:
        final_state = torch.empty((B, H, d, d), dtype=torch.float32, device=q.device)
        fp = final_state.data_ptr()
    if N == 0 or q.numel() == 0:
        return out.zero_() if rest else out, _hand_on(final_state, state)
    ws, wp, wn = _workspace(workspace, linear_workspace_bytes(B, N, H, d), q, dev)
    _check(_lib.sigattn_linear_fwd_ex(*head, scale, *pairs, sp, out.data_ptr(), ol.strides, fp, rest, wp, wn,
                                      _stream(None)), "linear_fwd")
    return out, final_state


def linear_bwd(q, k, v, do, log_decay, lengths=None, cu_seqlens=None, max_seqlen=None, state=None, dstate=None,
               scale: Optional[float] = None, dq=None, dk=None, dv=None, dstate_out=None, workspace=None, stream=None):
    """(dq, dk, dv, dstate_out): gradients of linear_fwd from do and, for a loss that uses the
    final state, its gradient ``dstate``.  dstate_out, the gradient of ``state``, is None where
    there was no state (unless a buffer for it is given).  Rows of no sequence as in linear_fwd."""
    if stream is not None:
        return _in_order(stream, linear_bwd, locals())
    dev = _here()
    head, (sp, ep, gp), pairs, lay = _linear_args(
        q, ((k, "k"), (v, "v"), (do, "do")), log_decay, lengths, cu_seqlens, max_seqlen,
        ((state, "state"), (dstate, "dstate"), (dstate_out, "dstate_out")), dev)
    B, N, _, H, d = head[:5]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    rest = sum(1 << i for i, t in enumerate((dq, dk, dv)) if t is None)
    (dq, dql), (dk, dkl), (dv, dvl) = _out(dq, q, lay, "dq", dev), _out(dk, k, lay, "dk", dev), _out(dv, v, lay, "dv", dev)
    if state is not None and dstate_out is None:
        dstate_out = torch.empty_like(state)
        gp = dstate_out.data_ptr()
    if N == 0 or q.numel() == 0:
        return *(t.zero_() if rest >> i & 1 else t for i, t in enumerate((dq, dk, dv))), _hand_on(dstate_out, dstate)
    ws, wp, wn = _workspace(workspace, linear_workspace_bytes(B, N, H, d, True), q, dev)
    _check(_lib.sigattn_linear_bwd_ex(*head, scale, *pairs, sp, ep, dq.data_ptr(), dql.strides, dk.data_ptr(), dkl.strides,
                                      dv.data_ptr(), dvl.strides, gp, rest, wp, wn, _stream(None)), "linear_bwd")
    return dq, dk, dv, dstate_out


def linear_step(q, k, v, log_decay, state, lengths=None, scale: Optional[float] = None, state_out=None, out=None,
                stream=None) -> torch.Tensor:
    """o of one token of each sequence, q, k, v bf16 [B, H, d]; ``state`` fp32 [B, H, d, d] is
    updated in place, or kept and its update written to ``state_out``.  Sequences with
    lengths[b] = 0 have no token: o is 0 and their state stays."""
    if stream is not None:
        return _in_order(stream, linear_step, locals())
    dev = _here()
    ql, kl, vl = _tensor(q, "q", dev, (3,)), _tensor(k, "k", dev, (3,)), _tensor(v, "v", dev, (3,))
    if kl.shape != ql.shape or vl.shape != ql.shape:
        raise ValueError(f"k and v must have q's shape {ql.shape}")
    B, H, d = ql.shape
    square = (B, H, d, d)
    lp = _small(lengths, "lengths", torch.int32, (B,), dev)
    gp = _small(log_decay, "log_decay", _f32, (H,), dev)
    sp = _small(state, "state", _f32, square, dev)
    if gp is None or sp is None:
        raise ValueError("log_decay and state are needed")
    np_ = sp if state_out is None else _small(state_out, "state_out", _f32, square, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, ol = _out(out, q, ql, "out", dev)
    if q.numel() == 0:
        return out
    _check(_lib.sigattn_linear_step(B, H, d, lp, gp, scale, q.data_ptr(), ql.strides2, k.data_ptr(), kl.strides2,
                                    v.data_ptr(), vl.strides2, sp, np_, out.data_ptr(), ol.strides2, _stream(None)),
           "linear_step")
    return out


def get_status(stream=None) -> int:
    """Synchronises the stream; returns and clears the device status word (0 or TIMEOUT)."""
    return _lib.sigattn_get_status(_stream(stream))


def set_wait_limit_ns(ns: int):
    _check(_lib.sigattn_set_wait_limit_ns(int(ns)), "set_wait_limit_ns")


def selftest_wait_timeout(ns: int, stream=None):
    _check(_lib.sigattn_selftest_wait_timeout(int(ns), _stream(stream)), "selftest_wait_timeout")
