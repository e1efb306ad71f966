"""ctypes binding of libqlora's 8-bit activation checkpoints and of the adapters
of many requests beside one shared projection (include/qlora.h).  Argument
marshalling only, as in _lib.py.

The tensors of a call are on one GPU.  Outputs that are not passed in are
allocated there; work goes to that GPU's current stream."""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import NamedTuple, Optional, Union

import torch

from . import _lib
from ._lib import _check
from ._train import _TYPES, _addr, _call, _matrix_type, _need, _out, _room

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_BF16, _F32, _I32, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
_SMALL_M = 16   # a layer call of so many tokens reads no saved dropout mask


class _Packed(ctypes.Structure):
    _fields_ = [("M", _I64), ("d", _I64), ("codes", _P), ("scale", _P)]


class _Bank(ctypes.Structure):
    _fields_ = [("slots", _I64), ("r", _I64), ("d_in", _I64), ("d_out", _I64), ("A", _P), ("B", _P),
                ("scale", _P)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of this module's entry points."""
    i, sz, pp, bp = ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(_Packed), ctypes.POINTER(_Bank)
    psz = ctypes.POINTER(sz)
    L.qlora_pack8_sizes.argtypes = [_I64, _I64, psz, psz]
    L.qlora_pack8.argtypes = [i, _P, pp, _P]
    L.qlora_unpack8.argtypes = [pp, i, _P, _P]
    L.qlora_linear_bwd_packed.argtypes = [ctypes.POINTER(_lib._Nf4), pp, _P, _I64, _P, _P, _I64, _F,
                                          ctypes.POINTER(_lib._Dropout), _P, _P, _P, _P, _P, sz, _P]
    L.qlora_adapters_plan_bytes.restype = sz
    L.qlora_adapters_plan_bytes.argtypes = [_I64, _I64]
    L.qlora_adapters_plan.argtypes = [_P, _I64, _I64, _P, sz, _P]
    L.qlora_adapters_workspace_bytes.restype = sz
    L.qlora_adapters_workspace_bytes.argtypes = [i, bp, _I64]
    L.qlora_adapters_fwd.argtypes = [bp, _P, sz, _P, _I64, _P, _P, _P, _P, sz, _P]
    L.qlora_adapters_bwd.argtypes = [bp, _P, sz, _P, pp, _P, _P, _I64, _P, _P, _P, _P, _P, sz, _P]


# ------------------------------------------------------- activations in 8 bits

def _blocks(d: int) -> int:
    return -(-d // _lib.BLOCK)


class Packed8:
    """A matrix [M, d] kept in 8 bits: codes int8 [M, ceil(d / 64) * 64] and
    scale FP32 [ceil(d / 64), M], one for 64 values of a row."""

    __slots__ = ("M", "d", "codes", "scale", "c")

    def __init__(self, M: int, d: int, codes: torch.Tensor, scale: torch.Tensor):
        nb = _blocks(d)
        at = codes.get_device()
        if at < 0:
            raise ValueError(f"codes: expected on the GPU, got {codes.device}")
        _need(codes, _I8, (M, nb * _lib.BLOCK), "codes", at)
        _need(scale, _F32, (nb, M), "scale", at)
        self.M, self.d, self.codes, self.scale = M, d, codes, scale
        self.c = _Packed(M, d, codes.data_ptr(), scale.data_ptr())

    @staticmethod
    def empty(M: int, d: int, device="cuda") -> "Packed8":
        nb = _blocks(d)
        p = Packed8.__new__(Packed8)   # buffers made here have no shapes to check
        p.M, p.d = M, d
        p.codes = torch.empty((M, nb * _lib.BLOCK), dtype=_I8, device=device)
        p.scale = torch.empty((nb, M), dtype=_F32, device=device)
        if p.codes.get_device() < 0:
            raise ValueError(f"device: expected a GPU, got {p.codes.device}")
        p.c = _Packed(M, d, p.codes.data_ptr(), p.scale.data_ptr())
        return p

    @property
    def device(self):
        return self.codes.device

    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scale.numel()


def qlora_pack8_sizes(M: int, d: int) -> tuple[int, int]:
    """Bytes of the codes and of the scales."""
    out = [ctypes.c_size_t(), ctypes.c_size_t()]
    _check(_lib.lib().qlora_pack8_sizes(M, d, *[ctypes.byref(o) for o in out]), "qlora_pack8_sizes")
    return out[0].value, out[1].value


def qlora_pack8(X: torch.Tensor, out: Optional[Packed8] = None) -> Packed8:
    """X (BF16 or FP32 [M, d]) in 8 bits."""
    ty, at = _matrix_type(X, "X")
    M, d = X.shape
    if not X.is_contiguous():
        _lib._need(X, X.dtype, X.shape, "X")
    if out is None:
        out = Packed8.empty(M, d, X.device)
    elif (out.M, out.d, out.codes.get_device()) != (M, d, at):
        raise ValueError(f"out: expected a [{M}, {d}] checkpoint on GPU {at}, got [{out.M}, {out.d}] "
                         f"on {out.device}")
    _call("qlora_pack8", at, ty, X.data_ptr(), out.c)
    return out


def qlora_unpack8(p: Packed8, dtype: torch.dtype = torch.bfloat16,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that p stands for, as BF16 or FP32 [M, d]."""
    if dtype not in _TYPES:
        raise ValueError(f"dtype: expected bfloat16 or float32, got {dtype}")
    at = p.codes.get_device()
    out = _out(out, (p.M, p.d), dtype, p.device, "out", at)
    _call("qlora_unpack8", at, p.c, _TYPES[dtype], out.data_ptr())
    return out


def qlora_linear_bwd_packed(q: _lib.NF4Weight, X8: Packed8, dY: torch.Tensor, A: torch.Tensor,
                            B: torch.Tensor, lora_alpha: float, T_saved: torch.Tensor,
                            dropout: Optional[_lib.Dropout] = None, need_dx: bool = True,
                            dX: Optional[torch.Tensor] = None, dA: Optional[torch.Tensor] = None,
                            dB: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None):
    """(dX or None, dA, dB): qlora_linear_bwd (with dropout
    qlora_linear_bwd_dropout) from an input kept in 8 bits and the forward's T."""
    M, at, dev = X8.M, X8.codes.get_device(), X8.device
    r = A.shape[0]
    if X8.d != q.d_in:
        raise ValueError(f"X8: expected {q.d_in} values a row, got {X8.d}")
    if q.codes.get_device() != at:
        raise ValueError(f"q: expected on GPU {at}, got {q.device}")
    _need(dY, _BF16, (M, q.d_out), "dY", at)
    _need(A, _BF16, (r, q.d_in), "A", at)
    _need(B, _BF16, (q.d_out, r), "B", at)
    _need(T_saved, _F32, (M, r), "T_saved", at)
    if dropout is not None and M > _SMALL_M and dropout.keep_rows is not None and dropout.keep_cols is not None:
        _need(dropout.keep_rows, _I32, (M, q.d_in // 32), "dropout.keep_rows", at)
        _need(dropout.keep_cols, _I32, (q.d_in, (M + 31) // 32), "dropout.keep_cols", at)
    dX = _out(dX, (M, q.d_in), _BF16, dev, "dX", at) if need_dx else None
    dA = _out(dA, (r, q.d_in), _F32, dev, "dA", at)
    dB = _out(dB, (q.d_out, r), _F32, dev, "dB", at)
    if workspace is None:
        op = _lib.QLORA_OP_BWD_PACKED if dropout is None else _lib.QLORA_OP_BWD_PACKED_DROPOUT
        workspace = _lib._workspace(_lib.qlora_workspace_bytes(op, q.d_out, q.d_in, M, r), dev)
    _call("qlora_linear_bwd_packed", at, q.c_struct(), X8.c, dY.data_ptr(), M, A.data_ptr(),
          B.data_ptr(), r, float(lora_alpha), None if dropout is None else dropout.c_struct(),
          T_saved.data_ptr(), _addr(dX), dA.data_ptr(), dB.data_ptr(), workspace.data_ptr(),
          _room(workspace, at))
    return dX, dA, dB


# --------------------------------------------------- adapters of many requests

class AdapterBank:
    """Adapters of one rank for one projection: A BF16 [slots, r, d_in], B BF16
    [slots, d_out, r], scale FP32 [slots] (lora_alpha / r of each).  The tensors
    are used in place and must keep their storage; writing a slot's part of them
    exchanges its adapter."""

    __slots__ = ("A", "B", "scale", "slots", "r", "d_in", "d_out", "at", "c")

    def __init__(self, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor):
        at = A.get_device()
        if A.dim() != 3 or B.dim() != 3 or at < 0:
            raise ValueError("A, B: expected [slots, r, d_in] and [slots, d_out, r] on the GPU, got "
                             f"{tuple(A.shape)} and {tuple(B.shape)} on {A.device}")
        self.slots, self.r, self.d_in = A.shape
        self.d_out = B.shape[1]
        _need(A, _BF16, (self.slots, self.r, self.d_in), "A", at)
        _need(B, _BF16, (self.slots, self.d_out, self.r), "B", at)
        _need(scale, _F32, (self.slots,), "scale", at)
        self.A, self.B, self.scale, self.at = A, B, scale, at
        self.c = _Bank(self.slots, self.r, self.d_in, self.d_out, A.data_ptr(), B.data_ptr(),
                       scale.data_ptr())


@dataclass
class AdapterPlan:
    """A batch's tokens sorted by slot; for all projections whose banks have
    this number of slots."""
    M: int
    slots: int
    buffer: torch.Tensor


class AdapterOut(NamedTuple):
    Y: torch.Tensor                # BF16 [M, d_out]
    T: Optional[torch.Tensor]      # FP32 [M, r], for the backward


class AdapterGrads(NamedTuple):
    dX: Optional[torch.Tensor]     # BF16 [M, d_in]
    dA: torch.Tensor               # FP32 [slots, r, d_in]
    dB: torch.Tensor               # FP32 [slots, d_out, r]


def qlora_adapters_plan_bytes(M: int, slots: int) -> int:
    return int(_lib.lib().qlora_adapters_plan_bytes(M, slots))


def qlora_adapters_plan(index: torch.Tensor, slots: int,
                        out: Optional[AdapterPlan] = None) -> AdapterPlan:
    """The plan of a batch whose token m takes adapter index[m] (int32 [M]; a
    value outside [0, slots): none).  It is read on the GPU: a plan `out` that
    is filled anew serves calls captured into a graph."""
    at = index.get_device()
    M = index.numel()
    if at < 0:
        raise ValueError(f"index: expected on the GPU, got {index.device}")
    _need(index, _I32, (M,), "index", at)
    need = qlora_adapters_plan_bytes(M, slots)
    if out is None:
        out = AdapterPlan(M, slots, _lib._workspace(need, index.device))
    elif (out.M, out.slots) != (M, slots):
        raise ValueError(f"out: a plan of {out.M} tokens and {out.slots} slots, not {M} and {slots}")
    _call("qlora_adapters_plan", at, index.data_ptr(), M, slots, out.buffer.data_ptr(),
          _room(out.buffer, at))
    return out


def qlora_adapters_workspace_bytes(bank: AdapterBank, M: int, backward: bool = False) -> int:
    return int(_lib.lib().qlora_adapters_workspace_bytes(1 if backward else 0, bank.c, M))


def _planned(bank: AdapterBank, plan: AdapterPlan, M: int) -> None:
    if plan.M != M or plan.slots != bank.slots:
        raise ValueError(f"plan: made for {plan.M} tokens and {plan.slots} slots, the call has {M} "
                         f"and {bank.slots}")


def qlora_adapters_fwd(X: torch.Tensor, bank: AdapterBank, plan: AdapterPlan,
                       Y0: Optional[torch.Tensor] = None, Y: Optional[torch.Tensor] = None,
                       T: Optional[torch.Tensor] = None, save_T: bool = True,
                       workspace: Optional[torch.Tensor] = None) -> AdapterOut:
    """Y = Y0 + scale_a (X A_a^T) B_a^T, each token with its own adapter a.  Y
    may be Y0; save_T=False leaves out what only the backward needs."""
    at, M = bank.at, X.shape[0]
    _need(X, _BF16, (M, bank.d_in), "X", at)
    _planned(bank, plan, M)
    if Y0 is not None:
        _need(Y0, _BF16, (M, bank.d_out), "Y0", at)
    Y = _out(Y, (M, bank.d_out), _BF16, X.device, "Y", at)
    T = _out(T, (M, bank.r), _F32, X.device, "T", at) if save_T else None
    if workspace is None:
        workspace = _lib._workspace(qlora_adapters_workspace_bytes(bank, M), X.device)
    _call("qlora_adapters_fwd", at, bank.c, plan.buffer.data_ptr(), _room(plan.buffer, at),
          X.data_ptr(), M, _addr(Y0), Y.data_ptr(), _addr(T), workspace.data_ptr(),
          _room(workspace, at))
    return AdapterOut(Y, T)


def qlora_adapters_bwd(dY: torch.Tensor, X: Union[torch.Tensor, Packed8], T: torch.Tensor,
                       bank: AdapterBank, plan: AdapterPlan, dX0: Optional[torch.Tensor] = None,
                       need_dx: bool = True, dX: Optional[torch.Tensor] = None,
                       dA: Optional[torch.Tensor] = None, dB: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> AdapterGrads:
    """Backward of qlora_adapters_fwd from its X (BF16, or kept in 8 bits) and T:
    the adapters' part of the input gradient is added to dX0, the shared
    projection's; dX may be dX0."""
    at, M = bank.at, dY.shape[0]
    _need(dY, _BF16, (M, bank.d_out), "dY", at)
    _planned(bank, plan, M)
    X8 = None
    if isinstance(X, Packed8):
        if (X.M, X.d) != (M, bank.d_in) or X.codes.get_device() != at:
            raise ValueError(f"X: expected a [{M}, {bank.d_in}] checkpoint on GPU {at}, got "
                             f"[{X.M}, {X.d}] on {X.device}")
        X, X8 = None, X.c
    else:
        _need(X, _BF16, (M, bank.d_in), "X", at)
    _need(T, _F32, (M, bank.r), "T", at)
    dev = dY.device
    if need_dx:
        if dX0 is not None:
            _need(dX0, _BF16, (M, bank.d_in), "dX0", at)
        dX = _out(dX, (M, bank.d_in), _BF16, dev, "dX", at)
    else:
        dX = dX0 = None
    dA = _out(dA, (bank.slots, bank.r, bank.d_in), _F32, dev, "dA", at)
    dB = _out(dB, (bank.slots, bank.d_out, bank.r), _F32, dev, "dB", at)
    if workspace is None:
        workspace = _lib._workspace(qlora_adapters_workspace_bytes(bank, M, backward=True), dev)
    _call("qlora_adapters_bwd", at, bank.c, plan.buffer.data_ptr(), _room(plan.buffer, at), _addr(X),
          X8, T.data_ptr(), dY.data_ptr(), M, _addr(dX0), _addr(dX), dA.data_ptr(), dB.data_ptr(),
          workspace.data_ptr(), _room(workspace, at))
    return AdapterGrads(dX, dA, dB)
