"""ctypes binding of libqlora's entry points around the linear layers
(include/qlora.h): norms, token log-probabilities, the preference loss and the
clipped policy loss.  Argument marshalling only, as in _lib.py.

The tensors of a call are on one GPU.  Outputs that are not passed in are
allocated there; work goes to that GPU's current stream."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import _check

QLORA_BF16, QLORA_F32 = 0, 1
QLORA_NORM_LAYER, QLORA_NORM_RMS = 0, 1
QLORA_PREF_SIGMOID, QLORA_PREF_HINGE, QLORA_PREF_SQUARED = 0, 1, 2
QLORA_POLICY_TOKEN_MEAN, QLORA_POLICY_SEQUENCE_MEAN = 0, 1
IGNORE_INDEX = -100

_TYPES = {torch.bfloat16: QLORA_BF16, torch.float32: QLORA_F32}
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float


class _Logits(ctypes.Structure):
    _fields_ = [("logits", _P), ("targets", _P), ("rows", _I64), ("vocab", _I64), ("ld", _I64),
                ("ignore_index", _I64), ("type", ctypes.c_int), ("scale", _F)]


class _Preference(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("length_normalize", ctypes.c_int), ("beta", _F),
                ("label_smoothing", _F), ("margin", _F), ("weight", _F)]


class _Policy(ctypes.Structure):
    _fields_ = [("reduction", ctypes.c_int), ("per_token", ctypes.c_int), ("clip_low", _F),
                ("clip_high", _F), ("kl_coef", _F), ("weight", _F)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of this module's entry points."""
    i, sz, lp = ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(_Logits)
    L.qlora_norm_fwd.argtypes = [i, i, _P, _P, _I64, _I64, i, _P, _P, _F, _P, _P, _P, _P, _P]
    L.qlora_norm_bwd.argtypes = [i, i, _P, _P, _P, _I64, _I64, i, _P, _P, _P, _P, _P, _P, _P, sz,
                                 _P]
    L.qlora_norm_workspace_bytes.restype = sz
    L.qlora_norm_workspace_bytes.argtypes = [_I64, _I64]
    L.qlora_token_logp.argtypes = [lp, _P, _P, _P]
    L.qlora_token_logp_bwd.argtypes = [lp, _P, _P, _P, _I64, _P]
    L.qlora_preference_workspace_bytes.restype = sz
    L.qlora_preference_workspace_bytes.argtypes = [_I64]
    L.qlora_preference_loss.argtypes = [lp, _P, _I64, _P, ctypes.POINTER(_Preference), _P, _P, _P,
                                        _P, _I64, _P, sz, _P]
    L.qlora_policy_workspace_bytes.restype = sz
    L.qlora_policy_workspace_bytes.argtypes = [_I64, _I64]
    L.qlora_policy_loss.argtypes = [lp, _P, _I64, _P, _P, _P, ctypes.POINTER(_Policy), _P, _P, _P,
                                    _I64, _P, sz, _P]


# A call on a few rows is bound by host time: the helpers below stay cheap.

# (None in a PyTorch without GPU support, which still imports this package)
_current_gpu = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # a handle, no Stream object


def _call(name: str, at: int, *args) -> None:
    """The entry point on the current stream of GPU `at`, which is made the
    current GPU (the default stream's handle is 0 on every one)."""
    f = getattr(_lib.lib(), name)
    if _current_gpu() == at:
        status = f(*args, _raw_stream(at))
    else:
        with torch.cuda.device(at):
            status = f(*args, _raw_stream(at))
    if status:
        _check(status, name)


def _need(t: torch.Tensor, dtype, shape, name, at: int):
    """_lib._need, with the passing case first, and on GPU `at` like the call's
    first tensor."""
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == at):
        _lib._need(t, dtype, shape, name)
        raise ValueError(f"{name}: expected on GPU {at}, got {t.device}")


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _room(ws: torch.Tensor, at: int) -> int:
    """The bytes of a caller's workspace, of whatever type."""
    if not (ws.get_device() == at and ws.is_contiguous()):
        raise ValueError(f"workspace: expected a contiguous tensor on GPU {at}, got strides "
                         f"{ws.stride()} on {ws.device}")
    return ws.numel() * ws.element_size()


def _out(t, shape, dtype, device, name, at):
    """The caller's output after a check, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, dtype, shape, name, at)
    return t


def _out_like(t, X, name, at):
    """The same for an output of X's type and shape."""
    if t is None:
        return torch.empty_like(X)
    _need(t, X.dtype, X.shape, name, at)
    return t


# ---------------------------------------------------------------------- norms

class NormOut(NamedTuple):
    Y: torch.Tensor
    H: torch.Tensor                 # X + residual (X itself without one)
    mean: Optional[torch.Tensor]    # FP32 [M], layer norm only
    rstd: Optional[torch.Tensor]    # FP32 [M]


class NormGrads(NamedTuple):
    dX: torch.Tensor
    dgamma: Optional[torch.Tensor]
    dbeta: Optional[torch.Tensor]


def _weight_type(gamma, beta, d, at):
    wt = _TYPES.get(gamma.dtype)
    if wt is None:
        raise ValueError(f"gamma: expected bfloat16 or float32, got {gamma.dtype}")
    _need(gamma, gamma.dtype, (d,), "gamma", at)
    if beta is not None:
        _need(beta, gamma.dtype, (d,), "beta", at)
    return wt


def _matrix_type(X, name):
    """The element type of the call's first tensor, and its GPU."""
    t, at = _TYPES.get(X.dtype), X.get_device()
    if t is None or at < 0 or X.dim() != 2:
        raise ValueError(f"{name}: expected a bfloat16 or float32 matrix on the GPU, got {X.dtype} "
                         f"{tuple(X.shape)} on {X.device}")
    return t, at


def qlora_norm_fwd(X: torch.Tensor, gamma: torch.Tensor, beta: Optional[torch.Tensor] = None,
                   eps: float = 1e-5, kind: int = QLORA_NORM_LAYER,
                   residual: Optional[torch.Tensor] = None, H: Optional[torch.Tensor] = None,
                   Y: Optional[torch.Tensor] = None, save_stats: bool = True) -> NormOut:
    """Norm of X, or of H = X + residual, over the last axis.  Y may be given,
    and with a residual H, which may be X or the residual.  save_stats=False
    leaves out what only the backward needs."""
    ty, at = _matrix_type(X, "X")
    shape = X.shape
    M, d = shape
    dev = X.device
    if not X.is_contiguous():
        _lib._need(X, X.dtype, shape, "X")
    wt = _weight_type(gamma, beta, d, at)
    if residual is not None:
        _need(residual, X.dtype, shape, "residual", at)
        H = _out_like(H, X, "H", at)
    elif H is not None:
        raise ValueError("H: only with a residual, without one the norm is that of X")
    Y = _out_like(Y, X, "Y", at)
    mean = rstd = None
    if save_stats:
        rstd = torch.empty(M, dtype=torch.float32, device=dev)
        if kind == QLORA_NORM_LAYER:
            mean = torch.empty(M, dtype=torch.float32, device=dev)
    _call("qlora_norm_fwd", at, kind, ty, X.data_ptr(), _addr(residual), M, d, wt,
          gamma.data_ptr(), _addr(beta), eps,
          H.data_ptr() if residual is not None else None, Y.data_ptr(),
          _addr(mean), _addr(rstd))
    return NormOut(Y, H if residual is not None else X, mean, rstd)


def qlora_norm_workspace_bytes(M: int, d: int) -> int:
    return int(_lib.lib().qlora_norm_workspace_bytes(M, d))


def qlora_norm_bwd(dY: torch.Tensor, H: torch.Tensor, gamma: torch.Tensor,
                   mean: Optional[torch.Tensor], rstd: torch.Tensor,
                   kind: int = QLORA_NORM_LAYER, dH: Optional[torch.Tensor] = None,
                   need_dgamma: bool = True, need_dbeta: bool = False,
                   dX: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                   dbeta: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> NormGrads:
    """Backward of qlora_norm_fwd for its H, mean and rstd; dH is the gradient
    that reaches H past the norm.  dX may be dY or dH.  need_dbeta is for the
    layer norm alone."""
    ty, at = _matrix_type(H, "H")
    shape = H.shape
    M, d = shape
    dev = H.device
    if not H.is_contiguous():
        _lib._need(H, H.dtype, shape, "H")
    _need(dY, H.dtype, shape, "dY", at)
    wt = _weight_type(gamma, None, d, at)
    _need(rstd, torch.float32, (M,), "rstd", at)
    if kind == QLORA_NORM_LAYER:
        if mean is None:
            raise ValueError("mean: the layer norm's backward needs it")
        _need(mean, torch.float32, (M,), "mean", at)
    if dH is not None:
        _need(dH, H.dtype, shape, "dH", at)
    dX = _out_like(dX, H, "dX", at)
    ws, nbytes = None, 0
    if need_dgamma or need_dbeta:
        dgamma = _out(dgamma, (d,), torch.float32, dev, "dgamma", at) if need_dgamma else None
        dbeta = _out(dbeta, (d,), torch.float32, dev, "dbeta", at) if need_dbeta else None
        if workspace is None:
            nbytes = qlora_norm_workspace_bytes(M, d)
            ws = _lib._workspace(nbytes, dev)
        else:
            ws, nbytes = workspace, _room(workspace, at)
    else:
        dgamma = dbeta = None
    _call("qlora_norm_bwd", at, kind, ty, dY.data_ptr(), H.data_ptr(), _addr(dH), M, d, wt,
          gamma.data_ptr(), _addr(mean), rstd.data_ptr(),
          dX.data_ptr(), _addr(dgamma), _addr(dbeta), _addr(ws),
          nbytes)
    return NormGrads(dX, dgamma, dbeta)


# ---------------------------------------------------------- losses on logits

def _logits(logits, targets, ignore_index, scale):
    """The C description of a logits batch, and its GPU.  Rows may be strided (a padded
    vocabulary); their elements are contiguous."""
    ty, at = _matrix_type(logits, "logits")
    rows, vocab = logits.shape
    ld, inner = logits.stride()
    if rows <= 1:
        ld = max(ld, vocab)
    if (vocab > 1 and inner != 1) or ld < vocab:
        raise ValueError(f"logits: expected rows of contiguous elements, got strides "
                         f"{logits.stride()}")
    _need(targets, torch.int64, (rows,), "targets", at)
    l = _Logits(logits.data_ptr(), targets.data_ptr(), rows, vocab, ld, ignore_index, ty, scale)
    return l, at


def _dlogits(dlogits, logits, l, at):
    """The gradient's buffer and its row stride.  By default the rows are laid
    out as the logits' where these are padded by less than 128 elements or a
    quarter of the vocabulary, else (logits that are a slice of a larger array)
    without gaps."""
    if dlogits is None:
        near = l.ld - l.vocab < 128 or 4 * l.ld <= 5 * l.vocab
        ldd = l.ld if near else l.vocab
        dlogits = torch.empty_strided((l.rows, l.vocab), (ldd, 1), dtype=logits.dtype,
                                      device=logits.device)
        return dlogits, ldd
    ldd = dlogits.stride(0) if l.rows > 1 else max(dlogits.stride(0), l.vocab)
    if (dlogits.dtype != logits.dtype or dlogits.shape != logits.shape or
            dlogits.get_device() != at or (l.vocab > 1 and dlogits.stride(1) != 1) or
            ldd < l.vocab):
        raise ValueError(f"dlogits: expected {logits.dtype} {tuple(logits.shape)} on GPU {at} with "
                         f"contiguous elements in a row, got {dlogits.dtype} "
                         f"{tuple(dlogits.shape)} on {dlogits.device} with strides "
                         f"{dlogits.stride()}")
    return dlogits, ldd


def _space(workspace, need, device, at):
    """(workspace, its bytes): the caller's, or a new one of `need` bytes."""
    if workspace is None:
        return _lib._workspace(need, device), need
    return workspace, _room(workspace, at)


def qlora_token_logp(logits: torch.Tensor, targets: torch.Tensor,
                     ignore_index: int = IGNORE_INDEX, scale: float = 1.0,
                     logp: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None):
    """(logp, lse), FP32 [rows]: log-probability of each row's target under
    softmax(scale * logits) and the log of the row's summed exponentials."""
    l, at = _logits(logits, targets, ignore_index, scale)
    dev = logits.device
    logp = _out(logp, (l.rows,), torch.float32, dev, "logp", at)
    lse = _out(lse, (l.rows,), torch.float32, dev, "lse", at)
    _call("qlora_token_logp", at, l, logp.data_ptr(), lse.data_ptr())
    return logp, lse


def qlora_token_logp_bwd(logits: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                         dlogp: torch.Tensor, ignore_index: int = IGNORE_INDEX, scale: float = 1.0,
                         dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits from upstream gradients of qlora_token_logp's
    log-probabilities, with the lse of that call on the same logits, targets and
    scale; dlogits may be the logits themselves.  A new one has the
    logits' padding, unless that is 128 elements and a quarter of the vocabulary
    or more; the losses' gradients are laid out the same."""
    l, at = _logits(logits, targets, ignore_index, scale)
    _need(lse, torch.float32, (l.rows,), "lse", at)
    _need(dlogp, torch.float32, (l.rows,), "dlogp", at)
    dlogits, ldd = _dlogits(dlogits, logits, l, at)
    _call("qlora_token_logp_bwd", at, l, lse.data_ptr(), dlogp.data_ptr(),
          dlogits.data_ptr(), ldd)
    return dlogits


class PreferenceOut(NamedTuple):
    loss: torch.Tensor                # FP32 [pairs]
    seq_logp: torch.Tensor            # FP32 [2 pairs]
    logp: torch.Tensor                # FP32 [rows]
    dlogits: Optional[torch.Tensor]   # as the logits, padding included


def qlora_preference_workspace_bytes(rows: int) -> int:
    return int(_lib.lib().qlora_preference_workspace_bytes(rows))


def qlora_preference_loss(logits: torch.Tensor, targets: torch.Tensor, offsets: torch.Tensor,
                          ref_logp: Optional[torch.Tensor] = None, kind: int = QLORA_PREF_SIGMOID,
                          beta: float = 0.1, label_smoothing: float = 0.0, margin: float = 0.0,
                          length_normalize: bool = False, weight: Optional[float] = None,
                          ignore_index: int = IGNORE_INDEX, scale: float = 1.0,
                          need_grad: bool = True, dlogits: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None) -> PreferenceOut:
    """Preference loss of the pairs (sequence p preferred to sequence pairs +
    p; offsets int64 [2 pairs + 1] are the sequences' first rows) and the
    gradient of weight * sum of the losses (weight None: 1 / pairs, the mean).
    dlogits may be the logits themselves."""
    l, at = _logits(logits, targets, ignore_index, scale)
    dev = logits.device
    n = offsets.numel()
    if n % 2 == 0:
        raise ValueError(f"offsets: expected 2 pairs + 1 of them, got {n}")
    pairs = n // 2
    _need(offsets, torch.int64, (n,), "offsets", at)
    if ref_logp is not None:
        _need(ref_logp, torch.float32, (l.rows,), "ref_logp", at)
    par = _Preference(kind, 1 if length_normalize else 0, beta, label_smoothing, margin,
                      1.0 / max(1, pairs) if weight is None else weight)
    need = qlora_preference_workspace_bytes(l.rows) if workspace is None else 0
    ws, nbytes = _space(workspace, need, dev, at)
    # each output has memory of its own: whoever keeps one keeps nothing beside it
    logp = torch.empty(l.rows, dtype=torch.float32, device=dev)
    seq_logp, loss = logp.new_empty(2 * pairs), logp.new_empty(pairs)
    ldd = 0
    if need_grad:
        dlogits, ldd = _dlogits(dlogits, logits, l, at)
    else:
        dlogits = None
    _call("qlora_preference_loss", at, l, offsets.data_ptr(), pairs, _addr(ref_logp), par,
          logp.data_ptr(), seq_logp.data_ptr(), loss.data_ptr(),
          _addr(dlogits), ldd, ws.data_ptr(), nbytes)
    return PreferenceOut(loss, seq_logp, logp, dlogits)


class PolicyOut(NamedTuple):
    stats: torch.Tensor               # FP32 [4]: loss, policy term, KL, clipped share
    logp: torch.Tensor                # FP32 [rows]
    dlogits: Optional[torch.Tensor]   # as the logits, padding included


def qlora_policy_workspace_bytes(rows: int, sequences: int) -> int:
    return int(_lib.lib().qlora_policy_workspace_bytes(rows, sequences))


def qlora_policy_loss(logits: torch.Tensor, targets: torch.Tensor, offsets: torch.Tensor,
                      advantages: torch.Tensor, old_logp: Optional[torch.Tensor] = None,
                      ref_logp: Optional[torch.Tensor] = None, clip_low: float = 0.2,
                      clip_high: float = 0.2, kl_coef: float = 0.0, per_token: bool = False,
                      reduction: int = QLORA_POLICY_TOKEN_MEAN, weight: float = 1.0,
                      ignore_index: int = IGNORE_INDEX, scale: float = 1.0,
                      need_grad: bool = True, dlogits: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None) -> PolicyOut:
    """Clipped policy loss with a KL term over the sequences whose first rows
    are offsets (int64 [sequences + 1]), and the gradient of weight * loss.
    advantages: FP32 [sequences], or [rows] with per_token.  dlogits may be
    the logits themselves."""
    l, at = _logits(logits, targets, ignore_index, scale)
    dev = logits.device
    seqs = offsets.numel() - 1
    if seqs < 0:
        raise ValueError("offsets: expected sequences + 1 of them")
    _need(offsets, torch.int64, (seqs + 1,), "offsets", at)
    _need(advantages, torch.float32, (l.rows if per_token else seqs,), "advantages", at)
    if old_logp is not None:
        _need(old_logp, torch.float32, (l.rows,), "old_logp", at)
    if ref_logp is not None:
        _need(ref_logp, torch.float32, (l.rows,), "ref_logp", at)
    par = _Policy(reduction, 1 if per_token else 0, clip_low, clip_high, kl_coef, weight)
    need = qlora_policy_workspace_bytes(l.rows, seqs) if workspace is None else 0
    ws, nbytes = _space(workspace, need, dev, at)
    logp = torch.empty(l.rows, dtype=torch.float32, device=dev)
    stats = logp.new_empty(4)   # memory of its own: whoever keeps it keeps nothing beside it
    ldd = 0
    if need_grad:
        dlogits, ldd = _dlogits(dlogits, logits, l, at)
    else:
        dlogits = None
    _call("qlora_policy_loss", at, l, offsets.data_ptr(), seqs, advantages.data_ptr(),
          _addr(old_logp), _addr(ref_logp), par, logp.data_ptr(),
          stats.data_ptr(), _addr(dlogits), ldd, ws.data_ptr(),
          nbytes)
    return PolicyOut(stats, logp, dlogits)
