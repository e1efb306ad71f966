"""Host checks of the entry points around the linear layers: every bad argument
is refused before anything is enqueued (fake device addresses are never
dereferenced), and the binding refuses tensors it cannot describe."""
import ctypes

import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from bit_quantized_lora_quantize_amd import _train

OK, ENULL, ESHAPE, EALIGN, EWS = 0, -1, -2, -3, -4
P = ctypes.c_void_p
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    import os
    from bit_quantized_lora_quantize_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return q.lib()


def _fwd(L, **kw):
    a = dict(kind=0, type=0, X=0x1000, R=None, M=4, d=64, w_type=1, gamma=0x2000, beta=0x3000,
             eps=1e-5, H=None, Y=0x4000, mean=0x5000, rstd=0x6000)
    a.update(kw)
    return L.qlora_norm_fwd(*a.values(), None)


def test_norm_forward_refusals(L):
    assert _fwd(L, kind=2) == ESHAPE and _fwd(L, type=2) == ESHAPE and _fwd(L, w_type=-1) == ESHAPE
    assert _fwd(L, M=-1) == ESHAPE and _fwd(L, M=(1 << 21) + 1) == ESHAPE
    assert _fwd(L, d=0) == ESHAPE and _fwd(L, d=(1 << 21) + 1) == ESHAPE
    assert _fwd(L, eps=-1.0) == ESHAPE and _fwd(L, eps=float("nan")) == ESHAPE
    assert _fwd(L, kind=1) == ESHAPE                       # an RMS norm has no beta
    for name in ("X", "gamma", "Y"):
        assert _fwd(L, **{name: None}) == ENULL
    assert _fwd(L, R=0x7000) == ENULL                      # a residual needs H
    for name in ("X", "Y"):
        assert _fwd(L, **{name: 0x1001}) == EALIGN
        assert _fwd(L, **{name: 0x1002, "type": 1}) == EALIGN
    assert _fwd(L, gamma=0x2002) == EALIGN and _fwd(L, rstd=0x6001) == EALIGN
    assert _fwd(L, M=0, X=None, Y=None, gamma=None) == OK


def _bwd(L, **kw):
    a = dict(kind=0, type=1, dY=0x1000, H=0x2000, dH=None, M=4, d=64, w_type=0, gamma=0x3000,
             mean=0x4000, rstd=0x5000, dX=0x6000, dgamma=0x7000, dbeta=0x8000, ws=0x9000, n=BIG)
    a.update(kw)
    return L.qlora_norm_bwd(*a.values(), None)


def test_norm_backward_refusals(L):
    assert _bwd(L, kind=-1) == ESHAPE and _bwd(L, type=7) == ESHAPE and _bwd(L, w_type=2) == ESHAPE
    assert _bwd(L, M=-1) == ESHAPE and _bwd(L, d=0) == ESHAPE
    for name in ("dY", "H", "gamma", "mean", "rstd", "dX", "ws"):
        assert _bwd(L, **{name: None}) == ENULL
    assert _bwd(L, dY=0x1002) == EALIGN and _bwd(L, dH=0x1001) == EALIGN
    assert _bwd(L, ws=0x9008) == EALIGN and _bwd(L, dgamma=0x7002) == EALIGN
    need = q.qlora_norm_workspace_bytes(4, 64)
    assert need > 0 and _bwd(L, n=need - 1) == EWS
    assert _bwd(L, M=0, dgamma=None, dbeta=None, ws=None, n=0) == OK
    assert q.qlora_norm_workspace_bytes(-1, 64) == 0 and q.qlora_norm_workspace_bytes(4, 0) == 0
    assert q.qlora_norm_workspace_bytes(1 << 21, 64) > 0


def _l(**kw):
    a = dict(logits=0x1000, targets=0x2000, rows=4, vocab=100, ld=100, ignore_index=-100, type=0,
             scale=1.0)
    a.update(kw)
    return _train._Logits(*a.values())


BAD_LOGITS = [({"rows": -1}, ESHAPE), ({"rows": (1 << 21) + 1}, ESHAPE), ({"vocab": 0}, ESHAPE),
              ({"vocab": (1 << 24) + 1, "ld": 1 << 25}, ESHAPE), ({"ld": 99}, ESHAPE),
              ({"type": 2}, ESHAPE), ({"scale": 0.0}, ESHAPE), ({"scale": float("inf")}, ESHAPE),
              ({"scale": float("nan")}, ESHAPE), ({"logits": None}, ENULL),
              ({"targets": None}, ENULL), ({"logits": 0x1001}, EALIGN),
              ({"logits": 0x1002, "type": 1}, EALIGN), ({"targets": 0x2004}, EALIGN)]


def _pref(L, l, **kw):
    a = dict(off=0x3000, pairs=1, ref=0x4000, par=None, logp=0x5000, seq=0x6000, loss=0x7000,
             d=0x8000, ldd=100, ws=0x9000, n=BIG)
    par = dict(kind=0, length_normalize=0, beta=0.1, label_smoothing=0.0, margin=0.0, weight=1.0)
    par.update({k: kw.pop(k) for k in list(kw) if k in par})
    a.update(kw)
    if "par" not in kw:
        a["par"] = ctypes.byref(_train._Preference(*par.values()))
    return L.qlora_preference_loss(l, *a.values(), None)


def _pol(L, l, **kw):
    a = dict(off=0x3000, seqs=1, adv=0x3800, old=0x4000, ref=0x4800, par=None, logp=0x5000,
             stats=0x6000, d=0x8000, ldd=100, ws=0x9000, n=BIG)
    par = dict(reduction=0, per_token=0, clip_low=0.2, clip_high=0.2, kl_coef=0.1, weight=1.0)
    par.update({k: kw.pop(k) for k in list(kw) if k in par})
    a.update(kw)
    if "par" not in kw:
        a["par"] = ctypes.byref(_train._Policy(*par.values()))
    return L.qlora_policy_loss(l, *a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_LOGITS)
def test_bad_logits_are_refused_everywhere(L, bad, status):
    l = _l(**bad)
    assert L.qlora_token_logp(l, P(0x5000), P(0x6000), None) == status
    assert L.qlora_token_logp_bwd(l, P(0x5000), P(0x6000), P(0x7000), 1 << 25, None) == status
    assert _pref(L, l, ldd=1 << 25) == status
    assert _pol(L, l, ldd=1 << 25) == status


def test_token_logp_refusals(L):
    f, b = L.qlora_token_logp, L.qlora_token_logp_bwd
    l = _l()
    assert f(None, P(0x5000), None, None) == ENULL and f(l, None, P(0x5000), None) == ENULL
    assert f(l, P(0x5002), None, None) == EALIGN and f(l, P(0x5000), P(0x6002), None) == EALIGN
    assert f(_l(rows=0, logits=None, targets=None), None, None, None) == OK
    ok = (P(0x5000), P(0x6000), P(0x7000))
    for i in range(3):
        assert b(l, *[None if i == j else p for j, p in enumerate(ok)], 100, None) == ENULL
    assert b(l, *ok, 99, None) == ESHAPE
    assert b(l, P(0x5000), P(0x6000), P(0x7001), 100, None) == EALIGN
    assert b(l, P(0x5000), P(0x6000), P(0x1000), 101, None) == ESHAPE   # in place: the same rows
    assert b(_l(rows=0, logits=None, targets=None), None, None, None, 0, None) == OK


def test_preference_refusals(L):
    l = _l()
    assert _pref(L, None) == ENULL and _pref(L, l, par=None) == ENULL
    assert _pref(L, l, pairs=-1) == ESHAPE and _pref(L, l, pairs=(1 << 20) + 1) == ESHAPE
    assert _pref(L, l, kind=3) == ESHAPE
    for beta in (0.0, -1.0, float("inf"), float("nan")):
        assert _pref(L, l, beta=beta) == ESHAPE
    assert _pref(L, l, label_smoothing=1.0) == ESHAPE
    assert _pref(L, l, label_smoothing=-0.1) == ESHAPE
    assert _pref(L, l, kind=1, label_smoothing=0.1) == ESHAPE
    assert _pref(L, l, kind=2, margin=0.1) == ESHAPE
    assert _pref(L, l, margin=float("inf")) == ESHAPE
    assert _pref(L, l, weight=float("nan")) == ESHAPE
    for name in ("off", "logp", "seq", "loss", "ws"):
        assert _pref(L, l, **{name: None}) == ENULL
    assert _pref(L, l, off=0x3004) == EALIGN and _pref(L, l, ref=0x4002) == EALIGN
    assert _pref(L, l, ws=0x9004) == EALIGN and _pref(L, l, d=0x8001) == EALIGN
    assert _pref(L, l, ldd=99) == ESHAPE
    need = q.qlora_preference_workspace_bytes(4)
    assert need > 0 and _pref(L, l, n=need - 1) == EWS
    assert q.qlora_preference_workspace_bytes(-1) == 0
    assert _pref(L, _l(rows=0), pairs=0) == OK


def test_policy_refusals(L):
    l = _l()
    assert _pol(L, None) == ENULL and _pol(L, l, par=None) == ENULL
    assert _pol(L, l, seqs=-1) == ESHAPE and _pol(L, l, reduction=2) == ESHAPE
    assert _pol(L, l, clip_low=-0.1) == ESHAPE and _pol(L, l, clip_low=1.1) == ESHAPE
    assert _pol(L, l, clip_high=-0.1) == ESHAPE and _pol(L, l, clip_high=float("inf")) == ESHAPE
    assert _pol(L, l, kl_coef=-1.0) == ESHAPE and _pol(L, l, weight=float("inf")) == ESHAPE
    assert _pol(L, l, ref=None) == ENULL                   # a KL term needs the reference
    for name in ("off", "adv", "logp", "stats", "ws"):
        assert _pol(L, l, **{name: None}) == ENULL
    assert _pol(L, l, adv=0x3802) == EALIGN and _pol(L, l, old=0x4001) == EALIGN
    assert _pol(L, l, d=0x8001) == EALIGN and _pol(L, l, ldd=99) == ESHAPE
    need = q.qlora_policy_workspace_bytes(4, 1)
    assert need > 0 and _pol(L, l, n=need - 1) == EWS
    assert q.qlora_policy_workspace_bytes(-1, 1) == 0 and q.qlora_policy_workspace_bytes(1, -1) == 0


def test_binding_refuses_tensors_it_cannot_describe(L):
    """On the host alone: tensors that are not on the GPU, of the wrong type or
    shape are refused before any call."""
    x, g = torch.zeros(4, 64), torch.ones(64)
    t, off = torch.zeros(4, dtype=torch.int64), torch.tensor([0, 2, 4])
    for bad in (lambda: q.qlora_norm_fwd(x, g), lambda: q.qlora_norm_fwd(x.half(), g),
                lambda: q.qlora_norm_fwd(x[0], g),
                lambda: q.qlora_norm_bwd(x, x, g, None, torch.ones(4)),
                lambda: q.qlora_token_logp(x, t), lambda: q.qlora_token_logp(x.t(), t),
                lambda: q.qlora_token_logp(x.to(torch.int32), t),
                lambda: q.qlora_preference_loss(x, t, off),
                lambda: q.qlora_policy_loss(x, t, off, torch.ones(2))):
        with pytest.raises(ValueError):
            bad()


def test_rms_norm_backward_has_no_beta(L):
    """An RMS norm takes no beta, so its gradient is refused as the forward refuses beta."""
    assert _bwd(L, kind=1, mean=None) == ESHAPE
    assert _bwd(L, kind=1, mean=None, dgamma=None) == ESHAPE
    assert _bwd(L, kind=1, mean=None, dY=None, dbeta=None) == ENULL
