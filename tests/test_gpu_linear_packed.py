"""The NF4 layer's backward from an input kept in 8 bits, on the GPU, against the
layer's definition in 64 bits and against the backward from the restored
input."""
import pytest
import torch

import adapters_ref as ref
import bit_quantized_lora_quantize_amd as q
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _layer(seed, M, d_in, d_out, r):
    g = torch.Generator().manual_seed(seed)
    W = torch.randn(d_out, d_in, generator=g) * 0.02
    bf = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    A, B = (bf(r, d_in).float() / d_in ** 0.5).bfloat16(), (bf(d_out, r).float() * 0.1).bfloat16()
    w = q.qlora_quantize_nf4(W.to(DEV))
    return w, bf(M, d_in), bf(M, d_out), A, B


def _exact(w, X, T, dY, A, B, s, keep=None, rest=1.0):
    """{dX, dA, dB} and bounds; keep: the LoRA branch's mask, rest: 1 / (1 - p) in s already."""
    Wh = ref.f64(q.qlora_dequant_bf16(w))
    X, T, dY, A, B = (ref.f64(t) for t in (X, T, dY, A, B))
    M, N = dY.shape
    r = A.shape[0]
    if keep is None:
        keep = torch.ones_like(X)
    U = dY @ B * s
    eU = (N + 2) * ref.ADD * (dY.abs() @ B.abs()) * abs(s)
    dX = dY @ Wh + keep * (U @ A)
    mag = dY.abs() @ Wh.abs() + U.abs() @ A.abs()
    e = (eU + ref.U16 * U.abs()) @ A.abs() + (N + 2 * r + 2) * ref.ADD * mag
    out = {"dX": dX, "dA": U.t() @ (keep * X), "dB": dY.t() @ T}
    t = ref.U24 + (3 * M + 2) * ref.ADD
    bound = {"dX": ref.SLACK * (e + ref.U8 * (dX.abs() + e)),
             "dA": ref.SLACK * ((eU + t * U.abs()).t() @ (keep * X).abs()),
             "dB": ref.SLACK * t * (dY.abs().t() @ T.abs())}
    return out, bound


@pytest.mark.parametrize("M,d_in,d_out,r", [(9, 64, 3, 4), (300, 128, 7, 64), (1, 64, 1, 1), (1, 64, 64, 8), (5, 128, 77, 3), (16, 256, 200, 16), (17, 64, 128, 16), (100, 320, 136, 20),
                                            (130, 512, 257, 64), (333, 192, 520, 50), (257, 256, 264, 128), (90, 128, 96, 256),
                                            (2500, 128, 128, 16), (700, 192, 1100, 16), (16400, 64, 64, 8), (16390, 64, 67, 8)])
def test_backward(M, d_in, d_out, r):
    say(f"packed backward M={M} {d_in}->{d_out} r={r}")
    w, X, dY, A, B = _layer(M + r, M, d_in, d_out, r)
    alpha = 2.0 * r
    Xd, dYd, Ad, Bd = (t.to(DEV) for t in (X, dY, A, B))
    T = torch.empty(M, r, device=DEV)
    q.qlora_linear_fwd(w, Xd, Ad, Bd, alpha, T_save=T)
    X8 = q.qlora_pack8(Xd)
    back = q.qlora_unpack8(X8)
    dX, dA, dB = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, alpha, T)
    want, bound = _exact(w, back, T, dY, A, B, 2.0)
    for name, got in (("dA", dA), ("dB", dB), ("dX", dX)):
        ref.inside(got, want[name], bound[name], name)
    # dX does not see X: two roundings of the same sum from the BF16 input's
    other = q.qlora_linear_bwd(w, back, dYd, Ad, Bd, alpha, T_saved=T)[0]
    ref.inside(dX, ref.f64(other), 2 * bound["dX"], "dX against the BF16 input's")
    none, dA2, dB2 = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, alpha, T, need_dx=False)
    assert none is None and torch.equal(dA2, dA) and torch.equal(dB2, dB)


@pytest.mark.parametrize("M", [7, 16, 40, 200, 16700])
@pytest.mark.parametrize("saved", [False, True])
def test_dropout(M, saved):
    d_in, d_out, r, p = (128, 96, 16, 0.25) if M < 1000 else (64, 64, 8, 0.25)
    w, X, dY, A, B = _layer(M, M, d_in, d_out, r)
    drop = q.Dropout(p, seed=77, offset=5)
    if saved:
        drop = drop.saved_mask(M, d_in)
    Xd, dYd, Ad, Bd = (t.to(DEV) for t in (X, dY, A, B))
    T = torch.empty(M, r, device=DEV)
    alpha = 2.0 * r
    q.qlora_linear_fwd_dropout(w, Xd, Ad, Bd, alpha, drop, T_save=T)
    ones = torch.ones(M, d_in, dtype=torch.bfloat16, device=DEV)
    keep = ref.f64(q.qlora_dropout_mask(ones, q.Dropout(p, seed=77, offset=5))[0])
    assert 0.5 < float(keep.mean()) < 0.95
    X8 = q.qlora_pack8(Xd)
    back = q.qlora_unpack8(X8)
    dX, dA, dB = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, alpha, T, dropout=drop)
    s = float(torch.tensor(2.0) / (torch.tensor(1.0) - torch.tensor(p)))
    want, bound = _exact(w, back, T, dY, A, B, s, keep)
    for name, got in (("dA", dA), ("dB", dB), ("dX", dX)):
        ref.inside(got, want[name], bound[name], name)
    other = q.qlora_linear_bwd_dropout(w, back, dYd, Ad, Bd, alpha, drop, T_saved=T)[0]
    ref.inside(dX, ref.f64(other), 2 * bound["dX"], "dX against the BF16 input's")


def test_without_dropped_elements_as_without_dropout():
    w, X, dY, A, B = _layer(3, 70, 128, 64, 8)
    Xd, dYd, Ad, Bd = (t.to(DEV) for t in (X, dY, A, B))
    T = torch.empty(70, 8, device=DEV)
    q.qlora_linear_fwd(w, Xd, Ad, Bd, 16.0, T_save=T)
    X8 = q.qlora_pack8(Xd)
    a = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, 16.0, T)
    b = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, 16.0, T, dropout=q.Dropout(0.0, seed=1))
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_tokens_and_given_buffers():
    w, X, dY, A, B = _layer(4, 60, 64, 72, 8)
    Xd, dYd, Ad, Bd = (t.to(DEV) for t in (X, dY, A, B))
    dA, dB = torch.full((8, 64), 4.0, device=DEV), torch.full((72, 8), 4.0, device=DEV)
    q.qlora_linear_bwd_packed(w, q.qlora_pack8(Xd[:0]), dYd[:0], Ad, Bd, 16.0, torch.empty(0, 8, device=DEV), dA=dA, dB=dB)
    assert (dA == 0).all() and (dB == 0).all()
    T = torch.empty(60, 8, device=DEV)
    q.qlora_linear_fwd(w, Xd, Ad, Bd, 16.0, T_save=T)
    X8 = q.qlora_pack8(Xd)
    ws = torch.full((q.qlora_workspace_bytes(q.QLORA_OP_BWD_PACKED, 72, 64, 60, 8) // 4 + 4,), float("nan"), device=DEV)
    first = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, 16.0, T, workspace=ws)
    second = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, 16.0, T, dA=dA, dB=dB)
    assert torch.equal(first[1], dA) and torch.equal(first[2], dB) and torch.equal(first[0], second[0])
