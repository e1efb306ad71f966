"""GPU parity of the norms (forward with the residual addition, backward with
and without weight gradients) against float64, over widths around every vector
and register boundary, odd sizes, unaligned rows and in-place outputs.

Tolerances: BF16 outputs one rounding (2^-8 of the value).  FP32 outputs: a
value passes about ten FP32 operations and two tree sums, each 2^-24, so 1e-6
relative in norm and 5e-6 of the largest value leave a factor of ten.  Weight
gradients are sums over up to 4096 rows in FP32: rounding grows as sqrt(rows)
2^-24 = 4e-6, bound 1e-5."""
import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from parity_util import assert_close, say
import train_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
KINDS = {"layer": q.QLORA_NORM_LAYER, "rms": q.QLORA_NORM_RMS}
EPS = 1e-5


def _draw(seed, shape, dtype, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype)


def _tol(dtype, f32_fro=1e-6, f32_max=5e-6):
    return ((ref.BF16_TOL, ref.BF16_TOL) if dtype == torch.bfloat16 else (f32_fro, f32_max))


def _unaligned(t, by=1):
    """The same values on the GPU, starting `by` elements into an allocation."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)
    v = buf[by:].view(t.shape)
    v.copy_(t)
    return v


WIDTHS = [1, 2, 7, 8, 9, 63, 64, 65, 255, 511, 512, 520, 1000, 1024, 1025, 2048, 2056, 4096, 5003,
          8192, 8200, 11008, 16384, 16392, 22016, 32768, 40001, 70000]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_forward(width, kind, dtype):
    rows = 5 if width > 1024 else 37
    residual = width % 2 == 0
    wt = torch.float32 if width % 3 == 0 else torch.bfloat16
    say(f"norm forward: {kind} {rows}x{width} {dtype} residual={residual} weights {wt}")
    X = _draw(width, (rows, width), dtype, 2.0, 0.5)
    R = _draw(width + 1, (rows, width), dtype) if residual else None
    gamma = _draw(width + 2, (width,), wt, 0.2, 1.0)
    beta = _draw(width + 3, (width,), wt, 0.2) if kind == "layer" and width % 5 else None
    dev = [None if t is None else t.to(DEV) for t in (X, R, gamma, beta)]
    o = q.qlora_norm_fwd(dev[0], dev[2], dev[3], eps=EPS, kind=KINDS[kind], residual=dev[1])
    y, h, mean, rstd = ref.norm_fwd(X, R, gamma, beta, EPS, kind == "layer")
    if residual:
        assert torch.equal(o.H.cpu().double(), h), "H is not the rounded sum"
    else:
        assert o.H is dev[0]
    # a layer norm of width 1 or 2 of near-equal values has rstd ~ 1 / sqrt(eps):
    # the centred value's absolute rounding (2^-24 of |H|) is scaled by it
    amp = float((h.abs().amax(1) * rstd).max())
    fro, mx = _tol(dtype, 1e-6 + 2.0 ** -23 * amp * (width <= 2), 5e-6 + 2.0 ** -22 * amp * (width <= 2))
    assert_close("Y", ref.f64(o.Y), y, fro, mx)
    assert_close("rstd", ref.f64(o.rstd), rstd, 2e-6, 5e-6)
    if kind == "layer":
        assert ref.max_err(o.mean, mean) <= 1e-6 * float(h.abs().max())
    else:
        assert o.mean is None
    lean = q.qlora_norm_fwd(dev[0], dev[2], dev[3], eps=EPS, kind=KINDS[kind], residual=dev[1],
                            save_stats=False)
    assert lean.rstd is None and torch.equal(lean.Y, o.Y)


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward(width, kind, dtype):
    rows = 9 if width > 1024 else 301
    wt = torch.float32 if width % 3 == 0 else torch.bfloat16
    with_dh = width % 2 == 1
    say(f"norm backward: {kind} {rows}x{width} {dtype} dH={with_dh} weights {wt}")
    # values of spread 2 around distinct levels: no row of width 2 is near constant
    X = _draw(width, (rows, width), dtype, 2.0, 0.5)
    if width == 2:
        X[:, 1] = X[:, 0] + 1.0 + X[:, 1].abs()
    dY = _draw(width + 1, (rows, width), dtype)
    dH = _draw(width + 2, (rows, width), dtype) if with_dh else None
    gamma = _draw(width + 3, (width,), wt, 0.2, 1.0)
    _, _, mean, rstd = ref.norm_fwd(X, None, gamma, None, EPS, kind == "layer")
    dx, dg, db = ref.norm_bwd(X, gamma, EPS, kind == "layer", dY, dH)
    Xd, dYd, dHd, gd = (None if t is None else t.to(DEV) for t in (X, dY, dH, gamma))
    md = mean.float().to(DEV) if kind == "layer" else None
    rd = rstd.float().to(DEV)
    o = q.qlora_norm_bwd(dYd, Xd, gd, md, rd, kind=KINDS[kind], dH=dHd, need_dgamma=True,
                         need_dbeta=kind == "layer")
    # narrow layer norms: dX is a difference of values of size rstd |u| that
    # nearly cancel, so the bound is on those
    big = float((ref.f64(dY) * ref.f64(gamma) * rstd[:, None]).abs().max())
    fro, mx = _tol(dtype, 2e-6, 1e-5)
    if width <= 2:
        assert ref.max_err(o.dX, dx) <= mx * max(big, float(dx.abs().max()))
    else:
        assert_close("dX", ref.f64(o.dX), dx, fro, mx)
    if width > 2:
        assert_close("dgamma", ref.f64(o.dgamma), dg, 1e-5, 1e-5)
    if kind == "layer":
        assert_close("dbeta", ref.f64(o.dbeta), db, 1e-5, 1e-5)
    frozen = q.qlora_norm_bwd(dYd, Xd, gd, md, rd, kind=KINDS[kind], dH=dHd, need_dgamma=False)
    assert frozen.dgamma is None and torch.equal(frozen.dX, o.dX)
    again = q.qlora_norm_bwd(dYd, Xd, gd, md, rd, kind=KINDS[kind], dH=dHd, need_dgamma=True,
                             need_dbeta=kind == "layer")
    assert torch.equal(again.dX, o.dX) and torch.equal(again.dgamma, o.dgamma)


@pytest.mark.parametrize("rows,width", [(1, 4096), (2, 64), (3, 1000), (4096, 256), (4097, 72),
                                        (1500, 4096), (2049, 1032)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_weight_gradients_over_many_rows(rows, width, dtype):
    say(f"norm weight gradients: {rows}x{width} {dtype}")
    X, dY = _draw(1, (rows, width), dtype, 1.5, 0.2), _draw(2, (rows, width), dtype)
    gamma = _draw(3, (width,), torch.float32, 0.2, 1.0)
    _, _, mean, rstd = ref.norm_fwd(X, None, gamma, None, EPS, True)
    n = (ref.f64(X) - mean[:, None]) * rstd[:, None]
    o = q.qlora_norm_bwd(dY.to(DEV), X.to(DEV), gamma.to(DEV), mean.float().to(DEV),
                         rstd.float().to(DEV), need_dgamma=True, need_dbeta=True)
    assert_close("dgamma", ref.f64(o.dgamma), (ref.f64(dY) * n).sum(0), 1e-5, 1e-5)
    assert_close("dbeta", ref.f64(o.dbeta), ref.f64(dY).sum(0), 1e-5, 1e-5)
    only = q.qlora_norm_bwd(dY.to(DEV), X.to(DEV), gamma.to(DEV), mean.float().to(DEV),
                            rstd.float().to(DEV), need_dgamma=False, need_dbeta=True)
    assert only.dgamma is None and torch.equal(only.dbeta, o.dbeta)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradient_against_differences(kind):
    rows, width = 6, 96
    X = _draw(5, (rows, width), torch.float32, 1.5, 0.3)
    gamma, beta = _draw(6, (width,), torch.float32, 0.2, 1.0), torch.zeros(width)
    dY, dH = _draw(7, (rows, width), torch.float32), _draw(8, (rows, width), torch.float32)
    fw = q.qlora_norm_fwd(X.to(DEV), gamma.to(DEV), eps=EPS, kind=KINDS[kind])
    o = q.qlora_norm_bwd(dY.to(DEV), fw.H, gamma.to(DEV), fw.mean, fw.rstd, kind=KINDS[kind],
                         dH=dH.to(DEV), need_dgamma=True)
    layer = kind == "layer"
    fx = lambda h: ref.norm_loss(h, f[0], f[1], EPS, layer, f[2], f[3])  # noqa: E731
    f = [ref.f64(t) for t in (gamma, beta, dY, dH)]
    v = ref.f64(_draw(9, (rows, width), torch.float32)) + ref.f64(o.dX)
    got = float((ref.f64(o.dX) * v).sum())
    # the difference's own error is step^2 of the third derivative, about 1e-8
    assert abs(got - ref.slope(fx, ref.f64(X), v, 1e-4)) <= 2e-5 * abs(got)
    fg = lambda g: ref.norm_loss(ref.f64(X), g, f[1], EPS, layer, f[2], f[3])  # noqa: E731
    v = ref.f64(_draw(10, (width,), torch.float32)) + ref.f64(o.dgamma)
    got = float((ref.f64(o.dgamma) * v).sum())
    assert abs(got - ref.slope(fg, f[0], v, 1e-4)) <= 2e-5 * abs(got)


@pytest.mark.parametrize("width", [72, 1001, 4096, 40001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unaligned_and_in_place_give_the_same_bits(width, dtype):
    rows = 11
    X, R = _draw(11, (rows, width), dtype), _draw(12, (rows, width), dtype)
    gamma, beta = _draw(13, (width,), dtype, 0.2, 1.0), _draw(14, (width,), dtype)
    dY, dH = _draw(15, (rows, width), dtype), _draw(16, (rows, width), dtype)
    d = [t.to(DEV) for t in (X, R, gamma, beta, dY, dH)]
    base = q.qlora_norm_fwd(d[0], d[2], d[3], eps=EPS, residual=d[1])
    u = [_unaligned(t) for t in (X, R, gamma, beta)]
    o = q.qlora_norm_fwd(u[0], u[2], u[3], eps=EPS, residual=u[1], H=u[1], Y=_unaligned(X, 3))
    assert o.H.data_ptr() == u[1].data_ptr()
    assert torch.equal(o.H, base.H) and torch.equal(o.rstd, base.rstd)
    # other alignments may round a row's sums in another order
    assert_close("Y", ref.f64(o.Y), ref.f64(base.Y), *_tol(dtype))
    in_x = d[0].clone()
    o = q.qlora_norm_fwd(in_x, d[2], d[3], eps=EPS, residual=d[1], H=in_x)
    assert torch.equal(in_x, base.H) and torch.equal(o.Y, base.Y)
    plain = q.qlora_norm_fwd(d[0], d[2], d[3], eps=EPS)
    in_x = d[0].clone()
    q.qlora_norm_fwd(in_x, d[2], d[3], eps=EPS, Y=in_x)
    assert torch.equal(in_x, plain.Y)
    gr = q.qlora_norm_bwd(d[4], base.H, d[2], base.mean, base.rstd, dH=d[5], need_dbeta=True)
    for into in (4, 5):
        buf = d[into].clone()
        args = [buf if into == 4 else d[4], base.H, d[2], base.mean, base.rstd]
        o = q.qlora_norm_bwd(*args, dH=buf if into == 5 else d[5], need_dbeta=True, dX=buf)
        assert torch.equal(buf, gr.dX) and torch.equal(o.dgamma, gr.dgamma)
        assert torch.equal(o.dbeta, gr.dbeta)
    o = q.qlora_norm_bwd(_unaligned(dY), _unaligned(base.H.cpu()), u[2], base.mean, base.rstd,
                         dH=_unaligned(dH, 3), need_dbeta=True)
    assert_close("dX", ref.f64(o.dX), ref.f64(gr.dX), *_tol(dtype, 2e-6, 1e-5))
    assert_close("dgamma", ref.f64(o.dgamma), ref.f64(gr.dgamma), 1e-5, 1e-5)


def test_rows_of_zeros_infinities_and_offsets():
    """Constant rows have variance 0 (rstd = 1 / sqrt(eps)); an infinity or NaN
    stays in its row; a large common offset does not spoil the variance."""
    width = 1000
    X = _draw(20, (6, width), torch.float32)
    X[0] = 0.0
    X[1] = 3.25
    X[2, 5] = float("inf")
    X[3, 7] = float("nan")
    X[4] += 1000.0
    gamma = torch.ones(width)
    o = q.qlora_norm_fwd(X.to(DEV), gamma.to(DEV), eps=EPS)
    y = o.Y.cpu()
    assert (y[0] == 0).all()
    # the mean of a constant row is the constant within its rounding
    assert y[1].abs().max() <= 3.25 * 2.0 ** -23 / EPS ** 0.5
    assert torch.isnan(y[2]).any() and torch.isnan(y[3]).all()
    want = ref.norm_fwd(X[4:], None, gamma, None, EPS, True)[0]
    # row 4: values of size 1000 with spread 1 carry 1000 * 2^-24 = 6e-5 each from the mean
    assert ref.max_err(y[4], want[0]) <= 1000 * 2.0 ** -23
    assert ref.max_err(y[5], want[1]) <= 2e-5
    r = q.qlora_norm_fwd(torch.zeros(2, width, device=DEV), gamma.to(DEV), eps=0.0,
                         kind=q.QLORA_NORM_RMS)
    assert torch.isinf(r.rstd).all()


def test_empty_batch_and_another_stream():
    gamma = torch.ones(64, device=DEV)
    e = torch.empty(0, 64, device=DEV)
    assert q.qlora_norm_fwd(e, gamma).Y.shape == (0, 64)
    dg, db = torch.full((64,), 7.0, device=DEV), torch.full((64,), 7.0, device=DEV)
    q.qlora_norm_bwd(e, e, gamma, torch.empty(0, device=DEV), torch.empty(0, device=DEV),
                     need_dbeta=True, dgamma=dg, dbeta=db)
    assert (dg == 0).all() and (db == 0).all()
    X = _draw(30, (513, 1024), torch.bfloat16).to(DEV)
    gamma = torch.ones(1024, device=DEV)
    want = q.qlora_norm_fwd(X, gamma).Y
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = q.qlora_norm_fwd(X, gamma).Y
    st.synchronize()
    assert torch.equal(got, want)
