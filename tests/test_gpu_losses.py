"""GPU parity of the token log-probabilities, the preference loss and the
clipped policy loss against float64, with gradients from float64 autograd and
from differences.

Tolerances.  A log-probability of size up to 40 is a difference of FP32 values
plus the log of a sum: 5e-6 + 1e-6 |value|.  A probability's exponent of size up
to 60 is rounded at 2^-24 of it, 4e-6, so FP32 gradients hold 1e-5 in norm; a
loss's slope adds the error of the log-probabilities it comes from (up to 100
tokens x 5e-6 x beta = 0.1 .. 0.5, partly cancelling): 5e-5.  BF16 gradients: one
rounding, 2^-8 of the value, on top."""
import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from parity_util import assert_close, say
import train_ref as ref
from train_ref import IGNORE

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
INF = float("inf")
KINDS = {"sigmoid": q.QLORA_PREF_SIGMOID, "hinge": q.QLORA_PREF_HINGE,
         "squared": q.QLORA_PREF_SQUARED}


def _logits(seed, rows, vocab, dtype, pad=0, shift=0, lift=6.0):
    """(view on the GPU, targets on the CPU): rows of stride vocab + pad that
    start `shift` elements into the allocation; everything around is NaN."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 2.5
    t = torch.randint(0, vocab, (rows,), generator=g)
    z.scatter_(1, t[:, None], lift + 2.0 * torch.randn(rows, 1, generator=g))
    z = z.to(dtype)
    ld = vocab + pad
    buf = torch.full((rows * ld + shift + 8,), float("nan"), dtype=dtype, device=DEV)
    v = buf[shift:shift + rows * ld].view(rows, ld)[:, :vocab]
    v.copy_(z)
    return v, t


def _drop(t, share, seed):
    g = torch.Generator().manual_seed(seed)
    t = t.clone()
    t[torch.rand(t.numel(), generator=g) < share] = IGNORE
    return t


def _close_logp(got, want):
    err = (ref.f64(got) - want).abs()
    bound = 5e-6 + 1e-6 * want.abs()
    say(f"  logp: largest error {float(err.max()) if err.numel() else 0:.2e}")
    assert (err <= bound).all()


def _close_grad(name, got, want, slope=False):
    tol = 5e-5 if slope else 1e-5
    if got.dtype == torch.bfloat16:
        tol += ref.BF16_TOL
    assert_close(name, ref.f64(got), want, tol, tol)


VOCABS = [1, 2, 7, 8, 9, 31, 255, 256, 257, 1000, 2047, 2048, 2049, 4099, 8192, 8200, 16384, 16385,
          32000, 32003, 32768, 40000, 65536, 65537, 100003, 131072, 140000, 262147]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["dense", "padded", "shifted"])
def test_token_logp_and_backward(vocab, dtype, layout):
    rows = 3 if vocab > 20000 else 19
    pad, shift = {"dense": (0, 0), "padded": (-vocab % 64 or 5, 0), "shifted": (3, 1)}[layout]
    scale = 1.0 if vocab % 2 else 0.8
    say(f"token logp: {rows}x{vocab} {dtype} {layout} scale={scale}")
    z, t = _logits(vocab, rows, vocab, dtype, pad, shift)
    t = _drop(t, 0.3, vocab)
    t[0] = vocab - 1
    logp, lse = q.qlora_token_logp(z, t.to(DEV), scale=scale)
    x = ref.f64(z).requires_grad_()
    want, want_lse = ref.token_logp(x, t, scale)
    _close_logp(logp, want.detach())
    _close_logp(lse, want_lse.detach())
    g = torch.randn(rows, generator=torch.Generator().manual_seed(3))
    g[-1] = 0.0
    (want * g.double()).sum().backward()
    d = q.qlora_token_logp_bwd(z, t.to(DEV), lse, g.to(DEV), scale=scale)
    assert d.shape == z.shape and d.stride(0) == z.stride(0)
    _close_grad("dlogits", d, x.grad)
    assert (d.cpu()[t == IGNORE] == 0).all()
    # into the logits' own buffer, and into one of another alignment and stride
    other = torch.zeros(rows * (vocab + 2) + 8, dtype=dtype, device=DEV)
    o = other[3:3 + rows * (vocab + 2)].view(rows, vocab + 2)[:, :vocab]
    q.qlora_token_logp_bwd(z, t.to(DEV), lse, g.to(DEV), scale=scale, dlogits=o)
    assert torch.equal(o, d)
    guard = other.clone()
    guard[3:3 + rows * (vocab + 2)].view(rows, vocab + 2)[:, :vocab] = 0
    assert (guard == 0).all(), "written outside the gradient's rows"
    if pad or shift:
        edge = torch.cat([z.as_strided((rows, pad), (vocab + pad, 1), shift + vocab).reshape(-1)])
        assert torch.isnan(edge).all()
    q.qlora_token_logp_bwd(z, t.to(DEV), lse, g.to(DEV), scale=scale, dlogits=z)
    assert torch.equal(z, d)
    if pad:
        assert torch.isnan(z.as_strided((rows, pad), (vocab + pad, 1), shift + vocab)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_banned_tokens_and_special_values(dtype):
    """Banned columns at -inf or at the type's lowest value, rows of one
    allowed token, rows the mask empties, NaN and infinities, bad targets."""
    vocab = 2051
    z, t = _logits(5, 12, vocab, dtype)
    low = torch.finfo(dtype).min
    z[:, 100:900] = -INF
    z[1, :] = -INF
    z[1, 1500] = 2.0                # one allowed token
    z[2, :] = low
    z[2, 77] = 1.0
    z[3, :] = -INF                  # nothing allowed
    z[4, 3] = float("nan")
    z[5, 3] = INF
    z[6, :] = float("nan")          # does not count
    z[7, :] = low                   # all equal: uniform
    z[8, 100:] = low
    t = t.clamp(max=99)
    t[1], t[2], t[6], t[9], t[10], t[11] = 1500, 77, IGNORE, vocab, -1, 200
    logp, lse = q.qlora_token_logp(z, t.to(DEV))
    lp = logp.cpu()
    assert lp[1] == 0.0 and lp[2] == 0.0
    assert torch.isnan(lp[[3, 4, 5]]).all() and torch.isnan(lp[[9, 10]]).all()
    assert lp[6] == 0.0 and lse[6].item() == 0.0
    assert abs(lp[7].item() + torch.log(torch.tensor(float(vocab))).item()) <= 1e-5
    assert lp[11] == -INF           # a banned target
    want, _ = ref.token_logp(ref.f64(z)[[0, 8]], t[[0, 8]])
    _close_logp(logp[[0, 8]], want)
    d = q.qlora_token_logp_bwd(z, t.to(DEV), lse, torch.ones(12, device=DEV)).cpu().double()
    assert (d[1] == 0).all() and (d[2] == 0).all() and (d[6] == 0).all()
    assert torch.isnan(d[[9, 10]]).all()
    assert (d[0, 100:900] == 0).all()
    ok = d[[0, 8, 11]]
    assert torch.isfinite(ok).all()
    assert (ok.sum(1).abs() <= (vocab ** 0.5) * 2.0 ** -8).all()
    assert abs(float(d[11, 200]) - 1.0) <= 1e-6


def test_long_rows_past_32_bits():
    """Rows 2^28 elements apart: the last ones start past 2^31 elements and
    2^32 bytes."""
    rows, vocab, ld = 10, 1001, 1 << 28
    buf = torch.empty(rows * ld, dtype=torch.bfloat16, device=DEV)
    z = buf.view(rows, ld)[:, :vocab]
    src, t = _logits(6, rows, vocab, torch.bfloat16)
    z.copy_(src)
    logp, lse = q.qlora_token_logp(z, t.to(DEV))
    want, want_lse = q.qlora_token_logp(src, t.to(DEV))
    # rows are aligned otherwise than the dense ones: sums in another order
    assert ref.max_err(logp, want) <= 5e-6 and ref.max_err(lse, want_lse) <= 5e-6
    dense = q.qlora_token_logp_bwd(src, t.to(DEV), lse, logp)
    q.qlora_token_logp_bwd(z, t.to(DEV), lse, logp, dlogits=z)
    assert torch.equal(z, dense)


def _answers(lens, prompt, t, hollow=()):
    """Targets with each sequence's prompt (and hollow sequences) left out."""
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    t = t.clone()
    for i, n in enumerate(lens):
        t[off[i]:off[i] + (n if i in hollow else int(n * prompt))] = IGNORE
    return off, t


PREF_CASES = [
    # lens of 2P sequences, vocab, dtype, kind, beta, smoothing, margin, mean, ref, hollow
    ([1, 1], 7, torch.float32, "sigmoid", 0.1, 0.0, 0.0, False, True, ()),
    ([5, 9], 1000, torch.bfloat16, "sigmoid", 0.1, 0.0, 0.0, False, True, ()),
    ([40, 3, 0, 17], 2049, torch.float32, "sigmoid", 0.5, 0.1, 0.25, False, True, ()),
    ([40, 3, 21, 17], 2049, torch.float32, "sigmoid", 2.0, 0.0, 0.5, True, False, (1,)),
    ([30, 30, 30, 31, 29, 33], 4099, torch.bfloat16, "hinge", 0.3, 0.0, 0.0, False, True, (0, 3)),
    ([30, 12, 30, 31], 515, torch.float32, "hinge", 0.05, 0.0, 0.1, True, False, ()),
    ([30, 12, 30, 31], 515, torch.float32, "squared", 0.2, 0.0, 0.0, True, True, ()),
    ([300, 1, 2, 270], 131, torch.float32, "squared", 0.1, 0.0, 0.0, False, True, ()),
    ([11, 7], 65537, torch.bfloat16, "sigmoid", 0.1, 0.2, 0.0, False, True, ()),
    ([11, 7], 70001, torch.float32, "sigmoid", 0.1, 0.0, 0.0, False, True, ()),
]


@pytest.mark.parametrize("case", range(len(PREF_CASES)))
def test_preference_loss(case):
    lens, vocab, dtype, kind, beta, smooth, margin, mean, with_ref, hollow = PREF_CASES[case]
    before, after = case % 3, case % 2 * 2            # rows outside every sequence
    rows = before + sum(lens) + after
    say(f"preference loss: {lens} x {vocab} {dtype} {kind}")
    z, t = _logits(case, rows, vocab, dtype, pad=case % 4)
    off, inner = _answers(lens, 0.3, t[before:before + sum(lens)], hollow)
    t[before:before + sum(lens)] = inner
    off = [o + before for o in off]
    x = ref.f64(z).requires_grad_()
    base = ref.token_logp(x.detach(), t)[0]
    r = (base + 0.1 * torch.randn(rows, generator=torch.Generator().manual_seed(case)).double())
    r = r.float() if with_ref else None
    P = len(lens) // 2
    weight = None if case % 2 else 0.75
    o = q.qlora_preference_loss(z, t.to(DEV), torch.tensor(off, device=DEV),
                                None if r is None else r.to(DEV), kind=KINDS[kind], beta=beta,
                                label_smoothing=smooth, margin=margin, length_normalize=mean,
                                weight=weight)
    args = (t, off, ref.f64(r), kind, beta, smooth, margin, mean)
    loss, seq, logp = ref.preference(x, *args)
    w = 1.0 / P if weight is None else weight
    (w * loss.sum()).backward()
    _close_logp(o.logp, logp.detach())
    n = max(lens)
    assert ref.max_err(o.seq_logp, seq.detach()) <= (n ** 0.5) * 5e-6 + 2e-7 * float(seq.abs().max())
    big = max(1.0, float(loss.detach().abs().max()))
    assert ref.max_err(o.loss, loss.detach()) <= 5e-5 * big
    _close_grad("dlogits", o.dlogits, x.grad, slope=True)
    out = torch.ones(rows, dtype=torch.bool)
    out[off[0]:off[-1]] = False
    assert (o.dlogits.cpu()[out | (t == IGNORE)] == 0).all()
    if dtype == torch.float32:
        f = lambda y: w * ref.preference(y, *args)[0].sum()  # noqa: E731
        g = ref.f64(o.dlogits)
        if float(g.abs().max()) > 0:
            v = g / g.norm()
            got = float((g * v).sum())
            # a step of 1e-3 along the gradient stays on one side of the hinge
            assert abs(got - ref.slope(f, x.detach(), v, 1e-3)) <= 1e-4 * abs(got) + 1e-9
    alone = q.qlora_preference_loss(z, t.to(DEV), torch.tensor(off, device=DEV),
                                    None if r is None else r.to(DEV), kind=KINDS[kind], beta=beta,
                                    label_smoothing=smooth, margin=margin, length_normalize=mean,
                                    need_grad=False)
    assert alone.dlogits is None and torch.equal(alone.loss, o.loss)
    q.qlora_preference_loss(z, t.to(DEV), torch.tensor(off, device=DEV),
                            None if r is None else r.to(DEV), kind=KINDS[kind], beta=beta,
                            label_smoothing=smooth, margin=margin, length_normalize=mean,
                            weight=weight, dlogits=z)
    assert torch.equal(z, o.dlogits)


def test_preference_of_far_apart_answers():
    """Margins of thousands of nats: the loss is linear on one side and 0 on
    the other, without overflow; a banned answer gives an infinite loss with a
    finite slope."""
    vocab, n = 64, 200
    z = torch.zeros(4 * n, vocab, device=DEV)
    t = torch.zeros(4 * n, dtype=torch.int64)
    z[:n, 0] = 80.0                  # answer 0 is certain, its partner (rows 2n..) impossible
    z[2 * n:3 * n, 0] = -80.0
    z[n:2 * n, 0] = -80.0            # answer 1 the other way round
    z[3 * n:, 0] = 80.0
    off = torch.tensor([0, n, 2 * n, 3 * n, 4 * n], device=DEV)
    o = q.qlora_preference_loss(z, t.to(DEV), off, beta=1.0)
    want = n * (80.0 + float(torch.log(torch.tensor(63.0))))
    assert o.loss[0].item() == 0.0 and abs(o.loss[1].item() - want) <= 1e-5 * want
    assert (o.dlogits[:n] == 0).all() and torch.isfinite(o.dlogits).all()
    assert abs(o.dlogits[n, 0].item() + 0.5) <= 1e-6
    z[n, 0] = -INF
    o = q.qlora_preference_loss(z, t.to(DEV), off, beta=1.0)
    assert o.loss[1].item() == INF and torch.isfinite(o.dlogits).all()
    t[0] = 64                        # no such token: NaN in its pair alone
    o = q.qlora_preference_loss(z, t.to(DEV), off, beta=1.0)
    assert torch.isnan(o.loss[0]) and o.loss[1].item() == INF


POLICY_CASES = [
    # lens, vocab, dtype, lo, hi, kl, per_token, seq_mean, old, ref, hollow
    ([1], 7, torch.float32, 0.2, 0.2, 0.1, False, True, True, True, ()),
    ([3, 24], 4099, torch.float32, 0.2, 0.2, 0.05, False, True, True, True, ()),
    ([17, 0, 40, 9], 2048, torch.bfloat16, 0.2, 0.28, 0.04, False, True, True, True, (3,)),
    ([17, 5, 40, 9], 2049, torch.float32, 0.1, 0.1, 0.0, True, False, True, False, (0,)),
    ([60, 33], 1000, torch.float32, 0.0, 0.0, 0.02, True, False, True, True, ()),
    ([12, 8], 32003, torch.bfloat16, 0.2, 0.2, 0.0, False, False, False, True, ()),
    ([12, 8], 65536, torch.bfloat16, 0.2, 0.2, 0.1, True, True, True, True, ()),
    ([12, 8], 65536, torch.float32, 0.2, 0.2, 0.1, True, False, True, True, ()),
    ([5, 4], 140000, torch.bfloat16, 1.0, 0.5, 0.1, False, False, True, True, ()),
    ([5, 4], 131072, torch.float32, 0.2, 0.5, 0.1, False, True, True, True, ()),
    ([400, 700, 3], 65, torch.float32, 0.2, 0.2, 0.1, True, False, True, True, ()),
]


@pytest.mark.parametrize("case", range(len(POLICY_CASES)))
def test_policy_loss(case):
    lens, vocab, dtype, lo, hi, kl, per_token, seq_mean, with_old, with_ref, hollow = \
        POLICY_CASES[case]
    before, after = case % 2 * 3, case % 3
    rows = before + sum(lens) + after
    say(f"policy loss: {lens} x {vocab} {dtype} kl={kl}")
    z, t = _logits(100 + case, rows, vocab, dtype, pad=case % 3, shift=case % 2)
    off, inner = _answers(lens, 0.2, t[before:before + sum(lens)], hollow)
    t[before:before + sum(lens)] = inner
    off = [o + before for o in off]
    g = torch.Generator().manual_seed(case)
    x = ref.f64(z).requires_grad_()
    base = ref.token_logp(x.detach(), t)[0]
    old = (base + 0.2 * torch.randn(rows, generator=g).double()).float() if with_old else None
    rf = (base + 0.3 * torch.randn(rows, generator=g).double()).float() if with_ref else None
    adv = torch.randn(rows if per_token else len(lens), generator=g)
    red = q.QLORA_POLICY_SEQUENCE_MEAN if seq_mean else q.QLORA_POLICY_TOKEN_MEAN
    weight = 1.0 if case % 2 else 0.5
    kw = dict(old_logp=None if old is None else old.to(DEV),
              ref_logp=None if rf is None else rf.to(DEV), clip_low=lo, clip_high=hi, kl_coef=kl,
              per_token=per_token, reduction=red)
    offd = torch.tensor(off, device=DEV)
    o = q.qlora_policy_loss(z, t.to(DEV), offd, adv.to(DEV), weight=weight, **kw)
    args = (t, off, adv.double(), ref.f64(old), ref.f64(rf), lo, hi, kl, per_token, seq_mean)
    stats, logp = ref.policy(x, *args)
    (weight * stats[0]).backward()
    _close_logp(o.logp, logp.detach())
    assert ref.max_err(o.stats, stats.detach()) <= 2e-5 * max(1.0, float(adv.abs().max()))
    _close_grad("dlogits", o.dlogits, x.grad, slope=True)
    if dtype == torch.float32 and with_old:
        f = lambda y: weight * ref.policy(y, *args)[0][0]  # noqa: E731
        d = ref.f64(o.dlogits)
        v = d / d.norm()
        got = float((d * v).sum())
        # rows within the step of a clip edge add at most step * slope^2 each
        assert abs(got - ref.slope(f, x.detach(), v, 1e-5)) <= 1e-3 * abs(got) + 1e-9
    alone = q.qlora_policy_loss(z, t.to(DEV), offd, adv.to(DEV), need_grad=False, **kw)
    assert alone.dlogits is None and torch.equal(alone.stats, o.stats)
    again = q.qlora_policy_loss(z, t.to(DEV), offd, adv.to(DEV), weight=weight, **kw)
    assert torch.equal(again.dlogits, o.dlogits) and torch.equal(again.stats, o.stats)
    q.qlora_policy_loss(z, t.to(DEV), offd, adv.to(DEV), weight=weight, dlogits=z, **kw)
    assert torch.equal(z, o.dlogits)


def test_policy_clip_edges_and_empty_batches():
    """Equal branches take the unclipped one's gradient; a batch whose mask
    leaves nothing gives zeros, not NaN."""
    z = torch.zeros(4, 16, device=DEV)
    t = torch.tensor([1, 2, IGNORE, 3], device=DEV)
    lp, _ = q.qlora_token_logp(z, t)
    off = torch.tensor([0, 4], device=DEV)
    adv = torch.tensor([2.0], device=DEV)
    o = q.qlora_policy_loss(z, t, off, adv, old_logp=lp, clip_low=0.0, clip_high=0.0)
    assert o.stats[3].item() == 0.0 and abs(o.stats[0].item() + 2.0) <= 1e-6
    assert abs(o.dlogits[0, 1].item() + 2.0 / 3 * 15 / 16) <= 1e-6
    on = q.qlora_policy_loss(z, t, off, adv)
    assert torch.equal(on.dlogits, o.dlogits)
    for red in (q.QLORA_POLICY_TOKEN_MEAN, q.QLORA_POLICY_SEQUENCE_MEAN):
        none = torch.full((4,), IGNORE, device=DEV)
        zz = torch.full((4, 16), float("nan"), device=DEV)
        o = q.qlora_policy_loss(zz, none, off, adv, old_logp=lp, ref_logp=lp, kl_coef=0.1,
                                reduction=red)
        assert (o.stats == 0).all() and (o.dlogits == 0).all() and (o.logp == 0).all()
        e = q.qlora_policy_loss(z[:0], t[:0], torch.zeros(1, dtype=torch.int64, device=DEV),
                                adv[:0], reduction=red)
        assert (e.stats == 0).all() and e.dlogits.shape == (0, 16)
        o = q.qlora_policy_loss(z, t, torch.zeros(1, dtype=torch.int64, device=DEV), adv[:0],
                                reduction=red)
        assert (o.stats == 0).all() and (o.dlogits == 0).all()
    e = q.qlora_preference_loss(z, t, torch.zeros(1, dtype=torch.int64, device=DEV))
    assert e.loss.numel() == 0 and (e.dlogits == 0).all()
    e = q.qlora_preference_loss(z[:0], t[:0], torch.zeros(3, dtype=torch.int64, device=DEV))
    assert abs(e.loss.item() - 0.6931472) <= 1e-6


def test_offsets_outside_the_batch_are_clamped():
    """Offsets are device data: values outside [0, rows] or out of order never
    take a kernel out of its arrays."""
    z, t = _logits(9, 20, 300, torch.float32)
    for off in ([-5, 8, 1 << 40], [3, 1, 50], [-7, -3, -1], [30, 40, 50]):
        offd = torch.tensor(off, device=DEV)
        good = [min(max(o, 0), 20) for o in off]
        good = [good[0], max(good[0], good[1]), max(good[1], good[2])]
        o = q.qlora_preference_loss(z, t.to(DEV), offd)
        p = q.qlora_policy_loss(z, t.to(DEV), offd, torch.ones(2, device=DEV))
        if off == [-5, 8, 1 << 40]:
            want = q.qlora_preference_loss(z, t.to(DEV), torch.tensor([0, 8, 20], device=DEV))
            assert torch.equal(o.dlogits, want.dlogits) and torch.equal(o.loss, want.loss)
        assert torch.isfinite(o.dlogits).all() and torch.isfinite(p.dlogits).all()


def test_losses_on_another_stream():
    z, t = _logits(12, 700, 4099, torch.bfloat16)
    t = _drop(t, 0.2, 1).to(DEV)
    off = torch.tensor([0, 300, 700], device=DEV)
    adv = torch.randn(2, device=DEV)
    a, b = q.qlora_preference_loss(z, t, off), q.qlora_policy_loss(z, t, off, adv)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        c, d = q.qlora_preference_loss(z, t, off), q.qlora_policy_loss(z, t, off, adv)
    st.synchronize()
    assert torch.equal(a.dlogits, c.dlogits) and torch.equal(b.dlogits, d.dlogits)
    assert torch.equal(a.loss, c.loss) and torch.equal(b.stats, d.stats)


@pytest.mark.parametrize("rows,vocab", [(12, 700), (12, 4099), (1100, 700), (300, 9000),
                                        (2100, 900), (12, 70001), (6, 100003)])
def test_bad_targets_outside_the_sequences_have_no_gradient(rows, vocab):
    """A row that no sequence holds gets a zero gradient, whatever its target;
    in a sequence a bad target gives NaN."""
    z, t = _logits(31, rows, vocab, torch.float32)
    t[[0, -1]] = torch.tensor([vocab, -7])
    t = t.to(DEV)
    off = torch.tensor([1, rows // 2, rows - 1], device=DEV)
    adv = torch.ones(2, device=DEV)
    for run in (lambda: q.qlora_preference_loss(z, t, off),
                lambda: q.qlora_policy_loss(z, t, off, adv),
                lambda: q.qlora_policy_loss(z, t, off, adv, reduction=q.QLORA_POLICY_SEQUENCE_MEAN)):
        o = run()
        assert (o.dlogits[[0, -1]] == 0).all()
        assert torch.isfinite(o.dlogits).all() and (o.dlogits[1:-1] != 0).any(1).all()
        assert torch.isnan(o.logp[[0, -1]]).all() and torch.isfinite(o.logp[1:-1]).all()
        assert torch.isfinite(o[0]).all()
    t[1] = vocab
    o = q.qlora_policy_loss(z, t, off, adv)
    assert torch.isnan(o.dlogits[1]).all() and (o.dlogits[0] == 0).all()
    assert torch.isfinite(o.stats[0])          # on-policy: the ratio is 1 whatever the row
    o = q.qlora_policy_loss(z, t, off, adv, old_logp=torch.zeros(rows, device=DEV))
    assert torch.isnan(o.dlogits[1]).all() and (o.dlogits[0] == 0).all()
    assert torch.isnan(o.stats[0])


@pytest.mark.parametrize("seqs", [255, 256, 257, 700, 1500])
def test_policy_loss_over_many_sequences(seqs):
    """Both reductions against the per-sequence counts, where the rows' own
    workgroups sum them and where they are summed once."""
    rows, vocab = 1400, 300
    z, t = _logits(41, rows, vocab, torch.float32)
    t = _drop(t, 0.3, 5)
    g = torch.Generator().manual_seed(6)
    off = torch.sort(torch.randint(0, rows + 1, (seqs + 1,), generator=g)).values
    adv = torch.randn(seqs, generator=g)
    lp = torch.log_softmax(ref.f64(z), -1)
    seq = torch.full((rows,), -1)
    for s in range(seqs):
        seq[off[s]:off[s + 1]] = s
    counts = (t != IGNORE) & (seq >= 0)
    n = torch.bincount(seq[counts], minlength=seqs)
    for red in (q.QLORA_POLICY_TOKEN_MEAN, q.QLORA_POLICY_SEQUENCE_MEAN):
        w = torch.zeros(rows, dtype=torch.float64)
        w[counts] = (1.0 / int(counts.sum()) if red == q.QLORA_POLICY_TOKEN_MEAN
                     else 1.0 / (seqs * n[seq[counts]].double()))
        c = torch.zeros(rows, dtype=torch.float64)
        c[counts] = -w[counts] * adv.double()[seq[counts]]
        hot = torch.zeros(rows, vocab, dtype=torch.float64)
        hot[counts, t[counts]] = 1.0
        want = c[:, None] * (hot - lp.exp())
        o = q.qlora_policy_loss(z, t.to(DEV), off.to(DEV), adv.to(DEV), reduction=red)
        _close_grad(f"dlogits {seqs}", o.dlogits, want)
        assert abs(o.stats[0].item() - float(c.sum())) <= 1e-6 * float(c.abs().sum())
