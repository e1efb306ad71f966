"""What include/qlora.h and the binding promise about the norms and losses at
the edges of their ranges: large offsets and scales, memory that outputs and
gradients take, alignment, bad targets."""
import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from parity_util import say
import train_ref as ref
from train_ref import IGNORE

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _draw(seed, shape, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * std + mean


def test_backward_takes_the_lse_as_it_is():
    """p = exp(scale l - lse) for the FP32 lse given, with a scale that does not
    divide it.  With |scale l - lse| up to 8 nats, 12 in base 2: the scale's
    rounding 12 x 2^-23.4, the sum's 2^-21, the exponential and the product
    2^-22.5, times ln 2: 1.3e-6.  The lse, about 106, is spaced 7.6e-6, so an
    lse rounded once more would show as up to 3.8e-6."""
    rows, vocab, scale = 64, 512, 1.25
    z = _draw(1, (rows, vocab), 0.3, 80.0)
    t = torch.full((rows,), 3)
    _, lse = q.qlora_token_logp(z.to(DEV), t.to(DEV), scale=scale)
    d = q.qlora_token_logp_bwd(z.to(DEV), t.to(DEV), lse, torch.full((rows,), 1 / scale, device=DEV),
                               scale=scale)
    gap = z.double() * scale - ref.f64(lse)[:, None]
    assert float(gap.abs().max()) <= 8.0
    rel = (-ref.f64(d) / torch.exp(gap) - 1.0)
    rel[:, 3] = 0.0
    say(f"  largest relative error {float(rel.abs().max()):.2e}")
    assert float(rel.abs().max()) <= 1.6e-6


@pytest.mark.parametrize("vocab", [100, 4099, 32000, 131072])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [200.0, -1000.0, 30000.0, 1e30])
def test_backward_of_rows_far_from_zero(vocab, dtype, offset):
    """A common offset of a row's logits does not change its probabilities,
    though the FP32 lse holds none of the logits' differences at 1e30.  Inputs
    are rounded first; |scale (l - max)| is at most 16 nats at the offsets that
    leave differences, so 2e-5 as for other rows; in BF16 one rounding more."""
    rows = 5
    say(f"far from zero: {rows}x{vocab} {dtype} offset {offset}")
    z = (_draw(vocab, (rows, vocab)) + offset).to(dtype)
    t = torch.arange(rows) * (vocab // rows)
    t[4] = IGNORE
    dl = _draw(2, (rows,))
    buf = torch.empty(rows, vocab + 3, dtype=dtype, device=DEV)
    v = buf[:, :vocab]
    v.copy_(z)
    _, lse = q.qlora_token_logp(v, t.to(DEV))
    got = q.qlora_token_logp_bwd(v, t.to(DEV), lse, dl.to(DEV))
    p = torch.softmax(z.double(), 1)
    hot = torch.zeros_like(p)
    hot[torch.arange(4), t[:4]] = 1.0
    c = dl.double()[:, None] * (t != IGNORE)[:, None]
    want = c * (hot - p)
    # differences of 2^-8 of the offset, up to 128 nats at 30000 in BF16: the
    # exponent's rounding grows with them, the element shrinks below 1e-30
    bound = 2e-5 * c.abs() * p + 2.0 ** -23 * c.abs() * hot + 1e-30
    if dtype == torch.bfloat16:
        bound = bound + ref.BF16_TOL * (want.abs() + bound)
    assert ((ref.f64(got) - want).abs() <= bound).all()
    q.qlora_token_logp_bwd(v, t.to(DEV), lse, dl.to(DEV), dlogits=v)
    assert torch.equal(v, got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_backward_of_rows_at_the_lowest_value(dtype):
    """A row that a mask of the type's lowest value empties is uniform, also in
    the backward; beside one such row the others keep their values."""
    rows, vocab = 4, 2051
    z = _draw(3, (rows, vocab)).to(dtype)
    z[2] = torch.finfo(dtype).min
    t = torch.tensor([4, 5, 6, 7])
    _, lse = q.qlora_token_logp(z.to(DEV), t.to(DEV))
    got = ref.f64(q.qlora_token_logp_bwd(z.to(DEV), t.to(DEV), lse, torch.ones(rows, device=DEV)))
    # (not from a log of the sum: that holds nothing beside -3e38 in 64 bits either)
    want = -torch.softmax(z.double(), 1)
    want[torch.arange(rows), t] += 1.0
    tol = 2e-5 + (ref.BF16_TOL if dtype == torch.bfloat16 else 0.0)
    assert ((got - want).abs() <= tol * want.abs() + 2e-7).all()


def test_backward_at_scales_that_overflow_the_quotient():
    """lse / scale past the FP32 range, at scales of 1e-38: p is still uniform."""
    rows, vocab, scale = 3, 1000, 1e-38
    z = _draw(4, (rows, vocab))
    t = torch.tensor([0, 500, 999])
    _, lse = q.qlora_token_logp(z.to(DEV), t.to(DEV), scale=scale)
    got = ref.f64(q.qlora_token_logp_bwd(z.to(DEV), t.to(DEV), lse,
                                         torch.full((rows,), 1e38, device=DEV), scale=scale))
    hot = torch.zeros(rows, vocab, dtype=torch.float64)
    hot[torch.arange(rows), t] = 1.0
    assert ((got - (hot - 1.0 / vocab)).abs() <= 2e-5 / vocab + 1e-6 * hot).all()


def _batch(rows=2000, vocab=70):
    z, t = _draw(5, (rows, vocab)).to(DEV), torch.randint(0, vocab, (rows,), device=DEV)
    return z, t, torch.tensor([0, rows // 2, rows], device=DEV), torch.ones(2, device=DEV)


def test_losses_keep_nothing_alive_beside_an_output():
    """Each output holds its own values and no more, and takes an in-place
    operation with a tensor that needs a gradient."""
    z, t, off, adv = _batch()
    outs = [*q.qlora_preference_loss(z, t, off)[:3], *q.qlora_policy_loss(z, t, off, adv)[:2]]
    for o in outs:
        held = o.untyped_storage().nbytes()
        assert held == o.numel() * 4
        o.mul_(torch.ones((), device=DEV, requires_grad=True))
        assert o.requires_grad


def test_gradient_buffers_take_no_large_stride():
    """Logits that are a slice of a larger array: their gradient is dense, the
    padding of a row's end apart."""
    x = _draw(6, (9, 50, 700)).to(DEV)
    z = x[:, 7, :]                                   # stride 35000
    t = torch.arange(9, device=DEV)
    off, adv = torch.tensor([0, 5, 9], device=DEV), torch.ones(2, device=DEV)
    lp, lse = q.qlora_token_logp(z, t)
    calls = [lambda v: q.qlora_token_logp_bwd(v, t, lse, lp),
             lambda v: q.qlora_preference_loss(v, t, off).dlogits,
             lambda v: q.qlora_policy_loss(v, t, off, adv).dlogits]
    for call in calls:
        d = call(z)
        held = d.untyped_storage().nbytes()
        assert d.stride() == (700, 1) and held == 9 * 700 * 4
        dense = z.clone()
        assert ref.max_err(d, call(dense)) <= 5e-6
        padded = torch.empty(9, 704, device=DEV)[:, :700]
        padded.copy_(z)
        assert call(padded).stride() == (704, 1)


@pytest.mark.parametrize("vocab", [300, 2048, 2100])
@pytest.mark.parametrize("lens", [[32] + [0] * 15, [16, 16], [3, 4, 1, 8, 0, 9, 4, 3], [33, 0],
                                  [5, 6, 7, 9, 0, 6]])
def test_preference_of_few_rows(lens, vocab):
    """Batches on both sides of the rule that takes them in one launch, and the
    same pairs beside 64 rows that no sequence holds, which never do: one loss,
    one gradient (log-probabilities summed in another order: 5e-6 each)."""
    rows, P = sum(lens), len(lens) // 2
    say(f"few rows: {P} pairs of {rows} x {vocab}")
    z = _draw(11, (rows + 64, vocab), 2.0).to(DEV)
    t = torch.randint(0, vocab, (rows + 64,), generator=torch.Generator().manual_seed(1)).to(DEV)
    t[::7] = IGNORE
    off = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), device=DEV)
    a = q.qlora_preference_loss(z[:rows], t[:rows], off, beta=0.1)
    b = q.qlora_preference_loss(z, t, off, beta=0.1)
    assert ref.max_err(a.logp, b.logp[:rows]) <= 5e-6
    assert ref.max_err(a.loss, b.loss) <= 0.1 * rows * 5e-6
    assert ref.max_err(a.dlogits, b.dlogits[:rows]) <= 5e-5 * float(b.dlogits.abs().max())
    assert (b.dlogits[rows:] == 0).all()


def test_preference_with_all_rows_in_one_pair_is_not_slow():
    """The lengths of the pairs are not known to the host: a batch whose rows all
    lie in one pair takes no more than four times as long as an even one (it
    took seventeen times, by one workgroup)."""
    rows, vocab, P = 1000, 1000, 32
    z = _draw(12, (rows, vocab)).to(torch.bfloat16).to(DEV)
    t = torch.randint(0, vocab, (rows,), device=DEV)
    even = torch.arange(2 * P + 1, device=DEV) * rows // (2 * P)
    skew = torch.tensor([0, 500] + [500] * (P - 1) + [1000] * P, device=DEV)

    def us(off):
        times = []
        for _ in range(25):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                q.qlora_preference_loss(z, t, off)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 250)
        return sorted(times)[12]

    e, s = us(even), us(skew)
    say(f"  even {e:.1f} us, in one pair {s:.1f} us")
    assert s <= 4 * e


@pytest.mark.parametrize("width", [1, 7, 72, 515, 1001, 4096, 8200, 11009, 18432, 32769, 40001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", [q.QLORA_NORM_LAYER, q.QLORA_NORM_RMS])
def test_norms_give_the_same_bits_at_any_alignment(width, dtype, kind):
    rows, layer = 11, kind == q.QLORA_NORM_LAYER

    def at(seed, by, shape=(rows, width)):
        src = _draw(seed, shape).to(dtype)
        v = torch.empty(src.numel() + by, dtype=dtype, device=DEV)[by:].view(shape)
        v.copy_(src)
        return v

    found = []
    for by in (0, 1, 3):
        X, R, dY, dH = (at(k, by) for k in (1, 2, 3, 4))
        gamma, beta = at(5, by, (width,)), at(6, by, (width,)) if layer else None
        o = q.qlora_norm_fwd(X, gamma, beta, kind=kind, residual=R, Y=at(7, by), H=at(8, by))
        b = q.qlora_norm_bwd(dY, o.H, gamma, o.mean, o.rstd, kind=kind, dH=dH, need_dbeta=layer,
                             dX=at(9, by))
        found.append([o.Y, o.H, o.rstd, b.dX, b.dgamma] + ([o.mean, b.dbeta] if layer else []))
    for other in found[1:]:
        assert all(torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0)) for a, b in zip(found[0], other))


def test_bad_targets_by_entry_point():
    """A target outside the vocabulary: NaN log-probabilities everywhere; in the
    gradient NaN in its row alone, but zeros where dlogp is 0 or no sequence
    holds the row, and NaN in every row of its pair that counts."""
    z, t, off, adv = _batch(40, 70)
    t[3], t[25], t[6] = 70, -1, IGNORE
    off = torch.tensor([0, 10, 20, 30, 36], device=DEV)         # rows 36 .. 39 in none
    t[38] = 99
    lp, lse = q.qlora_token_logp(z, t)
    bad = torch.tensor([3, 25, 38], device=DEV)
    assert torch.isnan(lp[bad]).all() and torch.isnan(lse[bad]).all()
    up = torch.ones(40, device=DEV)
    up[25] = 0.0
    d = q.qlora_token_logp_bwd(z, t, lse, up)
    assert torch.isnan(d[[3, 38]]).all() and (d[25] == 0).all() and (d[6] == 0).all()
    assert torch.isfinite(d[[0, 24, 39]]).all()
    o = q.qlora_preference_loss(z, t, off)                      # pairs (0, 2) and (1, 3)
    assert torch.isnan(o.loss[0]) and torch.isfinite(o.loss[1])
    held = torch.arange(40, device=DEV)
    pair = ((held < 10) | (held >= 20) & (held < 30)) & (t != IGNORE)
    assert torch.isnan(o.dlogits[pair]).all() and torch.isfinite(o.dlogits[~pair]).all()
    assert (o.dlogits[36:] == 0).all()
    p = q.qlora_policy_loss(z, t, off, torch.ones(4, device=DEV), old_logp=torch.zeros(40, device=DEV))
    assert torch.isnan(p.dlogits[[3, 25]]).all() and (p.dlogits[36:] == 0).all()
    rest = torch.ones(40, dtype=torch.bool, device=DEV)
    rest[[3, 25]] = False
    assert torch.isfinite(p.dlogits[rest]).all()
