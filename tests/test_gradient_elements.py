"""Every element of the logits' gradients against float64, where
tests/test_gpu_losses.py and test_gpu_rows.py compare whole arrays: most
probabilities are far below the largest, so an element is judged by its own
size.

With c the gradient of a row's scaled log-probability, an element is c ((j ==
target) - p).  Its bound, all from the arithmetic:
- p = exp(E) with |E| up to 34 nats for these inputs (spread 2.5, targets up to
  14): E is rounded about five times, 2^-24 of at most 49 (in base 2) each, and
  the log of the sum (up to 256 terms a thread, then a tree) adds 1e-6: 5e-6
  altogether, and 2e-5 leaves a factor of four;
- c is off by dc, stated at each loss;
- the target's element c - c p is rounded at 2^-23 of c;
- BF16 adds one rounding to nearest, 2^-8 of the value."""
import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from parity_util import say
import train_ref as ref
from train_ref import IGNORE

DEV = torch.device("cuda:0")
P_REL = 2e-5


def largest_excess(got, z, t, c, dc, scale=1.0):
    """The largest error over its bound, over all elements: got [rows, vocab],
    z its float64 logits, c and dc float64 [rows]."""
    p = torch.exp(z * scale - torch.logsumexp(z * scale, 1, keepdim=True))
    hot = torch.zeros_like(p)
    counted = t != IGNORE
    hot[counted, t[counted]] = 1.0
    c, dc = (torch.where(counted, v, torch.zeros_like(v))[:, None] for v in (c, dc))
    want = c * (hot - p)
    bound = p * P_REL * c.abs() + dc * (hot - p).abs() + 2.0 ** -23 * c.abs() * (p + hot)
    if got.dtype == torch.bfloat16:
        bound = bound + ref.BF16_TOL * (want.abs() + bound)
    err = (ref.f64(got) - want).abs()
    assert (err[bound == 0] == 0).all()
    at = bound > 0
    return float((err[at] / bound[at]).max()) if at.any() else 0.0


def _inputs(seed, rows, vocab, dtype, pad=0, shift=0):
    """(values on the CPU, their rows on the GPU at stride vocab + pad from
    `shift` elements on, targets)."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 2.5
    t = torch.randint(0, vocab, (rows,), generator=g)
    z.scatter_(1, t[:, None], 6.0 + 2.0 * torch.randn(rows, 1, generator=g))
    z = z.to(dtype)
    t[torch.rand(rows, generator=g) < 0.2] = IGNORE
    return z, t, g


def _on_gpu(z, pad, shift):
    rows, vocab = z.shape
    buf = torch.full((rows * (vocab + pad) + shift,), float("nan"), dtype=z.dtype, device=DEV)
    v = buf[shift:].view(rows, vocab + pad)[:, :vocab]
    v.copy_(z)
    return v


def test_the_bound_sees_one_wrong_vector():
    """An oracle with eight small elements cleared, or with one vector's
    probabilities 1 % off, is refused; the right one, rounded, is not."""
    z, t, g = _inputs(1, 3, 32000, torch.float32)
    t[:] = torch.tensor([5, 31999, 12000])
    x, c = z.double(), torch.tensor([1.0, -0.3, 2e-4], dtype=torch.float64)
    dc = torch.zeros(3, dtype=torch.float64)
    p = torch.softmax(x, 1)
    hot = torch.zeros_like(p)
    hot[torch.arange(3), t] = 1.0
    right = c[:, None] * (hot - p)
    for dtype in (torch.float32, torch.bfloat16):
        assert largest_excess(right.to(dtype), x, t, c, dc) <= 1.0
        wrong = right.clone()
        wrong[1, 16384:16392] = 0.0
        assert largest_excess(wrong.to(dtype), x, t, c, dc) > 1.0
        wrong = right.clone()
        wrong[2, 8:16] *= 1.01
        assert largest_excess(wrong.to(dtype), x, t, c, dc) > 1.0


LAYOUTS = [(0, 0), (1, 0), (5, 1), (2, 1)]     # padding of a row, first element
WIDTHS = [1, 7, 8, 9, 65, 511, 512, 513, 2047, 2048, 2049, 4095, 4096, 4097, 8191, 8192, 8193, 16383,
          16384, 16385, 24576, 24577, 32000, 32003, 32768, 32769, 49152, 49153, 65536, 65537, 73729,
          98304, 98305, 131071, 131072, 131073]


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_token_logp_backward(vocab, dtype):
    rows = 3 if vocab > 20000 else 9
    scale = 1.25 if vocab % 2 else 1.0
    for pad, shift in LAYOUTS:
        say(f"token logp backward: {rows}x{vocab} {dtype} pad {pad} from {shift}")
        z, t, g = _inputs(vocab, rows, vocab, dtype)
        t[-1] = vocab - 1
        d = torch.randn(rows, generator=g)
        v = _on_gpu(z, pad, shift)
        _, lse = q.qlora_token_logp(v, t.to(DEV), scale=scale)
        got = q.qlora_token_logp_bwd(v, t.to(DEV), lse, d.to(DEV), scale=scale)
        c = d.double() * scale
        assert largest_excess(got, z.double(), t, c, 0.0 * c, scale) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("vocab", WIDTHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_loss(vocab, dtype):
    """dc: a log-probability is off by 5e-6 + 1e-6 of itself, which scales the
    ratio and the KL slope; their products are rounded a few times."""
    lens = [4, 0, 5]
    rows, kl, lo, hi = sum(lens), 0.1, 0.2, 0.28
    for turn, (pad, shift) in enumerate(LAYOUTS):
        say(f"policy loss: {rows}x{vocab} {dtype} pad {pad} from {shift}")
        z, t, g = _inputs(vocab + turn, rows, vocab, dtype)
        t[0] = vocab - 1
        lp = ref.token_logp(z.double(), t)[0]
        # ratios off the clip's edges, where the branch is a matter of rounding
        gap = 0.2 * torch.randn(rows, generator=g).double()
        for edge in (1 - lo, 1 + hi):
            gap = torch.where((torch.exp(gap) - edge).abs() < 1e-2, gap + 0.05, gap)
        old = (lp - gap).float()
        rf = (lp + 0.3 * torch.randn(rows, generator=g).double()).float()
        adv = torch.randn(len(lens), generator=g)
        o = q.qlora_policy_loss(_on_gpu(z, pad, shift), t.to(DEV), torch.tensor([0, 4, 4, 9], device=DEV),
                                adv.to(DEV), old_logp=old.to(DEV), ref_logp=rf.to(DEV), kl_coef=kl,
                                clip_low=lo, clip_high=hi)
        a = adv.double()[torch.tensor([0] * 4 + [2] * 5)]
        ratio, up = torch.exp(lp - old.double()), torch.exp(rf.double() - lp)
        held = ((a > 0) & (ratio > 1 + hi)) | ((a < 0) & (ratio < 1 - lo))
        free = torch.where(held, torch.zeros_like(a), -a * ratio)
        w = 1.0 / max(1, int((t != IGNORE).sum()))
        dl = 5e-6 + 1e-6 * lp.abs()
        dc = w * ((dl + 4e-7) * free.abs() + kl * ((dl + 4e-7) * up + 4e-7))
        assert largest_excess(o.dlogits, z.double(), t, w * (free + kl * (1 - up)), dc) <= 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("pairs,vocab", [(1, 7), (1, 1000), (1, 2049), (3, 4099), (2, 32003), (2, 65537),
                                         (30, 16385), (30, 32000), (9, 131072), (400, 200), (70, 8200)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_preference_loss(pairs, vocab, dtype):
    """Pairs taken in one launch, in two and in three.  dc: a pair has up to 10
    log-probabilities of size up to 20, off by 2.5e-5 each at most, so its
    margin by 0.1 x 2.5e-4 and the loss's slope by as much of itself; 5e-5
    with the slope's own rounding."""
    g = torch.Generator().manual_seed(pairs)
    lens = torch.randint(1, 6, (2 * pairs,), generator=g).tolist()
    rows, off = sum(lens), [0]
    for n in lens:
        off.append(off[-1] + n)
    pad, shift = LAYOUTS[pairs % 4]
    say(f"preference loss: {pairs} pairs, {rows}x{vocab} {dtype} pad {pad} from {shift}")
    z, t, _ = _inputs(vocab, rows, vocab, dtype)
    x = z.double()
    lp = ref.token_logp(x, t)[0]
    rf = (lp + 0.2 * torch.randn(rows, generator=g).double()).float()
    o = q.qlora_preference_loss(_on_gpu(z, pad, shift), t.to(DEV), torch.tensor(off, device=DEV),
                                rf.to(DEV), beta=0.1)
    gain = torch.where(t != IGNORE, lp - rf.double(), torch.zeros_like(lp))
    s = torch.stack([gain[a:b].sum() for a, b in zip(off, off[1:])])
    slope = -0.1 * torch.sigmoid(-0.1 * (s[:pairs] - s[pairs:])) / pairs
    c = torch.cat([slope, -slope])[torch.repeat_interleave(torch.arange(2 * pairs), torch.tensor(lens))]
    assert largest_excess(o.dlogits, x, t, c, 5e-5 * c.abs()) <= 1.0
