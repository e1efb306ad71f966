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
