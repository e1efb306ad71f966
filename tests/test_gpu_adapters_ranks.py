"""Ranks whose rows of B are no whole vectors, at widths that leave few rows behind
the last whole step or range of the long axis: forward, backward and the NF4
layer's backward, against their definition in 64 bits."""
import pytest
import torch

import adapters_ref as ref
import bit_quantized_lora_quantize_amd as q
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")

WIDTHS = [65, 66, 67, 70, 71, 72, 129, 257, 258, 262, 513, 519]


@pytest.mark.parametrize("r", [1, 2, 3, 4, 5, 7, 9, 65])
@pytest.mark.parametrize("d_out", WIDTHS)
def test_adapters(r, d_out):
    say(f"adapters rank {r} -> {d_out}")
    M, d_in, slots = 70, 72, 2
    b = ref.batch(1000 * r + d_out, M, d_in, d_out, r, slots, 30, none=0.1)
    d = {k: v.to(DEV) for k, v in b.items()}
    bank = q.AdapterBank(d["A"], d["B"], d["scale"])
    plan = q.qlora_adapters_plan(d["index"], slots)
    out = q.qlora_adapters_fwd(d["X"], bank, plan, Y0=d["Y0"])
    Y, T, eY, eT = ref.fwd(b["X"], b["index"], b["A"], b["B"], b["scale"], b["Y0"])
    ref.inside(out.T, T, eT, "T")
    ref.inside(out.Y, Y, eY, "Y")
    g = q.qlora_adapters_bwd(d["dY"], d["X"], out.T, bank, plan, dX0=d["dX0"])
    want, bound = ref.bwd(b["X"], b["index"], out.T, b["A"], b["B"], b["scale"], b["dY"], b["dX0"])
    for k in ("dA", "dB", "dX"):
        ref.inside(getattr(g, k), want[k], bound[k], k)


@pytest.mark.parametrize("r", [1, 2, 3, 5])
@pytest.mark.parametrize("d_out", [65, 66, 70, 257, 258])
def test_layer_from_a_checkpoint(r, d_out):
    """The layer's dA and dB are those of a bank of one adapter of scale alpha / r."""
    say(f"packed layer rank {r} -> {d_out}")
    M, d_in = 40, 64
    b = ref.batch(r + d_out, M, d_in, d_out, r, 1, 1, none=0.0)
    d = {k: v.to(DEV) for k, v in b.items()}
    w = q.qlora_quantize_nf4(torch.randn(d_out, d_in, generator=torch.Generator().manual_seed(r)).to(DEV) * 0.02)
    X8 = q.qlora_pack8(d["X"])
    T = 2.0 * (d["X"].float() @ d["A"][0].float().t())
    _, dA, dB = q.qlora_linear_bwd_packed(w, X8, d["dY"], d["A"][0], d["B"][0], 2.0 * r, T)
    index = torch.zeros(M, dtype=torch.int32)
    want, bound = ref.bwd(q.qlora_unpack8(X8), index, T, b["A"], b["B"], torch.full((1,), 2.0), b["dY"], None)
    ref.inside(dA[None], want["dA"], bound["dA"], "dA")
    ref.inside(dB[None], want["dB"], bound["dB"], "dB")
