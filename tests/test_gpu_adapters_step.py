"""The operators of a step that trains several adapters on one frozen base, run
together: the base's product, the adapters beside it, inputs kept in 8 bits, the
backward, the optimizer on the bank; and the example's layers with their inputs
in 8 bits."""
import os
import sys

import pytest
import torch

import adapters_ref as ref
import bit_quantized_lora_quantize_amd as q

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import tuning_step  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


class Layer:
    """A frozen NF4 projection with a bank of adapters and their AdamW state."""

    def __init__(self, d_in, d_out, r, slots, gen):
        rand = lambda *s: torch.randn(*s, generator=gen).to(DEV)  # noqa: E731
        self.w = q.qlora_quantize_nf4(rand(d_out, d_in) / d_in ** 0.5)
        self.params = []
        for p in (rand(slots, r, d_in) / d_in ** 0.5, 0.1 * rand(slots, d_out, r)):
            self.params.append(q.AdamwParam(p, torch.zeros_like(p), torch.zeros_like(p), torch.zeros_like(p), p.bfloat16()))
        self.scale = 0.5 + torch.rand(slots, generator=gen).to(DEV)
        self.bank = q.AdapterBank(self.params[0].param_bf16, self.params[1].param_bf16, self.scale)

    def forward(self, x, plan):
        y0 = q.qlora_linear_fwd(self.w, x, self.bank.A[0], self.bank.B[0], 0.0)   # the base alone
        self.y0 = y0.clone()
        out = q.qlora_adapters_fwd(x, self.bank, plan, Y0=y0, Y=y0)
        self.x8, self.T = q.qlora_pack8(x), out.T
        return out.Y

    def backward(self, dy, plan):
        x = q.qlora_unpack8(self.x8)
        dx0 = q.qlora_linear_bwd(self.w, x, dy, self.bank.A[0], self.bank.B[0], 0.0, T_saved=self.T)[0]
        self.dx0 = dx0.clone()
        a, b = self.params
        return q.qlora_adapters_bwd(dy, self.x8, self.T, self.bank, plan, dX0=dx0, dX=dx0, dA=a.grad, dB=b.grad)


def test_a_step_of_several_adapters():
    gen = torch.Generator().manual_seed(1)
    M, slots = 300, 4
    layers = [Layer(128, 192, 16, slots, gen), Layer(192, 64, 16, slots, gen)]
    index = torch.repeat_interleave(torch.tensor([2, -1, 0, 2]), torch.tensor([90, 40, 100, 70])).int()   # slot 1, 3 unused
    plan = q.qlora_adapters_plan(index.to(DEV), slots)   # one for both layers and both directions
    x = torch.randn(M, 128, generator=gen).bfloat16().to(DEV)
    dy = torch.randn(M, 64, generator=gen).bfloat16().to(DEV)
    acts = [x]
    for layer in layers:
        acts.append(layer.forward(acts[-1], plan))
        Y, T, eY, eT = ref.fwd(acts[-2], index, layer.bank.A, layer.bank.B, layer.scale, layer.y0)
        ref.inside(layer.T, T, eT, "T")
        ref.inside(acts[-1], Y, eY, "Y")
    for layer in reversed(layers):
        g = layer.backward(dy, plan)
        want, bound = ref.bwd(q.qlora_unpack8(layer.x8), index, layer.T, layer.bank.A, layer.bank.B, layer.scale, dy, layer.dx0)
        for k in ("dA", "dB", "dX"):
            ref.inside(getattr(g, k), want[k], bound[k], k)
        dy = g.dX
    before = [p.param.clone() for layer in layers for p in layer.params]
    params = q.AdamwParamSet([p for layer in layers for p in layer.params])
    sumsq = torch.zeros(1, dtype=torch.float64, device=DEV)
    q.qlora_grad_sumsq(params, sumsq)
    q.qlora_adamw_step(params, lr=1e-2, step=1, grad_sumsq=sumsq, max_grad_norm=1.0)
    for p, old in zip(params.params, before):
        moved = (p.param != old).flatten(1).any(1).cpu()
        assert moved.tolist() == [True, False, True, False]   # only the adapters that tokens used
    again = layers[0].forward(x, plan)
    Y, _, eY, _ = ref.fwd(x, index, layers[0].bank.A, layers[0].bank.B, layers[0].scale, layers[0].y0)
    ref.inside(again, Y, eY, "Y after the step")
    assert not torch.equal(again, acts[1]) and torch.equal(again[90:130], acts[1][90:130])


def test_the_same_adapter_for_all_is_the_single_layer():
    """A bank of one adapter beside the base: within the two roundings that the
    fused layer saves."""
    gen = torch.Generator().manual_seed(2)
    M, r = 100, 16
    layer = Layer(128, 96, r, 1, gen)
    alpha = 2.0 * r
    layer.scale.fill_(2.0)
    x = torch.randn(M, 128, generator=gen).bfloat16().to(DEV)
    plan = q.qlora_adapters_plan(torch.zeros(M, dtype=torch.int32, device=DEV), 1)
    T = torch.empty(M, r, device=DEV)
    one = q.qlora_linear_fwd(layer.w, x, layer.bank.A[0], layer.bank.B[0], alpha, T_save=T)
    y = layer.forward(x, plan)
    _, _, eY, eT = ref.fwd(x, torch.zeros(M), layer.bank.A, layer.bank.B, layer.scale, layer.y0)
    ref.inside(layer.T, ref.f64(T), 2 * eT, "T")
    room = 2 * eY + ref.U8 * (ref.f64(layer.y0).abs() + ref.f64(one).abs()) * ref.SLACK
    ref.inside(y, ref.f64(one), room, "Y")


@pytest.mark.parametrize("loss", ["preference", "policy"])
def test_example_with_inputs_in_8_bits(loss):
    """It runs, and its layers' gradients are their definition's from the restored
    inputs."""
    seen = []
    original = q.qlora_linear_bwd_packed

    def spy(w, x8, dy, a, b, alpha, T_saved=None, **kw):
        out = original(w, x8, dy, a, b, alpha, T_saved, **kw)
        if len(seen) < 3:
            seen.append((q.qlora_unpack8(x8), dy.clone(), a.clone(), b.clone(), alpha, T_saved.clone(), out[1].clone(), out[2].clone()))
        return out

    q.qlora_linear_bwd_packed = spy
    try:
        losses = tuning_step.run(loss, steps=2, pairs=2, longest=12, d=128, ff=192, vocab=200, show=lambda *_: None, kept="8bit")
    finally:
        q.qlora_linear_bwd_packed = original
    assert len(losses) == 2 and all(x == x for x in losses) and len(seen) == 3
    for x, dy, a, b, alpha, T, dA, dB in seen:
        M, r = dy.shape[0], a.shape[0]
        index = torch.zeros(M, dtype=torch.int32)
        want, bound = ref.bwd(x, index, T, a[None], b[None], torch.full((1,), alpha / r), dy, None)
        ref.inside(dA[None], want["dA"], bound["dA"], "dA")
        ref.inside(dB[None], want["dB"], bound["dB"], "dB")
