"""The example that runs the norms, the losses, the linear layers and the
optimizer together: a preference step lowers its loss from log 2, a policy
step's first gradient is that of the plain policy gradient, and the gradients
of a whole step agree with differences of the loss."""
import importlib.util
import math
import os

import pytest
import torch

import bit_quantized_lora_quantize_amd as q

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "tuning_step.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tuning_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_preference_steps_lower_the_loss(example):
    losses = example.run("preference", steps=8, show=lambda s: print(s, flush=True))
    # B starts at 0: policy and reference agree, every pair's loss is log 2
    assert abs(losses[0] - math.log(2.0)) <= 1e-6
    assert losses[-1] < 0.5 * losses[0]
    assert all(b < a for a, b in zip(losses, losses[1:]))


def test_policy_steps_lower_the_loss(example):
    losses = example.run("policy", steps=8, show=lambda s: print(s, flush=True))
    # on-policy (even) steps have ratio 1: minus the mean advantage, plus the KL term
    assert losses[1] < losses[0] and losses[3] < losses[2]
    assert all(math.isfinite(v) for v in losses)


def test_step_gradient_against_differences(example):
    """The loss's slope along a direction in A and B of every layer and in the
    norms' weights, against a central difference of the whole forward.  The
    forward rounds activations to BF16 (2^-8 of each value), which is noise in
    the difference: a large step along the gradient itself and a bound of 5 %."""
    dev = torch.device("cuda", 0)
    model = example.Model(256, 512, 1000, 3, dev)
    tokens, targets, offsets = example.answers(2, 24, 1000, 3, dev)
    ref, _ = q.qlora_token_logp(model.logits(tokens, alpha=0.0, save=False), targets)
    out = q.qlora_preference_loss(model.logits(tokens), targets, offsets, ref_logp=ref, beta=1.0)
    model.backward(out.dlogits)
    grads = [p.grad.clone() for p in model.params.params]
    norm2 = sum(float((g.double() ** 2).sum()) for g in grads)
    step = 0.05 / norm2 ** 0.5
    found = []
    for sign in (1.0, -1.0):
        for p, g in zip(model.params.params, grads):
            p.param.add_(g, alpha=sign * step)
            if p.param_bf16 is not None:
                p.param_bf16.copy_(p.param)
        o = q.qlora_preference_loss(model.logits(tokens, save=False), targets, offsets,
                                    ref_logp=ref, beta=1.0, need_grad=False)
        found.append(float(o.loss.double().mean()))
        for p, g in zip(model.params.params, grads):
            p.param.add_(g, alpha=-sign * step)
    slope = (found[0] - found[1]) / (2 * step)
    assert abs(slope - norm2) <= 0.05 * norm2, (slope, norm2)


def test_caller_workspaces():
    """A caller's workspace of any type gives the results of one's own; one on
    the host, strided or too small is refused."""
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(3)
    x = torch.randn(70, 600, generator=g).to(dev)
    t = torch.randint(0, 600, (70,), generator=g).to(dev)
    off, adv = torch.tensor([0, 40, 70], device=dev), torch.ones(2, device=dev)
    gamma = torch.ones(600, device=dev)
    n = q.qlora_norm_fwd(x, gamma)
    calls = [
        (q.qlora_norm_workspace_bytes(70, 600),
         lambda w: q.qlora_norm_bwd(x, n.H, gamma, n.mean, n.rstd, need_dbeta=True, workspace=w)),
        (q.qlora_preference_workspace_bytes(70),
         lambda w: q.qlora_preference_loss(x, t, off, workspace=w)),
        (q.qlora_policy_workspace_bytes(70, 2),
         lambda w: q.qlora_policy_loss(x, t, off, adv, workspace=w))]
    for need, call in calls:
        want = call(None)
        for ws in (torch.empty(need, dtype=torch.uint8, device=dev),
                   torch.empty((need + 3) // 4, dtype=torch.float32, device=dev)):
            got = call(ws)
            assert all(a is None and b is None or torch.equal(a, b) for a, b in zip(got, want))
        for ws in (torch.empty(need, dtype=torch.uint8),
                   torch.empty(2 * need, dtype=torch.uint8, device=dev)[::2]):
            with pytest.raises(ValueError):
                call(ws)
        with pytest.raises(q.QloraError):
            call(torch.empty(need - 1, dtype=torch.uint8, device=dev))
