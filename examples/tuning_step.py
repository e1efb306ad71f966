"""A tuning step made of this library's calls from the first norm to the
optimizer: QLoRA linear layers on a frozen NF4 base, norms in front of them, and
on the head's logits either

  preference   the loss over pairs of answers (preferred, other), or
  policy       the clipped policy loss with a KL term over sampled answers.

The reference model is the same base with the adapters switched off
(lora_alpha = 0), so it costs a forward and no memory.  The network is a small
residual block between an embedding and a head, with random weights and random
answers:

    H1, N1 = norm(X)          U = N1 W_up^T + lora      G = silu(U)
    D = G W_down^T + lora     H2, N2 = norm(D + H1)     logits = N2 W_head^T + lora

The SiLU and its derivative are PyTorch's; everything else runs in the library.

Usage: python examples/tuning_step.py [--loss preference|policy] [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_lora_quantize_amd as q  # noqa: E402

RANK, ALPHA = 16, 32.0


class Adapter:
    """An NF4 weight [d_out, d_in] with its LoRA factors and their AdamW state."""

    def __init__(self, d_out, d_in, gen, dev):
        self.w = q.qlora_quantize_nf4(torch.randn(d_out, d_in, generator=gen, device=dev) * 0.02)
        self.params = []
        for shape, std in (((RANK, d_in), 1.0 / RANK), ((d_out, RANK), 0.0)):
            p = torch.randn(shape, generator=gen, device=dev) * std
            self.params.append(q.AdamwParam(p, torch.zeros_like(p), torch.zeros_like(p),
                                            torch.zeros_like(p), p.to(torch.bfloat16)))

    def forward(self, x, alpha, save=True):
        a, b = self.params[0].param_bf16, self.params[1].param_bf16
        t = torch.empty((x.shape[0], RANK), dtype=torch.float32, device=x.device)
        y = q.qlora_linear_fwd(self.w, x, a, b, alpha, T_save=t)
        if save:
            self.x, self.t = x, t
        return y

    def backward(self, dy):
        a, b = self.params
        dx, _, _ = q.qlora_linear_bwd(self.w, self.x, dy, a.param_bf16, b.param_bf16, ALPHA,
                                      T_saved=self.t, dA=a.grad, dB=b.grad)
        return dx


class Norm:
    """An RMS norm whose FP32 weight trains."""

    def __init__(self, d, dev):
        p = torch.ones(d, device=dev)
        self.p = q.AdamwParam(p, torch.zeros_like(p), torch.zeros_like(p), torch.zeros_like(p))

    def forward(self, x, residual=None):
        self.out = q.qlora_norm_fwd(x, self.p.param, kind=q.QLORA_NORM_RMS, residual=residual)
        return self.out.H, self.out.Y

    def backward(self, dy, dh=None):
        return q.qlora_norm_bwd(dy, self.out.H, self.p.param, None, self.out.rstd,
                                kind=q.QLORA_NORM_RMS, dH=dh, dgamma=self.p.grad).dX


class Model:
    def __init__(self, d, ff, vocab, seed, dev):
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)
        self.embedding = torch.randn(vocab, d, generator=gen, device=dev).to(torch.bfloat16)
        self.up, self.down = Adapter(ff, d, gen, dev), Adapter(d, ff, gen, dev)
        self.head = Adapter(vocab, d, gen, dev)
        self.n1, self.n2 = Norm(d, dev), Norm(d, dev)
        params = [p for layer in (self.up, self.down, self.head) for p in layer.params]
        self.params = q.AdamwParamSet(params + [self.n1.p, self.n2.p])
        self.sumsq = torch.zeros(1, dtype=torch.float64, device=dev)
        self.steps = 0

    def logits(self, tokens, alpha=ALPHA, save=True):
        x = self.embedding[tokens]
        h1, y = self.n1.forward(x)
        u = self.up.forward(y, alpha, save)
        if save:
            self.u = u
        y = self.down.forward(torch.nn.functional.silu(u), alpha, save)
        _, y = self.n2.forward(y, residual=h1)
        return self.head.forward(y, alpha, save)

    def backward(self, dlogits):
        dh2 = self.n2.backward(self.head.backward(dlogits))   # of D and of H1
        u = self.u.float()
        s = torch.sigmoid(u)
        du = self.down.backward(dh2).float() * (s * (1 + u * (1 - s)))
        self.n1.backward(self.up.backward(du.to(torch.bfloat16)), dh=dh2)

    def update(self, lr, max_norm=1.0):
        self.steps += 1
        self.sumsq.zero_()
        q.qlora_grad_sumsq(self.params, self.sumsq)
        q.qlora_adamw_step(self.params, lr=lr, step=self.steps, grad_sumsq=self.sumsq,
                           max_grad_norm=max_norm)


def answers(pairs, longest, vocab, seed, dev):
    """(tokens, targets, offsets) of 2 * pairs random answers: the target of a
    token is its successor, a third of each answer is its prompt, which does
    not count, nor does the last token."""
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(longest // 2, longest + 1, (2 * pairs,), generator=gen).tolist()
    tokens = torch.randint(0, vocab, (sum(lens),), generator=gen)
    targets, offsets = torch.roll(tokens, -1), [0]
    for n in lens:
        a = offsets[-1]
        targets[a:a + n // 3] = q.IGNORE_INDEX
        targets[a + n - 1] = q.IGNORE_INDEX
        offsets.append(a + n)
    return tokens.to(dev), targets.to(dev), torch.tensor(offsets, device=dev)


def run(loss="preference", steps=10, pairs=4, longest=48, d=512, ff=1024, vocab=4000, lr=2e-3,
        seed=0, device="cuda", show=print):
    """The loss of every step (the policy loss is taken over two updates per
    batch of log-probabilities, so that its ratio moves)."""
    dev = torch.device(device, torch.cuda.current_device()) if device == "cuda" else device
    model = Model(d, ff, vocab, seed, dev)
    tokens, targets, offsets = answers(pairs, longest, vocab, seed, dev)
    ref, _ = q.qlora_token_logp(model.logits(tokens, alpha=0.0, save=False), targets)
    gen = torch.Generator().manual_seed(seed + 1)
    advantages = torch.randn(2 * pairs, generator=gen).to(dev)
    losses, old = [], None
    for step in range(steps):
        logits = model.logits(tokens)
        if loss == "preference":
            out = q.qlora_preference_loss(logits, targets, offsets, ref_logp=ref, beta=0.1,
                                          dlogits=logits)   # the gradient replaces the logits
            losses.append(out.loss.mean().item())
        else:
            if step % 2 == 0:
                old, _ = q.qlora_token_logp(logits, targets)
            out = q.qlora_policy_loss(logits, targets, offsets, advantages, old_logp=old,
                                      ref_logp=ref, kl_coef=0.01, dlogits=logits,
                                      reduction=q.QLORA_POLICY_SEQUENCE_MEAN)
            losses.append(out.stats[0].item())
        model.backward(out.dlogits)
        model.update(lr)
        show(f"step {step}: {loss} loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--loss", choices=("preference", "policy"), default="preference")
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    run(a.loss, a.steps)
