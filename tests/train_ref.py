"""The operators around the linear layers in 64 bits, from their definitions
(not a test module).  Gradients come from torch's float64 autograd on the CPU,
so no gradient formula is typed twice.  Inputs are the same seeded tensors the
HIP path receives."""
import numpy as np
import torch

IGNORE = -100

# One rounding to nearest BF16 (8 significant bits: values in [1, 2) are 2^-7
# apart) is at most 2^-8 of the value; the FP32 arithmetic before it adds next
# to nothing.
BF16_TOL = 2.0 ** -8 * 1.01


def f64(t):
    return None if t is None else t.detach().cpu().double()


def norm_fwd(X, R, gamma, beta, eps, layer):
    """(Y, H, mean, rstd) in float64; H rounded to X's type first."""
    h = f64(X)
    if R is not None:
        h = (h + f64(R)).to(X.dtype).double()
    mean = h.mean(1) if layer else torch.zeros(h.shape[0], dtype=torch.float64)
    c = h - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None] * f64(gamma)
    if beta is not None:
        y = y + f64(beta)
    return y, h, mean, rstd


def norm_loss(h, gamma, beta, eps, layer, dY, dH):
    """The scalar whose gradient the backward is: <dY, Y> + <dH, H>."""
    mean = h.mean(1, keepdim=True) if layer else 0.0
    c = h - mean
    y = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) * gamma + beta
    out = (dY * y).sum()
    return out + (dH * h).sum() if dH is not None else out


def norm_bwd(H, gamma, eps, layer, dY, dH):
    h = f64(H).requires_grad_()
    g = f64(gamma).requires_grad_()
    b = torch.zeros_like(g).requires_grad_()
    norm_loss(h, g, b, eps, layer, f64(dY), f64(dH)).backward()
    return h.grad, g.grad, b.grad


def token_logp(z, targets, scale=1.0):
    """Differentiable float64 (logp, lse) of logits z; 0 in rows that do not count."""
    x = z * scale
    counted = targets != IGNORE
    lse = torch.logsumexp(x, 1)
    at = torch.where(counted, targets, torch.zeros_like(targets))
    lp = x.gather(1, at[:, None])[:, 0] - lse
    zero = torch.zeros_like(lp)
    return torch.where(counted, lp, zero), torch.where(counted, lse, zero)


def preference(z, targets, offsets, ref, kind, beta, smoothing, margin, mean, scale=1.0):
    """(loss [P], seq_logp [2P], logp) of float64 logits z."""
    logp, _ = token_logp(z, targets, scale)
    P = (len(offsets) - 1) // 2
    s, g = [], []
    for i in range(2 * P):
        rows = slice(offsets[i], offsets[i + 1])
        counted = targets[rows] != IGNORE
        lp = logp[rows][counted]
        gain = lp - ref[rows][counted] if ref is not None else lp
        n = max(1, int(counted.sum())) if mean else 1
        s.append(lp.sum() / n)
        g.append(gain.sum() / n)
    losses = []
    for p in range(P):
        h = g[p] - g[P + p]
        v = beta * h - margin
        if kind == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            losses.append(-(1 - smoothing) * ls(v) - (smoothing * ls(-v) if smoothing else 0.0))
        elif kind == "hinge":
            losses.append(torch.relu(1 - v))
        else:
            losses.append((h - 1 / (2 * beta)) ** 2)
    empty = torch.zeros(0, dtype=torch.float64)
    return (torch.stack(losses) if losses else empty), (torch.stack(s) if s else empty), logp


def policy(z, targets, offsets, adv, old, ref, lo, hi, kl_coef, per_token, seq_mean, scale=1.0):
    """(stats [4], logp) of float64 logits z."""
    logp, _ = token_logp(z, targets, scale)
    S = len(offsets) - 1
    inside = torch.zeros(z.shape[0], dtype=torch.bool)
    for i in range(S):
        inside[offsets[i]:offsets[i + 1]] = True
    total = max(1, int(((targets != IGNORE) & inside).sum()))
    stats = torch.zeros(4, dtype=torch.float64)
    for i in range(S):
        rows = slice(offsets[i], offsets[i + 1])
        counted = targets[rows] != IGNORE
        n = int(counted.sum())
        if n == 0:
            continue
        lp = logp[rows][counted]
        a = adv[rows][counted] if per_token else adv[i]
        r = torch.exp(lp - old[rows][counted]) if old is not None else torch.exp(lp - lp.detach())
        free, held = -a * r, -a * r.clamp(1 - lo, 1 + hi)
        clipped = held > free
        pg = torch.where(clipped, held.detach(), free)
        kl = torch.zeros_like(lp)
        if ref is not None:
            gap = ref[rows][counted] - lp
            kl = torch.exp(gap) - gap - 1
        w = 1.0 / (S * n) if seq_mean else 1.0 / total
        stats = stats + torch.stack([(pg + kl_coef * kl).sum() * w, pg.sum() * w, kl.sum() * w,
                                     clipped.double().sum() * w])
    return stats, logp


def slope(f, x, v, step):
    """Central difference of the scalar f at x along v."""
    return float((f(x + step * v) - f(x - step * v)) / (2 * step))


def max_err(got, ref):
    got, ref = np.asarray(f64(got)), np.asarray(f64(ref))
    return float(np.abs(got - ref).max()) if ref.size else 0.0
