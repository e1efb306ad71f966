"""8-bit activation checkpoints and adapters of many requests in 64 bits, from
their definitions (not a test module), with bounds for each element.

The bounds count, to first order and with a margin of a few per cent (SLACK):
  a rounding to BF16            2^-8 of the value (torch.finfo.eps / 2)
  a BF16 hi + lo pair           2^-16 of the value
  three BF16 terms              2^-24 of the value
  an FP32 sum of n products     n 2^-23 of the sum of their magnitudes (a whole
                                step for each addition, in whatever order)
"""
import numpy as np
import torch

SLACK = 1.05
U8, U16, U24, ADD = 2.0 ** -8, 2.0 ** -16, 2.0 ** -24, 2.0 ** -23


def f64(t):
    return None if t is None else t.detach().cpu().double()


# ------------------------------------------------------------- 8-bit checkpoints

def pack(X):
    """(codes int64 [M, nb * 64], scale float32 [nb, M], restored float32): the
    quotient 127 x / a is correctly rounded in 64 bits from exact 127 x, and a
    quotient nearer to a border than that does not occur unless it is on it."""
    x = X.detach().cpu().float().numpy()
    M, d = x.shape
    nb = -(-d // 64)
    v = np.zeros((M, nb * 64), np.float32)
    v[:, :d] = x
    v = v.reshape(M, nb, 64)
    bad = ~np.isfinite(v).all(2)
    a = np.where(bad, np.float32(0), np.abs(np.where(np.isfinite(v), v, 0)).max(2)).astype(np.float32)
    tiny = a < np.float32(2.0 ** -119)
    most = np.float32(float.fromhex("0x1.020406p+121"))   # the largest whose 127-fold is finite
    scale = np.where(tiny, np.float32(0), np.minimum(a / np.float32(127), most)).astype(np.float32)
    scale = np.where(bad, np.float32(np.nan), scale)
    with np.errstate(all="ignore"):
        codes = np.rint(v.astype(np.float64) * 127.0 / a.astype(np.float64)[..., None])
    codes = np.where((tiny | bad)[..., None], 0.0, codes)
    restored = (codes.astype(np.float32) * scale[..., None]).reshape(M, nb * 64)[:, :d]
    return (torch.from_numpy(codes.astype(np.int64).reshape(M, nb * 64)),
            torch.from_numpy(np.ascontiguousarray(scale.T)), torch.from_numpy(restored.copy()))


# ------------------------------------------------------------- adapters

def rows_of(index, a):
    return torch.nonzero(index.cpu() == a).flatten()


def fwd(X, index, A, B, scale, Y0):
    """(Y, T) in float64, and the bounds of both."""
    X, A, B, scale = f64(X), f64(A), f64(B), f64(scale)
    M, r, K = X.shape[0], A.shape[1], X.shape[1]
    Y = f64(Y0) if Y0 is not None else torch.zeros(M, B.shape[1], dtype=torch.float64)
    T = torch.zeros(M, r, dtype=torch.float64)
    eT, eY = torch.zeros_like(T), torch.zeros_like(Y)
    for a in range(A.shape[0]):
        at = rows_of(index, a)
        if not len(at):
            continue
        x, s = X[at], scale[a]
        T[at] = x @ A[a].t() * s
        mag = (x.abs() @ A[a].abs().t()) * s.abs()
        eT[at] = SLACK * ((K + 2) * ADD) * mag
        Y[at] += T[at] @ B[a].t()
        tb = T[at].abs() @ B[a].abs().t()
        e = (eT[at] + U16 * T[at].abs()) @ B[a].abs().t() + (2 * r + 2) * ADD * tb
        eY[at] = SLACK * (e + U8 * (Y[at].abs() + e))
    return Y, T, eY, eT


def bwd(X, index, T, A, B, scale, dY, dX0):
    """({dX, dA, dB} in float64, their bounds); T as it is given."""
    X, T, A, B, scale, dY = (f64(t) for t in (X, T, A, B, scale, dY))
    M, N = dY.shape
    S, r, K = A.shape
    dX = f64(dX0) if dX0 is not None else torch.zeros(M, K, dtype=torch.float64)
    eX = torch.zeros_like(dX)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    eA, eB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(S):
        at = rows_of(index, a)
        n = len(at)
        if not n:
            continue
        dy, s = dY[at], scale[a]
        U = dy @ B[a] * s
        eU = (N + 2) * ADD * (dy.abs() @ B[a].abs()) * s.abs()
        dX[at] += U @ A[a]
        e = (eU + U16 * U.abs()) @ A[a].abs() + (2 * r + 2) * ADD * (U.abs() @ A[a].abs())
        eX[at] = SLACK * (e + U8 * (dX[at].abs() + e))
        dA[a] = U.t() @ X[at]
        eA[a] = SLACK * ((eU + (U24 + (3 * n + 2) * ADD) * U.abs()).t() @ X[at].abs())
        dB[a] = dy.t() @ T[at]
        eB[a] = SLACK * ((U24 + (3 * n + 2) * ADD) * (dy.abs().t() @ T[at].abs()))
    return {"dX": dX, "dA": dA, "dB": dB}, {"dX": eX, "dA": eA, "dB": eB}


def inside(got, want, bound, name):
    """Every element within its bound; where the bound is 0 the values agree."""
    d = (f64(got) - want).abs()
    over = ~(d <= bound)
    if bool(over.any()):
        at = torch.nonzero(over)[0].tolist()
        raise AssertionError(f"{name}: {int(over.sum())} of {d.numel()} past their bound, first at {at}: "
                             f"got {f64(got)[tuple(at)]:.9g}, want {want[tuple(at)]:.9g} +- {bound[tuple(at)]:.3g}")


def batch(seed, M, d_in, d_out, r, slots, run, none=0.2, base=True):
    """Seeded inputs on the CPU: dict of X, index, A, B, scale, Y0, dY, dX0."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    bf = lambda t: t.to(torch.bfloat16)  # noqa: E731
    index = []
    while len(index) < M:
        a = -1 if float(torch.rand(1, generator=g)) < none else int(torch.randint(0, slots, (1,), generator=g))
        index += [a] * (1 if run <= 1 else int(torch.randint(1, run + 1, (1,), generator=g)))
    return {"X": bf(rand(M, d_in)), "index": torch.tensor(index[:M], dtype=torch.int32),
            "A": bf(rand(slots, r, d_in) / d_in ** 0.5), "B": bf(rand(slots, d_out, r) * 0.3),
            "scale": 0.5 + torch.rand(slots, generator=g), "Y0": bf(rand(M, d_out)) if base else None,
            "dY": bf(rand(M, d_out)), "dX0": bf(rand(M, d_in)) if base else None}
