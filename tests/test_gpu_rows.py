"""The row kernels where their launch shape changes: batches of more rows than
one turn of the grid, rows that no workgroup group fills, arrays large enough to
pass the caches, every width at which the policy kernel changes its thread
count, and many sequences.  Tolerances as in test_gpu_norm.py and
test_gpu_losses.py."""
import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from parity_util import assert_close, say
import train_ref as ref
from train_ref import IGNORE

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
EPS = 1e-5


def _draw(seed, shape, dtype, std=1.0, mean=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)


def _tol(dtype, fro, mx):
    return (ref.BF16_TOL, ref.BF16_TOL) if dtype == torch.bfloat16 else (fro, mx)


@pytest.mark.parametrize("rows,width", [(20001, 72), (9001, 520), (4099, 1032), (3001, 4104),
                                        (1201, 8200), (700, 16384), (601, 20008)])
@pytest.mark.parametrize("kind", [q.QLORA_NORM_LAYER, q.QLORA_NORM_RMS])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norms_over_many_turns(rows, width, kind, dtype):
    """More rows than the persistent grid takes at once, the last turn ragged:
    every row equals that row computed in a batch of its own few, bit for bit,
    and the weight gradients hold."""
    say(f"norm turns: {rows}x{width} {dtype} kind={kind}")
    layer = kind == q.QLORA_NORM_LAYER
    X, R = _draw(1, (rows, width), dtype, 1.5, 0.2), _draw(2, (rows, width), dtype)
    dY, dH = _draw(3, (rows, width), dtype), _draw(4, (rows, width), dtype)
    gamma = _draw(5, (width,), torch.float32, 0.2, 1.0)
    beta = _draw(6, (width,), torch.float32) if layer else None
    o = q.qlora_norm_fwd(X, gamma, beta, eps=EPS, kind=kind, residual=R)
    b = q.qlora_norm_bwd(dY, o.H, gamma, o.mean, o.rstd, kind=kind, dH=dH, need_dbeta=layer)
    for at in (slice(0, 5), slice(rows // 2, rows // 2 + 7), slice(rows - 3, rows)):
        s = q.qlora_norm_fwd(X[at], gamma, beta, eps=EPS, kind=kind, residual=R[at])
        assert torch.equal(s.Y, o.Y[at]) and torch.equal(s.H, o.H[at])
        assert torch.equal(s.rstd, o.rstd[at])
        m = o.mean[at].contiguous() if layer else None
        t = q.qlora_norm_bwd(dY[at], s.H, gamma, m, s.rstd, kind=kind, dH=dH[at],
                             need_dgamma=False)
        assert torch.equal(t.dX, b.dX[at])
    y, h, mean, rstd = ref.norm_fwd(X[:64], R[:64], gamma, beta, EPS, layer)
    assert_close("Y", ref.f64(o.Y[:64]), y, *_tol(dtype, 1e-6, 5e-6))
    n = (o.H.double() - (o.mean.double()[:, None] if layer else 0.0)) * o.rstd.double()[:, None]
    # sums over up to 20001 rows: sqrt(rows) 2^-24 = 8.4e-6
    assert_close("dgamma", ref.f64(b.dgamma), ref.f64((dY.double() * n).sum(0)), 2e-5, 2e-5)
    if layer:
        assert_close("dbeta", ref.f64(b.dbeta), ref.f64(dY.double().sum(0)), 2e-5, 2e-5)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_arrays_that_pass_the_caches(dtype):
    """Arrays of 128 MB and more are read and written past the caches'
    retention: the same bits as in small batches."""
    width = 4104
    rows = (128 << 20) // (width * (2 if dtype == torch.bfloat16 else 4)) + 3
    say(f"norm past the caches: {rows}x{width} {dtype}")
    X, R, dY = (_draw(k, (rows, width), dtype) for k in (11, 12, 13))
    gamma = _draw(14, (width,), dtype, 0.2, 1.0)
    o = q.qlora_norm_fwd(X, gamma, eps=EPS, residual=R)
    b = q.qlora_norm_bwd(dY, o.H, gamma, o.mean, o.rstd, need_dbeta=True)
    f = q.qlora_norm_bwd(dY, o.H, gamma, o.mean, o.rstd, need_dgamma=False)
    assert torch.equal(f.dX, b.dX)
    for a in range(0, rows, 4000):
        at = slice(a, min(rows, a + 4000))
        s = q.qlora_norm_fwd(X[at], gamma, eps=EPS, residual=R[at])
        assert torch.equal(s.Y, o.Y[at]) and torch.equal(s.H, o.H[at])
        t = q.qlora_norm_bwd(dY[at], s.H, gamma, s.mean, s.rstd, need_dgamma=False)
        assert torch.equal(t.dX, b.dX[at])
    n = (o.H.double() - o.mean.double()[:, None]) * o.rstd.double()[:, None]
    assert_close("dgamma", ref.f64(b.dgamma), ref.f64((dY.double() * n).sum(0)), 2e-5, 2e-5)


def _batch(seed, lens, vocab, dtype, pad):
    rows = sum(lens)
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 2.5
    t = torch.randint(0, vocab, (rows,), generator=g)
    z.scatter_(1, t[:, None], 6.0 + 2.0 * torch.randn(rows, 1, generator=g))
    buf = torch.full((rows, vocab + pad), float("nan"), dtype=dtype, device=DEV)
    buf[:, :vocab] = z.to(dtype).to(DEV)
    off = [0]
    for n in lens:
        off.append(off[-1] + n)
    t[torch.rand(rows, generator=g) < 0.2] = IGNORE
    return buf[:, :vocab], t, off, g


def _check_policy(seed, lens, vocab, dtype, pad, per_token, seq_mean):
    z, t, off, g = _batch(seed, lens, vocab, dtype, pad)
    x = ref.f64(z).requires_grad_()
    base = ref.token_logp(x.detach(), t)[0]
    old = (base + 0.2 * torch.randn(len(base), generator=g).double()).float()
    rf = (base + 0.3 * torch.randn(len(base), generator=g).double()).float()
    adv = torch.randn(len(base) if per_token else len(lens), generator=g)
    red = q.QLORA_POLICY_SEQUENCE_MEAN if seq_mean else q.QLORA_POLICY_TOKEN_MEAN
    o = q.qlora_policy_loss(z, t.to(DEV), torch.tensor(off, device=DEV), adv.to(DEV),
                            old_logp=old.to(DEV), ref_logp=rf.to(DEV), kl_coef=0.1,
                            per_token=per_token, reduction=red)
    stats, logp = ref.policy(x, t, off, adv.double(), old.double(), rf.double(), 0.2, 0.2, 0.1,
                             per_token, seq_mean)
    stats[0].backward()
    assert ((ref.f64(o.logp) - logp.detach()).abs() <= 5e-6 + 1e-6 * logp.detach().abs()).all()
    assert ref.max_err(o.stats, stats.detach()) <= 2e-5 * max(1.0, float(adv.abs().max()))
    tol = 5e-5 + (ref.BF16_TOL if dtype == torch.bfloat16 else 0.0)
    assert_close("dlogits", ref.f64(o.dlogits), x.grad, tol, tol)


@pytest.mark.parametrize("vocab", [400, 511, 512, 513, 2048, 2055, 3000, 4096, 4097, 6000, 8193,
                                   12000, 16385, 20000, 24576, 24577, 30001, 32768, 32769, 45000,
                                   49152, 49153, 60001, 65537, 90000, 98304, 98305, 131073])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_policy_at_every_width(vocab, dtype):
    say(f"policy width: {vocab} {dtype}")
    _check_policy(vocab, [3, 0, 4], vocab, dtype, vocab % 3, vocab % 2 == 0, vocab % 4 < 2)


@pytest.mark.parametrize("lens", [[3] * 200, [5] + [0] * 63 + [7], [1, 0, 2] * 400, [2] * 1100,
                                  [1500, 3, 0, 700]])
@pytest.mark.parametrize("seq_mean", [False, True])
def test_policy_over_many_sequences(lens, seq_mean):
    say(f"policy sequences: {len(lens)} of {sum(lens)} rows")
    _check_policy(len(lens), lens, 97, torch.float32, 1, seq_mean, seq_mean)


@pytest.mark.parametrize("pairs,longest", [(1, 40), (70, 9), (3, 300), (130, 31)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_preference_over_many_pairs(pairs, longest, dtype):
    """Batches on both sides of the rule that takes a pair's rows in one
    workgroup."""
    g = torch.Generator().manual_seed(pairs)
    lens = torch.randint(0, longest + 1, (2 * pairs,), generator=g).tolist()
    z, t, off, g = _batch(pairs + 1, lens, 203, dtype, 1)
    say(f"preference pairs: {pairs} of {sum(lens)} rows")
    x = ref.f64(z).requires_grad_()
    rf = (ref.token_logp(x.detach(), t)[0] + 0.2 * torch.randn(sum(lens), generator=g)).float()
    o = q.qlora_preference_loss(z, t.to(DEV), torch.tensor(off, device=DEV), rf.to(DEV), beta=0.3)
    loss, seq, logp = ref.preference(x, t, off, rf.double(), "sigmoid", 0.3, 0.0, 0.0, False)
    loss.mean().backward()
    assert ((ref.f64(o.logp) - logp.detach()).abs() <= 5e-6 + 1e-6 * logp.detach().abs()).all()
    assert ref.max_err(o.loss, loss.detach()) <= 5e-5 * max(1.0, float(loss.detach().max()))
    tol = 5e-5 + (ref.BF16_TOL if dtype == torch.bfloat16 else 0.0)
    assert_close("dlogits", ref.f64(o.dlogits), x.grad, tol, tol)


@pytest.mark.parametrize("rows", [7, 1500])
def test_policy_without_sequences_needs_no_offsets(rows):
    """No sequences and no offsets array: no row counts, whichever way a row's
    place is found."""
    import ctypes

    from bit_quantized_lora_quantize_amd import _train
    z, t, _, _ = _batch(1, [rows], 50, torch.float32, 0)
    td = t.to(DEV)
    l = _train._Logits(z.data_ptr(), td.data_ptr(), rows, 50, 50, IGNORE, q.QLORA_F32, 1.0)
    par = _train._Policy(q.QLORA_POLICY_TOKEN_MEAN, 0, 0.2, 0.2, 0.0, 1.0)
    logp, stats = torch.empty(rows, device=DEV), torch.ones(4, device=DEV)
    d, n = torch.ones_like(z), q.qlora_policy_workspace_bytes(rows, 0)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    st = q.lib().qlora_policy_loss(ctypes.byref(l), None, 0, None, None, None, ctypes.byref(par),
                                   logp.data_ptr(), stats.data_ptr(), d.data_ptr(), 50,
                                   ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    assert st == 0
    assert (stats == 0).all() and (d == 0).all()
    assert torch.equal(logp, q.qlora_token_logp(z, td)[0]) or \
        ref.max_err(logp, q.qlora_token_logp(z, td)[0]) <= 5e-6


def test_captured_calls_replay_like_eager_ones():
    """A graph of the norms and losses, replayed several times over new inputs
    with eager work between, gives the eager calls' bits every time."""
    rows, width, vocab = 600, 1032, 2051
    X, R = _draw(21, (rows, width), torch.bfloat16), _draw(22, (rows, width), torch.bfloat16)
    gamma = _draw(23, (width,), torch.float32, 0.2, 1.0)
    z, t, _, g = _batch(24, [200, 100, 180, 120], vocab, torch.bfloat16, 1)
    z = z.contiguous()
    td, off = t.to(DEV), torch.tensor([0, 200, 300, 480, 600], device=DEV)
    adv = torch.randn(4, generator=g).to(DEV)
    old = torch.full((rows,), -3.0, device=DEV)

    def calls():
        n = q.qlora_norm_fwd(X, gamma, kind=q.QLORA_NORM_RMS, residual=R)
        b = q.qlora_norm_bwd(n.Y, n.H, gamma, None, n.rstd, kind=q.QLORA_NORM_RMS)
        p = q.qlora_preference_loss(z, td, off, ref_logp=old)
        c = q.qlora_policy_loss(z, td, off, adv, old_logp=old, ref_logp=old, kl_coef=0.1)
        return [n.Y, n.H, b.dX, b.dgamma, p.loss, p.logp, p.dlogits, c.stats, c.dlogits]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()                                  # the library is loaded before the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for turn in range(4):
        X.copy_(_draw(30 + turn, (rows, width), torch.bfloat16))
        z.copy_(_draw(40 + turn, (rows, vocab), torch.bfloat16, 2.0))
        old.fill_(-7.0 - turn)
        want = [w.clone() for w in calls()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for h, w in zip(held, want):
            assert torch.equal(h, w), turn
