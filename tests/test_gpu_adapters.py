"""Adapters of many requests on the GPU, forward and backward, against their
definition in 64 bits with a bound for every element."""
import math
import random

import pytest
import torch

import adapters_ref as ref
import bit_quantized_lora_quantize_amd as q
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def _gpu(b):
    return {k: v.to(DEV) if v is not None else None for k, v in b.items()}


def _bank(d):
    return q.AdapterBank(d["A"], d["B"], d["scale"])


def _forward(b, d=None):
    d = d or _gpu(b)
    plan = q.qlora_adapters_plan(d["index"], b["A"].shape[0])
    out = q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=d["Y0"])
    Y, T, eY, eT = ref.fwd(b["X"], b["index"], b["A"], b["B"], b["scale"], b["Y0"])
    ref.inside(out.T, T, eT, "T")
    ref.inside(out.Y, Y, eY, "Y")
    return out, plan, d


def _backward(b, plan, d, T, packed=False):
    bank = _bank(d)
    X, Xd = b["X"], d["X"]
    if packed:
        Xd = q.qlora_pack8(Xd)
        X = q.qlora_unpack8(Xd)
    out = q.qlora_adapters_bwd(d["dY"], Xd, T, bank, plan, dX0=d["dX0"])
    want, bound = ref.bwd(X, b["index"], T, b["A"], b["B"], b["scale"], b["dY"], b["dX0"])
    for k in ("dA", "dB", "dX"):
        ref.inside(getattr(out, k), want[k], bound[k], k)
    return out


# tokens, d_in, d_out, rank, slots, longest run
SHAPES = [(5, 3, 2100, 8, 2, 1), (70, 5, 7, 4, 2, 30), (2300, 40, 520, 6, 3, 300), (2100, 300, 64, 64, 4, 900),
          (1, 64, 64, 8, 1, 1), (1, 1, 1, 1, 1, 1), (2, 8, 24, 3, 2, 1), (15, 100, 72, 16, 3, 1), (16, 256, 264, 16, 16, 1),
          (17, 63, 65, 17, 4, 2), (40, 520, 129, 32, 40, 1), (63, 128, 1000, 8, 2, 70), (64, 1000, 128, 20, 1, 64),
          (65, 512, 512, 64, 2, 65), (130, 320, 200, 48, 3, 50), (257, 72, 520, 100, 5, 30), (300, 517, 333, 7, 4, 90),
          (333, 1000, 517, 8, 3, 40), (129, 264, 136, 128, 2, 129), (200, 136, 264, 160, 3, 40), (70, 264, 512, 256, 2, 40),
          (90, 77, 51, 255, 2, 33), (1000, 192, 64, 16, 7, 200), (1025, 64, 96, 16, 9, 3), (2500, 128, 72, 24, 6, 700)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("base", [True, False])
def test_forward_and_backward(shape, base):
    say(f"adapters {shape} base={base}")
    b = ref.batch(sum(shape), *shape, base=base)
    out, plan, d = _forward(b)
    plain = _backward(b, plan, d, out.T)
    kept = _backward(b, plan, d, out.T, packed=True)
    assert torch.equal(plain.dB, kept.dB) and torch.equal(plain.dX, kept.dX)
    # the packed input is the restored matrix, bit for bit
    d["X"] = q.qlora_unpack8(q.qlora_pack8(d["X"]))
    again = q.qlora_adapters_bwd(d["dY"], d["X"], out.T, _bank(d), plan, dX0=d["dX0"])
    assert torch.equal(again.dA, kept.dA)


@pytest.mark.parametrize("M,d_in,d_out,r,slots", [(4096, 512, 264, 16, 3), (9000, 64, 128, 8, 1), (6000, 256, 64, 64, 2),
                                                    (9000, 72, 4100, 30, 3), (9001, 2051, 64, 64, 2), (9000, 64, 4096, 100, 2),
                                                    (8500, 4100, 72, 100, 2), (8200, 64, 2051, 200, 1), (8200, 2056, 40, 200, 2)])
def test_many_tokens_of_one_slot(M, d_in, d_out, r, slots):
    """Slots of several token splits, whose partial results are added; wide rows,
    of which an item of the expansion takes several tiles, at every rank's width
    of its items."""
    b = ref.batch(M, M, d_in, d_out, r, slots, 3000, none=0.05)
    out, plan, d = _forward(b)
    _backward(b, plan, d, out.T)
    _backward(b, plan, d, out.T, packed=True)


@pytest.mark.parametrize("M,slots", [(1, 2048), (1024, 2048), (5000, 2048), (3000, 1), (4097, 300), (40000, 5)])
def test_plan_of_many_slots(M, slots):
    """T identifies which slot served a token: A_a = a + 1 in one column."""
    g = torch.Generator().manual_seed(M + slots)
    index = torch.randint(-2, slots + 2, (M,), generator=g, dtype=torch.int32)
    A = torch.zeros(slots, 1, 8)
    A[:, 0, 0], A[:, 0, 1] = torch.arange(slots) % 256, torch.arange(slots) // 256
    X = torch.zeros(M, 8)
    X[:, 0], X[:, 1] = 1.0, 256.0
    bank = q.AdapterBank(A.to(DEV).bfloat16(), torch.zeros(slots, 8, 1, device=DEV).bfloat16(), torch.ones(slots, device=DEV))
    plan = q.qlora_adapters_plan(index.to(DEV), slots)
    T = q.qlora_adapters_fwd(X.to(DEV).bfloat16(), bank, plan).T.cpu()[:, 0]
    want = torch.where((index >= 0) & (index < slots), index, torch.zeros_like(index)).float()
    assert torch.equal(T, want)
    # and each token once: dB of slot a counts its tokens
    ones = torch.ones(M, 8, device=DEV).bfloat16()
    dB = q.qlora_adapters_bwd(ones, X.to(DEV).bfloat16(), torch.ones(M, 1, device=DEV), bank, plan).dB.cpu()
    count = torch.bincount(index[(index >= 0) & (index < slots)].long(), minlength=slots).float()
    assert torch.equal(dB[:, 3, 0], count)


def test_tokens_without_an_adapter():
    """Their rows of X and dY are not read (NaN there reaches nothing), Y and dX are
    Y0's and dX0's bits, T is 0; a batch of nothing else leaves zero gradients."""
    b = ref.batch(1, 100, 96, 80, 16, 3, 5, none=0.4)
    none = b["index"] < 0
    assert none.any() and not none.all()
    b["X"][none] = float("nan")
    b["dY"][none] = float("nan")
    d = _gpu(b)
    plan = q.qlora_adapters_plan(d["index"], 3)
    out = q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=d["Y0"])
    T = out.T.clone()
    assert (T.cpu()[none] == 0).all()
    T[none.to(DEV)] = float("nan")
    g = q.qlora_adapters_bwd(d["dY"], d["X"], T, _bank(d), plan, dX0=d["dX0"])
    assert torch.equal(out.Y.cpu()[none], b["Y0"][none]) and torch.equal(g.dX.cpu()[none], b["dX0"][none])
    assert all(t.isfinite().all() for t in (out.Y, g.dX, g.dA, g.dB))
    plan = q.qlora_adapters_plan(torch.full((100,), -1, dtype=torch.int32, device=DEV), 3)
    out = q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=d["Y0"])
    g = q.qlora_adapters_bwd(d["dY"], d["X"], T, _bank(d), plan)
    assert torch.equal(out.Y, d["Y0"]) and (out.T == 0).all()
    assert (g.dX == 0).all() and (g.dA == 0).all() and (g.dB == 0).all()
    assert (q.qlora_adapters_fwd(d["X"], _bank(d), plan).Y == 0).all()


def test_a_tokens_nan_stays_with_it_and_its_slot():
    b = ref.batch(2, 90, 128, 72, 16, 3, 1, none=0.1)
    slot = int(b["index"][b["index"] >= 0][7])
    row = int(torch.nonzero(b["index"] == slot)[0])
    clean, _, _ = _forward(b)
    X, dY = b["X"].clone(), b["dY"].clone()
    X[row, 5] = float("nan")
    dY[row, 3] = float("inf")
    d = _gpu({**b, "X": X, "dY": dY})
    plan = q.qlora_adapters_plan(d["index"], 3)
    out = q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=d["Y0"])
    others = torch.arange(90) != row
    assert torch.equal(out.Y.cpu()[others], clean.Y.cpu()[others]) and out.Y[row].isnan().all()
    assert torch.equal(out.T.cpu()[others], clean.T.cpu()[others]) and out.T[row].isnan().all()
    g = q.qlora_adapters_bwd(d["dY"], d["X"], clean.T, _bank(d), plan, dX0=d["dX0"])
    rest = [a for a in range(3) if a != slot]
    assert g.dX.cpu()[others].isfinite().all() and not g.dX[row].isfinite().any()
    assert g.dA[rest].isfinite().all() and g.dB[rest].isfinite().all()
    assert not g.dA[slot].isfinite().any()
    assert not g.dB[slot, 3].isfinite().any() and g.dB[slot, 4:].isfinite().all()


def test_a_slots_nan_stays_with_its_tokens():
    """Also past the ranks and rows next to it in memory."""
    b = ref.batch(3, 90, 100, 70, 12, 3, 4, none=0.1)
    clean, plan, d = _forward(b)
    grads = _backward(b, plan, d, clean.T)
    for name in ("A", "B"):
        bad = {**d, name: d[name].clone()}
        bad[name][1] = float("nan")
        out = q.qlora_adapters_fwd(d["X"], _bank(bad), plan, Y0=d["Y0"])
        g = q.qlora_adapters_bwd(d["dY"], d["X"], clean.T, _bank(bad), plan, dX0=d["dX0"])
        keep = (b["index"] != 1).to(DEV)
        assert torch.equal(out.Y[keep], clean.Y[keep]) and torch.equal(g.dX[keep], grads.dX[keep])
        assert out.Y[~keep].isnan().all() and g.dX[~keep].isnan().all()
        assert torch.equal(g.dA[[0, 2]], grads.dA[[0, 2]]) and torch.equal(g.dB, grads.dB)


@pytest.mark.parametrize("shape", [(70, 130, 77, 9, 3, 20), (200, 256, 136, 16, 2, 64)])
def test_outputs_over_inputs_and_given_buffers(shape):
    b = ref.batch(4, *shape)
    out, plan, d = _forward(b)
    g = _backward(b, plan, d, out.T)
    Y, T = d["Y0"].clone(), torch.full_like(out.T, 9.0)
    ws = torch.full((q.qlora_adapters_workspace_bytes(_bank(d), shape[0], backward=True) // 4 + 4,), float("nan"), device=DEV)
    got = q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=Y, Y=Y, T=T, workspace=ws)
    assert got.Y is Y and torch.equal(Y, out.Y) and torch.equal(T, out.T)
    Y = d["Y0"].clone()
    q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=Y, Y=Y, save_T=False)
    assert torch.equal(Y, out.Y)
    dX, dA, dB = d["dX0"].clone(), torch.full_like(g.dA, 5.0), torch.full_like(g.dB, 5.0)
    ws.fill_(float("nan"))
    q.qlora_adapters_bwd(d["dY"], d["X"], out.T, _bank(d), plan, dX0=dX, dX=dX, dA=dA, dB=dB, workspace=ws)
    assert torch.equal(dX, g.dX) and torch.equal(dA, g.dA) and torch.equal(dB, g.dB)
    no_dx = q.qlora_adapters_bwd(d["dY"], d["X"], out.T, _bank(d), plan, need_dx=False)
    assert no_dx.dX is None and torch.equal(no_dx.dA, g.dA) and torch.equal(no_dx.dB, g.dB)


def _shifted(t):
    """The same values one element into a storage of their own, between sevens."""
    store = torch.full((t.numel() + 2,), 7.0, dtype=t.dtype, device=DEV)
    v = store[1:-1].view(t.shape)
    v.copy_(t)
    return v, store


@pytest.mark.parametrize("shape", [(70, 128, 64, 8, 3, 20), (33, 77, 51, 5, 2, 8)])
def test_arrays_off_alignment(shape):
    b = ref.batch(5, *shape)
    out, plan, d = _forward(b)
    g = _backward(b, plan, d, out.T)
    s = {k: _shifted(v)[0] if k in ("X", "A", "B", "Y0", "dY", "dX0", "scale") else v for k, v in d.items()}
    Y, Ys = _shifted(torch.zeros_like(out.Y))
    T, Ts = _shifted(torch.zeros_like(out.T))
    got = q.qlora_adapters_fwd(s["X"], _bank(s), plan, Y0=s["Y0"], Y=Y, T=T)
    wY, wT, eY, eT = ref.fwd(b["X"], b["index"], b["A"], b["B"], b["scale"], b["Y0"])
    ref.inside(got.Y, wY, eY, "Y")
    ref.inside(got.T, wT, eT, "T")
    dX, dXs = _shifted(torch.zeros_like(g.dX))
    dA, dAs = _shifted(torch.zeros_like(g.dA))
    dB, dBs = _shifted(torch.zeros_like(g.dB))
    q.qlora_adapters_bwd(s["dY"], s["X"], _shifted(out.T)[0], _bank(s), plan, dX0=s["dX0"], dX=dX, dA=dA, dB=dB)
    want, bound = ref.bwd(b["X"], b["index"], out.T, b["A"], b["B"], b["scale"], b["dY"], b["dX0"])
    for name, t in (("dX", dX), ("dA", dA), ("dB", dB)):
        ref.inside(t, want[name], bound[name], name)
    for store in (Ys, Ts, dXs, dAs, dBs):
        assert store[0] == 7 and store[-1] == 7


def test_order_of_requests_does_not_matter():
    """The same tokens in another order give the same rows, bit for bit."""
    b = ref.batch(6, 150, 200, 96, 16, 4, 20)
    out, _, d = _forward(b)
    perm = torch.randperm(150, generator=torch.Generator().manual_seed(1)).to(DEV)
    plan = q.qlora_adapters_plan(d["index"][perm].contiguous(), 4)
    got = q.qlora_adapters_fwd(d["X"][perm].contiguous(), _bank(d), plan, Y0=d["Y0"][perm].contiguous())
    assert torch.equal(got.Y, out.Y[perm]) and torch.equal(got.T, out.T[perm])


def test_same_bits_every_time():
    b = ref.batch(7, 3000, 256, 200, 16, 5, 60)
    out, plan, d = _forward(b)
    g = _backward(b, plan, d, out.T, packed=True)
    for _ in range(3):
        plan = q.qlora_adapters_plan(d["index"], 5)
        o2 = q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=d["Y0"])
        g2 = q.qlora_adapters_bwd(d["dY"], q.qlora_pack8(d["X"]), o2.T, _bank(d), plan, dX0=d["dX0"])
        assert torch.equal(o2.Y, out.Y) and torch.equal(o2.T, out.T)
        assert all(torch.equal(x, y) for x, y in zip(g2, g))


def test_plan_of_other_sizes_writes_nothing():
    """The binding refuses it; the kernels, given such a buffer, do nothing."""
    b = ref.batch(8, 50, 64, 64, 8, 3, 5)
    d = _gpu(b)
    plan = q.qlora_adapters_plan(d["index"][:40].contiguous(), 3)
    with pytest.raises(ValueError):
        q.qlora_adapters_fwd(d["X"], _bank(d), plan)
    room = torch.zeros(q.qlora_adapters_plan_bytes(50, 3), dtype=torch.uint8, device=DEV)
    for source in (plan.buffer, room):
        room.zero_()
        n = min(room.numel(), source.numel())
        room[:n] = source[:n]
        fake = q.AdapterPlan(50, 3, room)
        Y = torch.full((50, 64), 3.0, dtype=torch.bfloat16, device=DEV)
        T = torch.full((50, 8), 3.0, device=DEV)
        dA = torch.full((3, 8, 64), 3.0, device=DEV)
        q.qlora_adapters_fwd(d["X"], _bank(d), fake, Y0=d["Y0"], Y=Y, T=T)
        q.qlora_adapters_bwd(d["dY"], d["X"], T, _bank(d), fake, dX=Y, dA=dA)
        assert (Y == 3).all() and (T == 3).all() and (dA == 3).all()


def test_no_tokens():
    b = ref.batch(9, 0, 64, 72, 8, 3, 5)
    d = _gpu(b)
    plan = q.qlora_adapters_plan(d["index"], 3)
    out = q.qlora_adapters_fwd(d["X"], _bank(d), plan)
    dA, dB = torch.full((3, 8, 64), 5.0, device=DEV), torch.full((3, 72, 8), 5.0, device=DEV)
    g = q.qlora_adapters_bwd(d["dY"], d["X"], out.T, _bank(d), plan, dA=dA, dB=dB)
    assert out.Y.shape == (0, 72) and g.dX.shape == (0, 64) and (dA == 0).all() and (dB == 0).all()


def test_gradients_against_differences():
    """<G, Y> differs along a direction as the gradients say.  The forward is
    linear in X and in each factor, so a central difference in 64 bits has no
    error of its own; the gradients' is bounded by their elements' bounds."""
    b = ref.batch(10, 120, 96, 72, 16, 3, 11)
    out, plan, d = _forward(b)
    g = _backward(b, plan, d, out.T)
    want, bound = ref.bwd(b["X"], b["index"], out.T, b["A"], b["B"], b["scale"], b["dY"], b["dX0"])
    _, _, _, eT = ref.fwd(b["X"], b["index"], b["A"], b["B"], b["scale"], b["Y0"])
    gen = torch.Generator().manual_seed(11)
    G = ref.f64(b["dY"])

    def value(**kw):
        a = {**{k: ref.f64(b[k]) for k in ("X", "A", "B", "scale", "Y0")}, **kw}
        return float((G * ref.fwd(a["X"], b["index"], a["A"], a["B"], a["scale"], a["Y0"])[0]).sum())

    for name, grad, base in (("X", "dX", ref.f64(b["dX0"])), ("A", "dA", 0.0), ("B", "dB", 0.0)):
        v = torch.randn(b[name].shape, generator=gen, dtype=torch.float64)
        x = ref.f64(b[name])
        slope = (value(**{name: x + v}) - value(**{name: x - v})) / 2
        got = float(((ref.f64(getattr(g, grad)) - base) * v).sum())
        room = float((bound[grad] * v.abs()).sum())
        if name == "B":   # T entered as it was computed
            room += float(sum((G[ref.rows_of(b["index"], a)].abs().t() @ eT[ref.rows_of(b["index"], a)] * v[a].abs()).sum()
                              for a in range(3)))
        say(f"  {grad}: slope {slope:.6g}, gradient {got:.6g}, room {room:.2g}")
        assert abs(got - slope) <= room + 1e-9 * abs(slope)


def test_other_streams_and_two_calls_at_once():
    b1, b2 = ref.batch(11, 700, 256, 128, 16, 3, 90), ref.batch(12, 500, 128, 264, 32, 5, 9)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    d1, d2 = _gpu(b1), _gpu(b2)
    torch.cuda.synchronize()
    res = []
    for b, d, s in ((b1, d1, s1), (b2, d2, s2)):
        with torch.cuda.stream(s):
            plan = q.qlora_adapters_plan(d["index"], b["A"].shape[0])
            out = q.qlora_adapters_fwd(d["X"], _bank(d), plan, Y0=d["Y0"])
            res.append((out, q.qlora_adapters_bwd(d["dY"], q.qlora_pack8(d["X"]), out.T, _bank(d), plan, dX0=d["dX0"])))
    torch.cuda.synchronize()
    for b, d, (out, g) in ((b1, d1, res[0]), (b2, d2, res[1])):
        ref_out, plan, _ = _forward(b, d)
        again = _backward(b, plan, d, ref_out.T, packed=True)
        assert torch.equal(out.Y, ref_out.Y) and all(torch.equal(x, y) for x, y in zip(g, again))


def test_captured_and_replayed():
    """A graph of plan, forward, checkpoint and backward follows its inputs: other
    tokens, other slots, other factors, with eager work between the replays."""
    shape = (200, 128, 96, 16, 4, 30)
    b = ref.batch(13, *shape)
    d = _gpu(b)
    bank = _bank(d)
    room = q.qlora_adapters_plan(d["index"], 4)
    X8 = q.Packed8.empty(200, 128)
    ws = torch.empty(q.qlora_adapters_workspace_bytes(bank, 200, backward=True), dtype=torch.uint8, device=DEV)

    def step():
        plan = q.qlora_adapters_plan(d["index"], 4, out=room)
        out = q.qlora_adapters_fwd(d["X"], bank, plan, Y0=d["Y0"], workspace=ws)
        g = q.qlora_adapters_bwd(d["dY"], q.qlora_pack8(d["X"], out=X8), out.T, bank, plan, dX0=d["dX0"], workspace=ws)
        return (out.Y, out.T, *g)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(20, 24):
        for k, v in ref.batch(seed, *shape).items():
            d[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        assert all(torch.equal(x, y) for x, y in zip(got, step()))
        (torch.randn(1000, 1000, device=DEV) @ torch.randn(1000, 1000, device=DEV)).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, held))


def test_two_graphs_share_a_workspace_and_a_plan():
    """One projection's forward and another's backward captured apart over the same
    scratch memory and the same plan, replayed in turn in both orders."""
    b1, b2 = ref.batch(14, 300, 200, 90, 24, 3, 40), ref.batch(14, 300, 64, 264, 70, 3, 40)
    d1, d2 = _gpu(b1), _gpu(b2)
    n1, n2 = _bank(d1), _bank(d2)
    plan = q.qlora_adapters_plan(d1["index"], 3)
    room = max(q.qlora_adapters_workspace_bytes(n, 300, backward=True) for n in (n1, n2))
    ws = torch.empty(room, dtype=torch.uint8, device=DEV)
    T2 = q.qlora_adapters_fwd(d2["X"], n2, plan).T
    calls = [lambda **kw: q.qlora_adapters_fwd(d1["X"], n1, plan, Y0=d1["Y0"], **kw),
             lambda **kw: q.qlora_adapters_bwd(d2["dY"], d2["X"], T2, n2, plan, dX0=d2["dX0"], **kw)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    graphs, held = [], []
    for call in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            held.append(call(workspace=ws))
    for turn in ((0, 1), (1, 0), (1, 1), (0, 0), (0, 1)):
        ws.fill_(255)
        for out in held:
            for x in out:
                x.zero_()
        for i in turn:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in set(turn):
            assert all(torch.equal(x, y) for x, y in zip(held[i], want[i]))


def test_large_offsets():
    """Rows past 2^31 elements of X and Y, slots past 2^31 bytes of the factors."""
    M, d_in, d_out, r, slots = 70000, 32000, 8, 8, 2
    g = torch.Generator().manual_seed(14)
    X = torch.zeros(M, d_in, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(40, d_in, generator=g).bfloat16()
    X[-40:] = tail.to(DEV)
    index = torch.full((M,), -1, dtype=torch.int32)
    index[-40:] = torch.arange(40, dtype=torch.int32) % 2
    small = {"X": tail, "index": index[-40:].contiguous(), "A": (torch.randn(slots, r, d_in, generator=g) / 180).bfloat16(),
             "B": torch.randn(slots, d_out, r, generator=g).bfloat16(), "scale": torch.ones(slots), "Y0": None,
             "dY": torch.randn(40, d_out, generator=g).bfloat16(), "dX0": None}
    out, plan, d = _forward(small)
    part = _backward(small, plan, d, out.T)
    dY = torch.zeros(M, d_out, dtype=torch.bfloat16, device=DEV)
    dY[-40:] = d["dY"]
    plan = q.qlora_adapters_plan(index.to(DEV), slots)
    full = q.qlora_adapters_fwd(X, _bank(d), plan)
    assert (full.T[:-40] == 0).all()
    Y, T, eY, eT = ref.fwd(small["X"], small["index"], small["A"], small["B"], small["scale"], None)
    ref.inside(full.T[-40:], T, eT, "T")
    ref.inside(full.Y[-40:], Y, eY, "Y")
    T = torch.zeros(M, r, device=DEV)
    T[-40:] = out.T
    big = q.qlora_adapters_bwd(dY, X, T, _bank(d), plan)
    want, bound = ref.bwd(small["X"], small["index"], out.T, small["A"], small["B"], small["scale"], small["dY"], None)
    for name in ("dA", "dB"):
        ref.inside(getattr(big, name), want[name], bound[name], name)
    ref.inside(big.dX[-40:], want["dX"], bound["dX"], "dX")
    assert (big.dX[:100] == 0).all() and part.dX.shape == (40, d_in)
    del X, big, full
    slots, d_in = 300, 16384
    A = torch.zeros(slots, 256, d_in, dtype=torch.bfloat16, device=DEV)
    A[-1, :, 5], A[-1, 3, 7] = 1.0, 2.0
    bank = q.AdapterBank(A, torch.ones(slots, 8, 256, dtype=torch.bfloat16, device=DEV), torch.ones(slots, device=DEV))
    x = torch.zeros(2, d_in, dtype=torch.bfloat16, device=DEV)
    x[:, 5], x[1, 7] = 1.0, 1.0
    plan = q.qlora_adapters_plan(torch.tensor([299, 299], dtype=torch.int32, device=DEV), slots)
    o = q.qlora_adapters_fwd(x, bank, plan)
    assert (o.Y[0] == 256).all() and (o.Y[1] == 258).all()


@pytest.mark.parametrize("seed", range(12))
def test_shapes_at_random(seed):
    """Sizes over the range, odd ones among them, and requests of any length."""
    g = random.Random(seed)
    spread = lambda lo, hi: int(round(math.exp(g.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    shape = (spread(1, 3000), spread(1, 1500), spread(1, 1500), spread(1, 256), spread(1, 60), spread(1, 600))
    say(f"adapters {shape}")
    b = ref.batch(seed, *shape, base=seed % 3 > 0)
    out, plan, d = _forward(b)
    _backward(b, plan, d, out.T, packed=seed % 2 == 0)
