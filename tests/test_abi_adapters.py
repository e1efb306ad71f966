"""Host checks of the 8-bit checkpoints and of the adapters of many requests:
every bad argument is refused before anything is enqueued (fake device addresses
are never dereferenced), and the binding refuses tensors it cannot describe."""
import ctypes

import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from bit_quantized_lora_quantize_amd import _adapters, _lib

OK, ENULL, ESHAPE, EALIGN, EWS = 0, -1, -2, -3, -4
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return q.lib()


def _p(**kw):
    a = dict(M=4, d=100, codes=0x1000, scale=0x2000)
    a.update(kw)
    return _adapters._Packed(*a.values())


BAD_PACKED = [({"M": -1}, ESHAPE), ({"M": (1 << 21) + 1}, ESHAPE), ({"d": 0}, ESHAPE), ({"d": (1 << 21) + 1}, ESHAPE),
              ({"codes": None}, ENULL), ({"scale": None}, ENULL), ({"codes": 0x1008}, EALIGN), ({"scale": 0x2002}, EALIGN)]


@pytest.mark.parametrize("bad,status", BAD_PACKED)
def test_bad_checkpoints(L, bad, status):
    assert L.qlora_pack8(0, 0x3000, _p(**bad), None) == status
    assert L.qlora_unpack8(_p(**bad), 0, 0x3000, None) == status


def test_pack_refusals(L):
    for ty in (-1, 2):
        assert L.qlora_pack8(ty, 0x3000, _p(), None) == ESHAPE and L.qlora_unpack8(_p(), ty, 0x3000, None) == ESHAPE
    assert L.qlora_pack8(0, None, _p(), None) == ENULL and L.qlora_unpack8(_p(), 0, None, None) == ENULL
    assert L.qlora_pack8(0, 0x3000, None, None) == ENULL and L.qlora_unpack8(None, 0, 0x3000, None) == ENULL
    assert L.qlora_pack8(0, 0x3001, _p(), None) == EALIGN and L.qlora_unpack8(_p(), 1, 0x3002, None) == EALIGN
    assert L.qlora_pack8(0, None, _p(M=0, codes=None, scale=None), None) == OK
    assert L.qlora_unpack8(_p(M=0, codes=None, scale=None), 1, None, None) == OK
    assert q.qlora_pack8_sizes(3, 65) == (3 * 128, 3 * 2 * 4) and q.qlora_pack8_sizes(0, 1) == (0, 0)
    z = ctypes.c_size_t()
    assert L.qlora_pack8_sizes(-1, 5, z, z) == ESHAPE and L.qlora_pack8_sizes(5, 0, z, z) == ESHAPE
    assert L.qlora_pack8_sizes(5, 5, None, z) == ENULL


def test_plan_refusals(L):
    need = q.qlora_adapters_plan_bytes(100, 7)
    f = L.qlora_adapters_plan
    assert need > 0 and f(0x1000, 100, 7, 0x2000, need - 1, None) == EWS
    for M, slots in ((-1, 7), ((1 << 21) + 1, 7), (100, 0), (100, 2049)):
        assert f(0x1000, M, slots, 0x2000, BIG, None) == ESHAPE and q.qlora_adapters_plan_bytes(M, slots) == 0
    assert f(None, 100, 7, 0x2000, BIG, None) == ENULL and f(0x1000, 100, 7, None, BIG, None) == ENULL
    assert f(0x1002, 100, 7, 0x2000, BIG, None) == EALIGN and f(0x1000, 100, 7, 0x2008, BIG, None) == EALIGN
    assert q.qlora_adapters_plan_bytes(0, 1) > 0 and q.qlora_adapters_plan_bytes(1 << 21, 2048) > 0


def _bank(**kw):
    a = dict(slots=3, r=16, d_in=256, d_out=128, A=0x1000, B=0x2000, scale=0x3000)
    a.update(kw)
    return _adapters._Bank(*a.values())


BAD_BANK = [({"slots": 0}, ESHAPE), ({"slots": 2049}, ESHAPE), ({"r": 0}, ESHAPE), ({"r": 257}, ESHAPE), ({"d_in": 0}, ESHAPE),
            ({"d_in": (1 << 21) + 1}, ESHAPE), ({"d_out": 0}, ESHAPE), ({"d_out": (1 << 21) + 1}, ESHAPE), ({"A": None}, ENULL),
            ({"B": None}, ENULL), ({"scale": None}, ENULL), ({"A": 0x1001}, EALIGN), ({"B": 0x2001}, EALIGN), ({"scale": 0x3002}, EALIGN)]


def _fwd(L, bank=None, **kw):
    a = dict(plan=0x4000, pn=BIG, X=0x5000, M=10, Y0=0x6000, Y=0x7000, T=0x8000, ws=0x9000, n=BIG)
    a.update(kw)
    return L.qlora_adapters_fwd(bank if bank is not None else _bank(), *a.values(), None)


def _bwd(L, bank=None, **kw):
    a = dict(plan=0x4000, pn=BIG, X=0x5000, X8=None, T=0x8000, dY=0x6000, M=10, dX0=0xA000, dX=0xB000, dA=0xC000, dB=0xD000, ws=0x9000, n=BIG)
    a.update(kw)
    return L.qlora_adapters_bwd(bank if bank is not None else _bank(), *a.values(), None)


@pytest.mark.parametrize("bad,status", BAD_BANK)
def test_bad_banks(L, bad, status):
    assert _fwd(L, _bank(**bad)) == status and _bwd(L, _bank(**bad)) == status
    if status == ESHAPE:
        for back in (0, 1):
            assert L.qlora_adapters_workspace_bytes(back, _bank(**bad), 10) == 0


def test_forward_refusals(L):
    assert L.qlora_adapters_fwd(None, 0x4000, BIG, 0x5000, 10, None, 0x7000, None, 0x9000, BIG, None) == ENULL
    assert _fwd(L, M=-1) == ESHAPE and _fwd(L, M=(1 << 21) + 1) == ESHAPE
    for name in ("plan", "X", "Y", "ws"):
        assert _fwd(L, **{name: None}) == ENULL
    for name, at in (("plan", 0x4008), ("X", 0x5001), ("Y0", 0x6001), ("Y", 0x7001), ("T", 0x8002), ("ws", 0x9008)):
        assert _fwd(L, **{name: at}) == EALIGN
    need = L.qlora_adapters_workspace_bytes(0, _bank(), 10)
    assert need > 0 and _fwd(L, n=need - 1) == EWS and _fwd(L, pn=q.qlora_adapters_plan_bytes(10, 3) - 1) == EWS
    assert L.qlora_adapters_workspace_bytes(0, _bank(), -1) == 0 and L.qlora_adapters_workspace_bytes(0, None, 1) == 0
    assert _fwd(L, _bank(A=None, B=None, scale=None), M=0, plan=None, pn=0, X=None, Y0=None, Y=None, T=None, ws=None, n=0) == OK


def test_backward_refusals(L):
    assert _bwd(L, M=-1) == ESHAPE and _bwd(L, M=(1 << 21) + 1) == ESHAPE
    for name in ("plan", "X", "T", "dY", "dA", "dB", "ws"):
        assert _bwd(L, **{name: None}) == ENULL
    for name, at in (("plan", 0x4008), ("X", 0x5001), ("T", 0x8002), ("dY", 0x6001), ("dX0", 0xA001), ("dX", 0xB001), ("dA", 0xC002),
                     ("dB", 0xD001), ("ws", 0x9008)):
        assert _bwd(L, **{name: at}) == EALIGN
    x8 = dict(M=10, d=256)
    assert _bwd(L, X8=_p(**x8)) == ESHAPE                                  # both inputs
    for bad, status in (({"M": 9}, ESHAPE), ({"d": 255}, ESHAPE), ({"codes": None}, ENULL), ({"scale": None}, ENULL),
                        ({"codes": 0x1004}, EALIGN), ({"scale": 0x2001}, EALIGN)):
        assert _bwd(L, X=None, X8=_p(**{**x8, **bad})) == status
    assert _bwd(L, dX=0x6000) == ESHAPE and _bwd(L, dX=0x5000) == ESHAPE   # over dY, over X
    assert _bwd(L, dX=None) == ESHAPE                                      # dX0 without dX
    need = L.qlora_adapters_workspace_bytes(1, _bank(), 10)
    assert need > 0 and _bwd(L, n=need - 1) == EWS and _bwd(L, pn=q.qlora_adapters_plan_bytes(10, 3) - 1) == EWS


def _lin(L, **kw):
    nf = kw.pop("q", _lib._Nf4(128, 256, 0x1000, 0x2000, 0x3000, 0x4000))
    a = dict(X8=_p(M=10, d=256), dY=0x6000, M=10, A=0x7000, B=0x8000, r=16, alpha=32.0, drop=None, T=0x9000, dX=0xA000, dA=0xB000,
             dB=0xC000, ws=0xD000, n=BIG)
    a.update(kw)
    return L.qlora_linear_bwd_packed(nf, *a.values(), None)


def test_packed_linear_refusals(L):
    assert _lin(L, M=-1) == ESHAPE and _lin(L, r=0) == ESHAPE and _lin(L, r=257) == ESHAPE
    for name in ("X8", "dY", "A", "B", "T", "dA", "dB", "ws"):
        assert _lin(L, **{name: None}) == ENULL
    for name in ("dY", "A", "T", "dX", "dA", "dB", "ws"):
        assert _lin(L, **{name: 0xE008}) == EALIGN
    for bad, status in (({"M": 9}, ESHAPE), ({"d": 128}, ESHAPE), ({"codes": None}, ENULL), ({"codes": 0x1001}, EALIGN), ({"scale": 0x2003}, EALIGN)):
        assert _lin(L, X8=_p(**{"M": 10, "d": 256, **bad})) == status
    assert _lin(L, dX=0x6000) == ESHAPE
    assert _lin(L, q=_lib._Nf4(128, 250, 0x1000, 0x2000, 0x3000, 0x4000)) == ESHAPE
    for p in (-0.1, 1.0, float("nan")):
        assert _lin(L, drop=_lib._Dropout(p, 1, 2, None, None)) == ESHAPE
    need = q.qlora_workspace_bytes(q.QLORA_OP_BWD_PACKED, 128, 256, 10, 16)
    more = q.qlora_workspace_bytes(q.QLORA_OP_BWD_PACKED_DROPOUT, 128, 256, 10, 16)
    assert 0 < need < more and _lin(L, n=need - 1) == EWS
    assert _lin(L, n=more - 1, drop=_lib._Dropout(0.1, 1, 2, None, None)) == EWS
    assert q.qlora_workspace_bytes(q.QLORA_OP_BWD_PACKED, 128, 250, 10, 16) == 0
    assert q.qlora_workspace_bytes(q.QLORA_OP_BWD_PACKED, 128, 256, 10, 300) == 0
    assert q.qlora_workspace_bytes(7, 128, 256, 10, 16) == 0


def test_bounds_of_the_plans_lists():
    """The lists' sizes that the host reserves hold what the device counts, for
    any distribution of the tokens (the device's counting, done here)."""
    import random
    rng = random.Random(3)
    cdiv = lambda a, b: -(-a // b)  # noqa: E731
    for _ in range(3000):
        M = int(round(2 ** rng.uniform(0, 21)))
        slots = int(round(2 ** rng.uniform(0, 11)))
        left, counts = M, []
        for _ in range(slots):
            take = min(left, int(rng.choice([0, 1, 63, 64, 65, rng.randint(0, 1 + left), rng.randint(0, 300)])))
            counts.append(take)
            left -= take
        tiles = cdiv(M, 64)
        tps = max(min(16, max(8, cdiv(tiles, 4))), cdiv(tiles, 64))
        t = [cdiv(c, 64) for c in counts]
        s = [cdiv(x, tps) for x in t]
        assert sum(t) + cdiv(left, 64) <= min(M, M // 64 + slots + 1)
        assert sum(s) <= min(M, M // (64 * tps) + slots)
        assert sum(x for x in s if x > 1) <= 2 * M // (64 * tps)


def test_binding_refuses_tensors_off_the_gpu():
    with pytest.raises(ValueError):
        q.Packed8.empty(2, 64, "cpu")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.qlora_pack8(x)
    with pytest.raises(ValueError):
        q.Packed8(4, 64, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(1, 4))
    with pytest.raises(ValueError):
        q.AdapterBank(torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 64, 8, dtype=torch.bfloat16), torch.ones(2))
    with pytest.raises(ValueError):
        q.qlora_adapters_plan(torch.zeros(4, dtype=torch.int32), 2)
