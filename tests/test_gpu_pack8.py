"""Activations in 8 bits on the GPU: codes, scales and restored values bit for
bit against their definition."""
import pytest
import torch

import adapters_ref as ref
import bit_quantized_lora_quantize_amd as q
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TYPES = [torch.bfloat16, torch.float32]


def _check(X, note=""):
    p = q.qlora_pack8(X)
    codes, scale, restored = ref.pack(X)
    assert torch.equal(p.codes.cpu().long(), codes), f"codes {note}"
    assert torch.equal(p.scale.cpu().view(torch.int32), scale.view(torch.int32)) or \
        torch.equal(torch.nan_to_num(p.scale.cpu(), -1.0), torch.nan_to_num(scale, -1.0)), f"scales {note}"
    for dt in TYPES:
        got = q.qlora_unpack8(p, dt).cpu()
        want = restored.to(dt)
        assert got.shape == X.shape and got.dtype == dt
        assert torch.equal(torch.nan_to_num(got.float(), 12345.0), torch.nan_to_num(want.float(), 12345.0)), \
            f"restored {dt} {note}"
    return p


def _draw(seed, M, d, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, d, generator=g) * std
    x[:, :: max(1, d // 3)] *= 20.0
    return x.to(dtype)


@pytest.mark.parametrize("M,d", [(1, 1), (1, 63), (3, 64), (2, 65), (7, 128), (8, 100), (9, 255), (17, 256), (33, 257),
                                 (70, 1000), (5, 4096), (300, 517)])
@pytest.mark.parametrize("dtype", TYPES)
def test_pack_matches_definition(M, d, dtype):
    say(f"pack {M}x{d} {dtype}")
    _check(_draw(M * 1000 + d, M, d, dtype).to(DEV))


@pytest.mark.parametrize("dtype", TYPES)
def test_no_rows(dtype):
    p = q.qlora_pack8(torch.empty(0, 100, dtype=dtype, device=DEV))
    assert p.codes.shape == (0, 128) and q.qlora_unpack8(p, dtype).shape == (0, 100)


@pytest.mark.parametrize("dtype", TYPES)
def test_ties_go_to_even(dtype):
    """127 x / a = k + 1/2 exactly: a / 2 (63.5) in blocks of any a, and every half
    where a = 127 times a power of two."""
    tops = torch.tensor([1.0, 1.5, 127.0, 254.0, 3.0e-5, 7.0e20, 0.9921875]).to(dtype).float()
    X = torch.zeros(len(tops), 128)
    for i, a in enumerate(tops.tolist()):
        X[i, 0], X[i, 1], X[i, 2] = a, a / 2, -a / 2
        X[i, 64], X[i, 65] = -a, a / 2
        if a in (127.0, 254.0):
            k = torch.arange(-60, 60, dtype=torch.float32)[:60]
            X[i, 3:63] = (k + 0.5) * a / 127.0
    X = X.to(dtype)
    p = _check(X.to(DEV))
    assert (p.codes[:, 1] == 64).all() and (p.codes[:, 2] == -64).all()   # 63.5 to even


def test_next_to_a_border():
    """FP32 values a step beside a border fall to their own side."""
    g = torch.Generator().manual_seed(5)
    a = torch.rand(400, 1, generator=g) * 3 + 0.01
    k = torch.randint(0, 126, (400, 63), generator=g)
    b = ((k.double() + 0.5) * a.double() / 127.0).float()
    for step in (-1, 0, 1):
        x = (b.view(torch.int32) + step).view(torch.float32)
        _check(torch.cat([a, x], 1).to(DEV), f"step {step}")


@pytest.mark.parametrize("dtype", TYPES)
def test_extremes(dtype):
    """The smallest and largest values, zeros, and blocks with no number in them:
    these restore as NaN, their neighbours are untouched."""
    X = _draw(3, 12, 200, dtype).float()
    X[0] = 0.0
    X[1, :64] = 0.0
    X[2, :64] *= 2.0 ** -130          # below 2^-119: zeros
    X[3, 64:128] *= 2.0 ** -110
    X[4, 3] = float("inf")
    X[5, 70] = float("-inf")
    X[6, 199] = float("nan")
    X[7, 5] = torch.finfo(dtype).max
    X[8, :64] = torch.finfo(dtype).max
    X[9, :64] = 2.0 ** -119
    X[10, :64] = -0.0
    X = X.to(dtype)
    p = _check(X.to(DEV))
    r = q.qlora_unpack8(p, torch.float32).cpu()
    assert r[4, :64].isnan().all() and r[4, 64:].isfinite().all()
    assert r[5, 64:128].isnan().all() and r[6, 192:].isnan().all() and r[6, :192].isfinite().all()
    assert r[7:9].isfinite().all()
    assert (r[2, :64] == 0).all() and (r[9, :64] != 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_rows_off_alignment_and_untouched_surroundings(dtype):
    """X starts one element into its storage; what lies around the outputs stays."""
    M, d = 11, 133
    store = torch.zeros(M * d + 5, dtype=dtype, device=DEV)
    X = store[1:1 + M * d].view(M, d)
    X.copy_(_draw(9, M, d, dtype))
    p = _check(X)
    out = torch.full((M * d + 9,), 7.0, dtype=dtype, device=DEV)
    q.qlora_unpack8(p, dtype, out=out[3:3 + M * d].view(M, d))
    assert (out[:3] == 7).all() and (out[3 + M * d:] == 7).all()
    assert torch.equal(out[3:3 + M * d].view(M, d), q.qlora_unpack8(p, dtype))


def test_error_of_a_checkpoint():
    """Within half a step of a / 127, and BF16's rounding of the restored value."""
    X = _draw(11, 257, 1024, torch.bfloat16)
    r = q.qlora_unpack8(q.qlora_pack8(X.to(DEV))).cpu().double()
    a = X.double().abs().view(257, 16, 64).amax(2, keepdim=True)
    d = (r - X.double()).abs().view(257, 16, 64)
    assert (d <= a / 254 * 1.0001 + 2.0 ** -8 * r.abs().view(257, 16, 64)).all()


def test_large_offsets():
    """Rows past 2^31 elements of X: the last ones as they are alone."""
    M, d = 70000, 32000
    X = torch.empty(M, d, dtype=torch.bfloat16, device=DEV)
    X.fill_(1.0)
    tail = _draw(13, 5, d, torch.bfloat16).to(DEV)
    X[-5:] = tail
    p, alone = q.qlora_pack8(X), q.qlora_pack8(tail)
    assert torch.equal(p.codes[-5:], alone.codes) and torch.equal(p.scale[:, -5:].contiguous(), alone.scale)
    X.zero_()
    q.qlora_unpack8(p, out=X)
    assert torch.equal(X[-5:], q.qlora_unpack8(alone)) and bool((X[:1000] == 1).all())
