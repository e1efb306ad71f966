"""The layer's backward from a checkpoint stays within a workspace of the size that
it asks for, whatever that memory held before."""
import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("M,d_in,d_out,r", [(1, 64, 64, 8), (16, 128, 77, 3), (40, 128, 96, 16), (333, 192, 520, 50), (700, 512, 257, 100),
                                            (2500, 128, 128, 16), (8200, 1024, 64, 16)])
@pytest.mark.parametrize("p", [None, 0.25])
def test_workspace(M, d_in, d_out, r, p):
    say(f"packed workspace {M} {d_in}->{d_out} r={r} p={p}")
    g = torch.Generator(device=DEV)
    g.manual_seed(M + r)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    w = q.qlora_quantize_nf4(rand(d_out, d_in) * 0.02)
    X8, dY = q.qlora_pack8(rand(M, d_in).bfloat16()), rand(M, d_out).bfloat16()
    A, B, T = rand(r, d_in).bfloat16(), rand(d_out, r).bfloat16(), rand(M, r)
    drop = None if p is None else q.Dropout(p, 3, 4)
    op = q.QLORA_OP_BWD_PACKED if p is None else q.QLORA_OP_BWD_PACKED_DROPOUT
    need = q.qlora_workspace_bytes(op, d_out, d_in, M, r)
    results = []
    for fill in (0, 0x77, 0xFF):
        room = torch.full((need + 4096,), fill, dtype=torch.uint8, device=DEV)
        results.append(q.qlora_linear_bwd_packed(w, X8, dY, A, B, 16.0, T, dropout=drop, workspace=room[:need]))
        assert bool((room[need:] == fill).all())
    for other in results[1:]:
        assert all(torch.equal(x, y) for x, y in zip(results[0], other))
    assert all(bool(t.isfinite().all()) for t in results[0])
