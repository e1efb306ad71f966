"""Which product makes the input gradient of the layer's backward from a checkpoint:
up to 64 tiles of 256 x 256, and for rows that are no whole vectors, the one for few
tokens (its partial sums are in the workspace), above the fused GEMM; and both
against the definition in 64 bits at either side of the border."""
import pytest
import torch

import adapters_ref as ref
import bit_quantized_lora_quantize_amd as q
from test_gpu_linear_packed import _exact, _layer


@pytest.mark.parametrize("M,d_in,d_out,few", [(900, 4096, 4096, True), (769, 4096, 4096, True), (1025, 4096, 4096, False),
                                              (900, 4352, 4096, False), (900, 4352, 4097, True), (3, 64, 512, True)])
def test_rule(M, d_in, d_out, few):
    """Two ranges of outputs or more leave 8 M d_in bytes of partial sums at least."""
    rest = 4 * 8 * M * 8 + 4 * M * 32 + 2 * 2 * -(-M // 64) * 3 * 1024 + 4 * -(-M // 512) * 8 * (d_in + d_out) + 12 * 256
    have = q.qlora_workspace_bytes(q.QLORA_OP_BWD_PACKED, d_out, d_in, M, 8)
    assert (have >= 8 * M * d_in) if few else (have <= rest), (have, rest)


@pytest.mark.gpu
@pytest.mark.parametrize("M,d_in,d_out,r", [(16384, 64, 64, 8), (16385, 64, 64, 8), (1024, 4096, 72, 16), (900, 4096, 264, 16), (1025, 4096, 72, 16)])
def test_either_side(M, d_in, d_out, r):
    w, X, dY, A, B = _layer(M + r, M, d_in, d_out, r)
    dev = torch.device("cuda:0")
    Xd, dYd, Ad, Bd = (t.to(dev) for t in (X, dY, A, B))
    T = torch.empty(M, r, device=dev)
    q.qlora_linear_fwd(w, Xd, Ad, Bd, 2.0 * r, T_save=T)
    X8 = q.qlora_pack8(Xd)
    dX, dA, dB = q.qlora_linear_bwd_packed(w, X8, dYd, Ad, Bd, 2.0 * r, T)
    want, bound = _exact(w, q.qlora_unpack8(X8), T, dY, A, B, 2.0)
    for name, got in (("dA", dA), ("dB", dB), ("dX", dX)):
        ref.inside(got, want[name], bound[name], name)
