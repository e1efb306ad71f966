"""The workspace of the layer's backward from a checkpoint holds what that backward
uses, counted here from the operation, and nothing of the BF16 backward's."""
import random

import pytest

import bit_quantized_lora_quantize_amd as q

cdiv = lambda a, b: -(-a // b)  # noqa: E731


def _used(d_out, d_in, M, r, dropout):
    """Bytes of U's partial sums (at most 8 ranges), U as hi and lo, the contractions' operands (three terms of U and T
    for whole tiles of 64 tokens), their splits' results, the few-token input gradient's ranges (at most 8), mask words."""
    tiles = cdiv(M, 64)
    ranges = max(1, min(cdiv(1024, max(1, tiles)), cdiv(d_out, 256), 8))
    blocks = next(b for b in (1, 2, 4, 8, 16) if r <= 16 * b)
    tps = max(min(16, max(8, cdiv(max(tiles, 1), 4))), cdiv(max(tiles, 1), 64))
    splits = cdiv(tiles, tps)
    n = 4 * ranges * M * r + 4 * M * cdiv(r, 32) * 32 + 2 * 2 * tiles * 3 * blocks * 1024
    n += 4 * (splits if splits > 1 else 0) * r * (d_in + d_out)
    if d_out % 8 or cdiv(M, 256) * cdiv(d_in, 256) <= 64:
        parts = max(1, min(cdiv(1024, max(1, tiles * (d_in // 64))), cdiv(d_out, 128), 8))
        n += 4 * (parts if parts > 1 else 0) * M * d_in
    if dropout:
        n += 4 * M * (d_in // 32) + 4 * d_in * cdiv(max(M, 1), 32)
    return n


def _check(d_out, d_in, M, r):
    for op, dropout in ((q.QLORA_OP_BWD_PACKED, False), (q.QLORA_OP_BWD_PACKED_DROPOUT, True)):
        have, used = q.qlora_workspace_bytes(op, d_out, d_in, M, r), _used(d_out, d_in, M, r, dropout)
        assert have <= used + 12 * 256, (d_out, d_in, M, r, dropout, have, used)


@pytest.mark.parametrize("d_out,d_in,M,r", [(11008, 4096, 8192, 64), (4096, 4096, 2048, 64), (4096, 4096, 1, 16), (77, 128, 16, 3),
                                            (4096, 11008, 17, 256), (64, 64, 0, 8), (4099, 4096, 1 << 17, 8), (1, 64, 1 << 21, 256)])
def test_nothing_is_reserved_in_vain(d_out, d_in, M, r):
    _check(d_out, d_in, M, r)


def test_at_random_sizes():
    rng = random.Random(5)
    for _ in range(2000):
        _check(int(2 ** rng.uniform(0, 14)), 64 * int(2 ** rng.uniform(0, 8)), int(2 ** rng.uniform(0, 18)), int(2 ** rng.uniform(0, 8)))


def test_less_than_the_checkpoint_saves_next_to_the_bf16_backward():
    """8192 tokens, 4096 to 11008, rank 64: the inputs in 8 bits save 31 MB, and the workspace takes less than that more
    than the BF16 backward's."""
    M, d_in, d_out, r = 8192, 4096, 11008, 64
    saved = 2 * M * d_in - sum(q.qlora_pack8_sizes(M, d_in))
    more = q.qlora_workspace_bytes(q.QLORA_OP_BWD_PACKED, d_out, d_in, M, r) - q.qlora_workspace_bytes(q.QLORA_OP_BWD, d_out, d_in, M, r)
    assert more < saved
