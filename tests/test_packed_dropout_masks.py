"""A saved dropout mask of another batch, type or place is refused before the layer's
backward from a checkpoint: the kernels would read it past its end."""
import pytest
import torch

import bit_quantized_lora_quantize_amd as q


class OnGpu:
    """What the binding's checks see of a GPU tensor, where there is no GPU."""

    def __init__(self, dtype, *shape, at=0, contiguous=True):
        self.dtype, self.shape, self.at, self.contiguous = dtype, torch.Size(shape), at, contiguous
        self.device = f"cuda:{at}" if at >= 0 else "cpu"
        self.is_cuda = at >= 0

    def get_device(self):
        return self.at

    def is_contiguous(self):
        return self.contiguous


BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class Reached(Exception):
    pass


def _call(monkeypatch, M, rows, cols, d_in=128, d_out=64, r=8):
    x8 = q.Packed8.__new__(q.Packed8)
    x8.M, x8.d, x8.codes, x8.scale, x8.c = M, d_in, OnGpu(torch.int8, M, d_in), OnGpu(F32, d_in // 64, M), None
    w = q.NF4Weight(d_out, d_in, OnGpu(torch.uint8, d_out * d_in // 2), None, None, None)
    drop = q.Dropout(0.25, 1, 2, rows, cols)

    def stop(*a):
        raise Reached

    from bit_quantized_lora_quantize_amd import _adapters
    monkeypatch.setattr(_adapters, "_out", stop)   # the first allocation, behind every check
    q.qlora_linear_bwd_packed(w, x8, OnGpu(BF16, M, d_out), OnGpu(BF16, r, d_in), OnGpu(BF16, d_out, r), 16.0, OnGpu(F32, M, r), dropout=drop)


BAD = [("keep_rows", OnGpu(I32, 40, 4), OnGpu(I32, 128, 7)), ("keep_cols", OnGpu(I32, 200, 4), OnGpu(I32, 128, 2)),
       ("keep_rows", OnGpu(I32, 200, 2), OnGpu(I32, 128, 7)), ("keep_cols", OnGpu(I32, 200, 4), OnGpu(I32, 64, 7)),
       ("keep_rows", OnGpu(I32, 200, 4, at=-1), OnGpu(I32, 128, 7)), ("keep_cols", OnGpu(I32, 200, 4), OnGpu(I32, 128, 7, at=1)),
       ("keep_rows", OnGpu(torch.int8, 200, 4), OnGpu(I32, 128, 7)), ("keep_cols", OnGpu(I32, 200, 4), OnGpu(I32, 128, 7, contiguous=False))]


@pytest.mark.parametrize("name,rows,cols", BAD)
def test_refused(monkeypatch, name, rows, cols):
    with pytest.raises(ValueError, match=name):
        _call(monkeypatch, 200, rows, cols)


@pytest.mark.parametrize("M,rows,cols", [(200, OnGpu(I32, 200, 4), OnGpu(I32, 128, 7)), (200, None, None),
                                         (17, OnGpu(I32, 17, 4), OnGpu(I32, 128, 1)),
                                         (16, OnGpu(I32, 5, 4), OnGpu(I32, 128, 1)), (200, OnGpu(I32, 5, 4), None)])
def test_accepted(monkeypatch, M, rows, cols):
    """The call's own mask; and one that is not read (16 tokens or fewer, half of a pair)."""
    with pytest.raises(Reached):
        _call(monkeypatch, M, rows, cols)
