"""Host checks at the limits of the norms' and losses' arguments, and of the
binding's tensors (no GPU: batches without rows, fake tensors)."""
import ctypes

import pytest
import torch

import bit_quantized_lora_quantize_amd as q
from bit_quantized_lora_quantize_amd import _train

OK, ENULL, ESHAPE = 0, -1, -2
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    import os
    from bit_quantized_lora_quantize_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return q.lib()


def _empty_batch(**kw):
    a = dict(logits=None, targets=None, rows=0, vocab=100, ld=100, ignore_index=-100, type=0,
             scale=1.0)
    a.update(kw)
    return _train._Logits(*a.values())


@pytest.mark.parametrize("scale,status", [(2.0 ** 126, OK), (2.0 ** 126 * 1.25, ESHAPE),
                                          (3e38, ESHAPE), (1e-38, OK), (1e-45, OK)])
def test_scales_whose_base_2_form_overflows_are_refused(L, scale, status):
    """The kernels work with scale * log2(e): past the FP32 range it would turn
    the largest logit's own term, exp(0), into a NaN."""
    l = _empty_batch(scale=scale)
    assert L.qlora_token_logp(l, P(0x5000), P(0x6000), None) == status
    assert L.qlora_token_logp_bwd(l, P(0x5000), P(0x6000), P(0x7000), 100, None) == status
    par = _train._Preference(0, 0, 0.1, 0.0, 0.0, 1.0)
    assert L.qlora_preference_loss(l, None, 0, None, par, None, None, None, None, 0, None, 0,
                                   None) == status
    pol = _train._Policy(0, 0, 0.2, 0.2, 0.0, -1.0)
    want = ENULL if status == OK else status       # an empty batch still writes its averages
    assert L.qlora_policy_loss(l, None, 0, None, None, None, pol, None, None, None, 0, None, 0,
                               None) == want


def test_a_norm_without_residual_takes_no_buffer_for_the_sum(L):
    """H without a residual would stay unwritten: refused, not ignored."""
    call = lambda M, R, H: L.qlora_norm_fwd(0, 1, P(0x1000), R, M, 64, 1, P(0x2000), None, 1e-5,  # noqa: E731
                                            H, P(0x3000), None, None, None)
    assert call(0, None, None) == OK and call(0, P(0x4000), P(0x5000)) == OK
    assert call(0, None, P(0x5000)) == ESHAPE and call(4, None, P(0x5000)) == ESHAPE


class _OnGpu(torch.Tensor):
    """A host tensor that says it is on GPU 0, to reach the binding's checks."""
    is_cuda = True

    def get_device(self):
        return 0


def test_the_binding_refuses_a_buffer_for_the_sum_without_residual(L):
    x, g = (t.as_subclass(_OnGpu) for t in (torch.zeros(4, 64), torch.ones(64)))
    with pytest.raises(ValueError, match="residual"):
        q.qlora_norm_fwd(x, g, H=x)
