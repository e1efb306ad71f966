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


def test_row_strides_pairs_and_sequences_at_their_limits(L):
    l, far = _empty_batch(), 1 << 32
    assert L.qlora_token_logp(_empty_batch(ld=far), P(0x5000), None, None) == OK
    assert L.qlora_token_logp(_empty_batch(ld=far + 1), P(0x5000), None, None) == ESHAPE
    par = _train._Preference(0, 0, 0.1, 0.0, 0.0, 1.0)
    pref = lambda pairs: L.qlora_preference_loss(l, None, pairs, None, par, None, None, None, None,  # noqa: E731
                                                 0, None, 0, None)
    assert pref(1 << 20) == ENULL and pref((1 << 20) + 1) == ESHAPE
    pol = _train._Policy(0, 0, 0.2, 0.2, 0.0, 1.0)
    policy = lambda seqs: L.qlora_policy_loss(l, None, seqs, None, None, None, pol, None, None,  # noqa: E731
                                              None, 0, None, 0, None)
    assert policy(1 << 21) == ENULL and policy((1 << 21) + 1) == ESHAPE
    full = _train._Logits(0x1000, 0x2000, 4, 100, 100, -100, 0, 1.0)
    back = lambda ldd: L.qlora_token_logp_bwd(full, P(0x5000), P(0x6000), None if ldd <= far  # noqa: E731
                                              else P(0x7000), ldd, None)
    assert back(far) == ENULL and back(far + 1) == ESHAPE
    assert q.qlora_policy_workspace_bytes(0, 1 << 21) > 0
    assert q.qlora_policy_workspace_bytes(0, (1 << 21) + 1) == 0
    assert q.qlora_preference_workspace_bytes(1 << 21) > 0
    assert q.qlora_preference_workspace_bytes((1 << 21) + 1) == 0


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
    """A host tensor that says it is on a GPU, to reach the binding's checks."""
    is_cuda = True
    at = 0

    def get_device(self):
        return self.at


def _on(at, t):
    t = t.as_subclass(_OnGpu)
    t.at = at
    return t


def test_the_binding_refuses_a_buffer_for_the_sum_without_residual(L):
    x, g = _on(0, torch.zeros(4, 64)), _on(0, torch.ones(64))
    with pytest.raises(ValueError, match="residual"):
        q.qlora_norm_fwd(x, g, H=x)


def _calls():
    """Every entry point with all its tensors: (function, tensors by name)."""
    x, v, r = torch.zeros(4, 64), torch.ones(64), torch.zeros(4)
    t, off, d = torch.zeros(4, dtype=torch.int64), torch.tensor([0, 2, 4]), torch.zeros(4, 64)
    ws = torch.empty(1 << 16, dtype=torch.uint8)
    return [
        (q.qlora_norm_fwd, dict(X=x, gamma=v, beta=v.clone(), residual=x.clone(), H=d, Y=d.clone())),
        (q.qlora_norm_bwd, dict(dY=d, H=x, gamma=v, mean=r, rstd=r.clone(), dH=x.clone(),
                                dX=d.clone(), dgamma=v.clone(), dbeta=v.clone(), need_dbeta=True,
                                workspace=ws)),
        (q.qlora_token_logp, dict(logits=x, targets=t, logp=r, lse=r.clone())),
        (q.qlora_token_logp_bwd, dict(logits=x, targets=t, lse=r, dlogp=r.clone(), dlogits=d)),
        (q.qlora_preference_loss, dict(logits=x, targets=t, offsets=off, ref_logp=r, dlogits=d,
                                       workspace=ws)),
        (q.qlora_policy_loss, dict(logits=x, targets=t, offsets=off, advantages=torch.ones(2),
                                   old_logp=r, ref_logp=r.clone(), dlogits=d, workspace=ws))]


class _Recorder:
    """Stands in for the library: notes the current GPU and the stream."""

    def __init__(self, gpu):
        self.seen, self.gpu = [], gpu

    def __getattr__(self, name):
        def call(*args):
            self.seen.append((name, self.gpu[0], args[-1]))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    from bit_quantized_lora_quantize_amd import _lib
    gpu = [0]
    rec = _Recorder(gpu)

    class Device:
        def __init__(self, at):
            self.at = at

        def __enter__(self):
            self.before, gpu[0] = gpu[0], self.at

        def __exit__(self, *_):
            gpu[0] = self.before

    monkeypatch.setattr(_lib, "lib", lambda: rec)
    monkeypatch.setattr(_train, "_current_gpu", lambda: gpu[0])
    monkeypatch.setattr(_train, "_raw_stream", lambda at: 100 + at)
    monkeypatch.setattr(torch.cuda, "device", Device)
    return rec


@pytest.mark.parametrize("at", [0, 1])
def test_work_goes_to_the_tensors_gpu(fake, at):
    """The default stream has the same handle on every GPU: the tensors' one is
    current during the call, and only then."""
    for f, kw in _calls():
        fake.seen.clear()
        f(**{k: _on(at, v) if isinstance(v, torch.Tensor) else v for k, v in kw.items()})
        assert fake.seen[-1] == (f.__name__, at, 100 + at) and fake.gpu == [0]


def test_tensors_on_two_gpus_are_refused(fake):
    for f, kw in _calls():
        names = [k for k, v in kw.items() if isinstance(v, torch.Tensor)]
        for odd in names:
            with pytest.raises(ValueError):
                f(**{k: _on(int(k == odd), v) if k in names else v for k, v in kw.items()})
        assert not fake.seen
