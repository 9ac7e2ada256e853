"""The torch functions of the operators up to the library call, no GPU: torch's fake
tensors stand for CUDA ones, and the library's launching calls are recorded with the
device that was current, not made."""
import contextlib

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from tensor_adamw_optimizer_amd import _lib as L
from tensor_adamw_optimizer_amd import ops

LAUNCHING = ("apexw_gated_ffn_forward", "apexw_gated_ffn_backward", "apexw_linear_xent_forward",
             "apexw_linear_xent_backward", "apexw_qk_norm_rope_forward",
             "apexw_qk_norm_rope_backward")


@pytest.fixture
def calls(monkeypatch):
    """What is queued: (entry point, current device, arguments).  Device 0 is
    current, raw streams are 100 + the device's number."""
    made, current = [], [0]

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], torch.device(d).index if not isinstance(d, int) else d
        try:
            yield
        finally:
            current[0] = before

    def entry(name):
        return lambda *a: made.append((name, current[0], a))

    for name in LAUNCHING:
        monkeypatch.setattr(L, name, entry(name))
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(ops, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.Tensor, "data_ptr", lambda t: 1 << 20)
    monkeypatch.setattr(ops, "_plans", {})
    monkeypatch.setattr(ops, "_elements", {})
    with FakeTensorMode():
        yield made


def _ffn(dev, **kw):
    return [torch.empty(*s, device=dev, **kw) for s in ((3, 8), (16, 8), (16, 8), (8, 16))]


def _xent(dev):
    return (torch.empty(3, 8, device=dev), torch.empty(16, 8, device=dev),
            torch.empty(3, dtype=torch.int64, device=dev))


def _qk(dev):
    w = torch.empty(8, device=dev)
    return (torch.empty(3, 4, 8, device=dev), torch.empty(3, 2, 8, device=dev), w, w,
            torch.empty(3, dtype=torch.int64, device=dev))


def _each(dev):
    """Every entry point once, and the functions that stand on them."""
    f, x, k = _ffn(dev), _xent(dev), _qk(dev)
    ops.gated_ffn_forward(*f)
    ops.gated_ffn_backward(f[0], *f)
    ops.linear_cross_entropy_forward(*x)
    ops.linear_cross_entropy_backward(*x, torch.empty(3, device=dev), torch.empty((), device=dev))
    ops.qk_norm_rope_forward(*k)
    ops.qk_norm_rope_backward(k[0], k[1], *k)
    ops.gated_ffn(*f)
    ops.linear_cross_entropy(*x)
    ops.qk_norm_rope(*k)


@pytest.mark.parametrize("index", [0, 1, 3])
def test_the_tensors_device_is_current_for_each_call(calls, index):
    """A raw stream, and the default one, 0, above all, is taken as one of the
    thread's current device: each call is made with the tensors' device current,
    on that device's stream, and the thread's own device is current again after."""
    _each(torch.device("cuda", index))
    assert {name for name, _, _ in calls} == set(LAUNCHING) and len(calls) == 9
    for name, device, args in calls:
        assert device == index, name
        assert args[-1] == 100 + index, name
    assert torch.cuda.current_device() == 0


def _kept(calls):
    """The kept buffers' places that the forward passes were given."""
    return [args[6] for name, _, args in calls if name == "apexw_gated_ffn_forward"]


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_nothing_is_kept_where_no_backward_pass_can_follow(calls, mode):
    """Weights of a model require gradients in evaluation and decoding too."""
    f = [torch.nn.Parameter(t) for t in _ffn("cuda:0")]
    with mode():
        assert not ops.gated_ffn(*f).requires_grad
    assert not ops.gated_ffn(*(t.detach() for t in f)).requires_grad
    assert _kept(calls) == [0, 0]


@pytest.mark.parametrize("i", range(4))
def test_the_buffer_is_kept_where_a_gradient_is_asked_for(calls, i):
    f = _ffn("cuda:0")
    f[i].requires_grad_()
    assert ops.gated_ffn(*f).requires_grad and _kept(calls) == [1 << 20]


def test_a_kept_buffer_that_is_not_the_forward_passs_is_refused(calls):
    """Its address goes to the GPU as it is: a host tensor's would be read there."""
    f = _ffn("cuda:0")
    _, kept = ops.gated_ffn_forward(*f, keep=True)
    n = kept.numel()
    wrong = (torch.empty(n, dtype=torch.uint8),                            # on the host
             torch.empty(n, dtype=torch.uint8, device="cuda:1"),
             torch.empty(n, dtype=torch.float32, device="cuda:0"),
             torch.empty(n - 256, dtype=torch.uint8, device="cuda:0"),
             torch.empty(n + 256, dtype=torch.uint8, device="cuda:0"),     # of more tokens
             torch.empty(2 * n, dtype=torch.uint8, device="cuda:0")[::2])
    made = len(calls)
    for k in wrong:
        with pytest.raises(ValueError, match="kept"):
            ops.gated_ffn_backward(f[0], *f, kept=k)
    assert len(calls) == made
    ops.gated_ffn_backward(f[0], *f, kept=kept)
    assert calls[-1][0] == "apexw_gated_ffn_backward" and calls[-1][2][6:8] == (1 << 20, n)
