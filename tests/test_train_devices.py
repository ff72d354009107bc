"""Tensors that lie on another GPU than the plan's are refused before the library sees their addresses.  (No second GPU is
needed: the tensors only say that they lie there.)"""
import pytest
import torch

from conv2d_backward_implicit_bwd_gb300 import build as cbuild


class Elsewhere(torch.Tensor):
    """A tensor that calls itself one of cuda:1."""
    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        name = getattr(func, "__name__", "")
        if name == "get_device":
            return 1
        if name == "__get__" and getattr(func, "__self__", None) is torch.Tensor.is_cuda:
            return True
        return super().__torch_function__(func, types, args, kwargs or {})


def away(t):
    return t.as_subclass(Elsewhere)


def refused(T, device):
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device=device)  # noqa: E731
    i = lambda *s: z(*s, d=torch.int32)  # noqa: E731
    e = T.Experts(2, 16, 8, "f32")
    x, w, dy, off = z(4, 16), z(2, 8, 16), z(4, 8), i(3)
    yield "x", lambda: e.forward(away(x), w, off)
    c = T.GradClip.like([z(3), z(5)])
    yield r"grads\[0\]", lambda: c.norm([away(z(3)), away(z(5))])
    p = T.PolicyLoss(9, "f32")
    logits, a, f = z(4, 9), i(4), z(4)
    yield "logits", lambda: p.forward(away(logits), away(a), away(f), away(f))
    if device == "cpu":  # (a plan made without a device has none that its tensors could share)
        return
    yield "w", lambda: e.forward(x, away(w), off)
    yield "offsets", lambda: e.forward(x, w, away(off))
    yield "out", lambda: e.forward(x, w, off, out=away(z(4, 8)))
    yield "dy", lambda: e.backward_data(away(dy), w, off)
    yield "x", lambda: e.backward_weight(dy, away(x), off)
    yield "out", lambda: e.backward_weight(dy, x, off, out=away(z(2, 8, 16)))
    yield r"grads\[1\]", lambda: c.norm([z(3), away(z(5))])
    yield r"out\[0\]", lambda: c.clip([z(3), z(5)], 1.0, out=[away(z(3)), z(5)])
    yield "actions", lambda: p.forward(logits, away(a), f, f)
    yield "weight", lambda: p.forward_backward(logits, a, f, away(f))
    yield "ref_logp", lambda: p.forward(logits, a, f, f, ref_logp=away(f))
    yield "coef", lambda: p.backward(logits, a, f, away(f))
    yield "grad", lambda: p.backward(logits, a, f, f, grad=away(z(1)))
    yield "out", lambda: p.backward(logits, a, f, f, out=away(z(4, 9)))


def check(device):
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
    assert away(torch.zeros(2)).is_cuda and torch.Tensor.get_device(away(torch.zeros(2))) == 1
    for what, call in refused(T, device):
        with pytest.raises(ValueError, match=f"^{what}: "):
            call()


def test_refused_without_a_device():
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is there")
    check("cpu")


@pytest.mark.gpu
def test_refused_beside_the_plans_device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    check("cuda")
