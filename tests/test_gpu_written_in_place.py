"""What a call writes into a tensor of the caller's is known to autograd: a backward pass that saved the old values refuses,
instead of using the new ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_backward_implicit_bwd_gb300 import build as cbuild
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train
    return train


def calls(T):
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    i = lambda *s: z(*s, d=torch.int32)  # noqa: E731
    e, p = T.Experts(2, 16, 8, "f32"), T.PolicyLoss(9, "f32")
    off, w, a, f = i(3), z(2, 8, 16), i(4), z(4)
    yield "forward", (4, 8), lambda t: e.forward(z(4, 16), w, off, out=t)
    yield "data", (4, 16), lambda t: e.backward_data(z(4, 8), w, off, out=t)
    yield "weight", (2, 8, 16), lambda t: e.backward_weight(z(4, 8), z(4, 16), off, out=t, accumulate=True)
    yield "clip in place", (7,), lambda t: T.GradClip.like([t]).clip([t], 1.0)
    yield "clip", (7,), lambda t: T.GradClip.like([t]).clip([z(7)], 1.0, out=[t])
    yield "policy backward", (4, 9), lambda t: p.backward(z(4, 9), a, f, f, out=t)
    yield "policy, out=logits", (4, 9), lambda t: p.forward_backward(t, a, f, f, out=t)


def test_versions(T):
    for what, shape, call in calls(T):
        t = torch.ones(shape, device="cuda")
        before = t._version
        call(t)
        assert t._version > before, what
        with torch.inference_mode():  # tensors that keep no version
            call(torch.ones(shape, device="cuda"))


def test_a_saved_tensor_that_was_overwritten(T):
    for what, shape, call in calls(T):
        x = torch.ones(shape, device="cuda", requires_grad=True)
        y = torch.exp(x)  # saves its result
        call(y.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_inputs_keep_theirs(T):
    p = T.PolicyLoss(9, "f32")
    z, a, f = torch.ones(4, 9, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
    p.forward_backward(z, a, f, f)
    T.GradClip.like([z]).norm([z])
    T.GradClip.like([z]).clip([z], 1.0, out=[torch.empty_like(z)])
    assert z._version == 0 and f._version == 0 and a._version == 0
