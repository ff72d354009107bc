"""Where the training-step operators' results are allocated: on the tensors' device, and seen by dispatch modes."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from conv2d_backward_implicit_bwd_gb300 import build as cbuild


@pytest.fixture
def T():
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train
    return train


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.new = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func.name() == "aten::empty.memory_format":
            self.new.append(tuple(out.shape))
        return out


@pytest.fixture
def calls(T, monkeypatch):
    """Both ways of allocation, as names of what was called, without a GPU; cuda:0 is current."""
    seen = []
    monkeypatch.setattr(T, "_new", lambda shape, stride, dtype: seen.append(("own", shape, stride)) or "own")
    monkeypatch.setattr(T, "_current", lambda: 0)
    monkeypatch.setattr(T.torch, "empty", lambda shape, dtype, device: seen.append(("usual", shape, torch.device(device))) or "usual")
    return seen


HERE, THERE = torch.device("cuda", 0), torch.device("cuda", 1)


def test_another_device_than_the_current_one(T, calls):
    assert T._outputs(HERE, None)((4, 3), torch.float32) == "own" and calls == [("own", (4, 3), (3, 1))]
    assert T._outputs(THERE, None)((4,), torch.float32) == "usual" and calls[1] == ("usual", (4,), THERE)
    for device in (HERE, THERE):
        assert T._empty((2, 3), torch.float32, device, None) == "usual" and calls[-1] == ("usual", (2, 3), device)


def test_other_arguments(T, calls, monkeypatch):
    def wants_more(shape, stride, dtype, more):
        pass
    monkeypatch.setattr(T, "_new", wants_more)
    assert T._outputs(HERE, None)((4,), torch.float32) == "usual"


def test_under_a_mode(T, calls):
    with Seen():
        assert T._outputs(HERE, None)((4,), torch.float32) == "usual"
    assert T._outputs(HERE, None)((4,), torch.float32) == "own"


@pytest.mark.gpu
def test_modes_see_the_results(T):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    z, a = torch.randn(6, 50, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    plan = T.TokenLogp(50, "f32", top=3)
    want = plan.forward(z, a)
    with Seen() as seen:
        got = plan.forward(z, a)
        dz = plan.backward(z, a, got[2], grad_logp=torch.ones(6, device="cuda"))
    assert sorted(seen.new) == [(6,), (6,), (6,), (6, 3), (6, 3), (6, 50)]
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and dz.shape == (6, 50)
    with torch.inference_mode():
        assert all(t.is_inference() for t in plan.forward(z, a))
