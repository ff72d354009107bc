"""Plans of the token log-probabilities and the orthogonalised updates: on the CPU against a runtime that queues every copy
until its stream is synchronised; and tensors that lie on another GPU than the plan's are refused."""
import os
import shutil
import subprocess

import pytest
import torch
from test_train_devices import away

from conv2d_backward_implicit_bwd_gb300 import build as cbuild

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    """The test's program with the library's plan code; what create does not reach ends in one place."""
    tmp = tmp_path_factory.mktemp("plans")
    cxx, nm = shutil.which("g++"), shutil.which("nm")
    if not cxx or not nm:
        pytest.skip("no C++ compiler")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cbuild.nvcc()))), "include")

    def call(*args):
        r = subprocess.run(args, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout
    names = {}
    for src in (os.path.join(HERE, "more_plan_memory.cpp"), os.path.join(cbuild.CSRC, "train_capi.cpp")):
        obj = str(tmp / (os.path.basename(src) + ".o"))
        call(cxx, "-std=c++17", "-O1", "-DTRAIN", "-I", include, "-c", src, "-o", obj)
        names[obj] = [line.split()[-2:] for line in call(nm, obj).splitlines()]
    defined = {n for table in names.values() for kind, n in table if kind != "U"}
    rest = {n for table in names.values() for kind, n in table if kind == "U" and n.startswith(("_ZN3cbd", "cuda"))} - defined
    exe = str(tmp / "plans")
    call(cxx, *names, "-o", exe, *(f"-Wl,--defsym={n}=not_reached" for n in sorted(rest)), "-ldl", "-lpthread")
    return exe


@pytest.mark.parametrize("what", ["logp", "orth small", "orth", "orth batch"])
def test_plans_are_ready_when_made(program, what):
    r = subprocess.run([program, what], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def refused(T, device):
    z = lambda *s, d=torch.float32: torch.zeros(*s, dtype=d, device=device)  # noqa: E731
    i = lambda *s: z(*s, d=torch.int32)  # noqa: E731
    p, o = T.TokenLogp(9, "f32", top=2), T.Orthogonal(2, 5, 7, "f32")
    yield "logits", lambda: p.forward(away(z(4, 9)), away(i(4)))
    yield "x", lambda: o.apply(away(z(2, 5, 7)))
    yield "grad", lambda: o.update(z(2, 5, 7), away(z(2, 5, 7)), z(2, 5, 7), 0.1)
    if device == "cpu":  # (a plan made without a device has none that its tensors could share)
        return
    f = z(4)
    yield "tokens", lambda: p.forward(z(4, 9), away(i(4)))
    yield "lse", lambda: p.backward(z(4, 9), i(4), away(f), f, grad_logp=f)
    yield "entropy", lambda: p.backward(z(4, 9), i(4), f, away(f), grad_entropy=f)
    yield "grad_logp", lambda: p.backward(z(4, 9), i(4), f, f, grad_logp=away(f))
    yield "grad_entropy", lambda: p.backward(z(4, 9), i(4), f, f, grad_entropy=away(f))
    yield "out", lambda: p.backward(z(4, 9), i(4), f, f, grad_logp=f, out=away(z(4, 9)))
    yield "out", lambda: o.apply(z(2, 5, 7), out=away(z(2, 5, 7)))
    yield "weight", lambda: o.update(away(z(2, 5, 7)), z(2, 5, 7), z(2, 5, 7), 0.1)
    yield "momentum", lambda: o.update(z(2, 5, 7), z(2, 5, 7), away(z(2, 5, 7)), 0.1)
    yield "copy", lambda: o.update(z(2, 5, 7), z(2, 5, 7), z(2, 5, 7), 0.1, copy=away(z(2, 5, 7, d=torch.bfloat16)))
    # shapes, types, layouts
    yield "tokens", lambda: p.forward(z(4, 9), i(5))
    yield "tokens", lambda: p.forward(z(4, 9), i(4).long())
    yield "logits", lambda: p.forward(z(9, 4).t(), i(4))
    yield "out", lambda: p.backward(z(4, 9), i(4), f, f, grad_logp=f, out=z(5, 9))
    yield "x", lambda: o.apply(z(2, 7, 5).transpose(1, 2))
    yield "x", lambda: o.apply(z(1, 5, 7).expand(2, 5, 7))
    yield "x", lambda: o.apply(z(2, 5, 7).bfloat16())
    yield "weight", lambda: o.update(z(2, 5, 8)[:, :, :7], z(2, 5, 7), z(2, 5, 7), 0.1)
    yield "copy", lambda: o.update(z(2, 5, 7), z(2, 5, 7), z(2, 5, 7), 0.1, copy=z(2, 5, 7))


def check(device):
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
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
