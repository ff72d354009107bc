"""What create leaves on the GPU is there when it returns: a plan may run at once on a stream that is not ordered after
the default stream (every ``torch.cuda.Stream``).  On the CPU against a runtime that queues every copy and memset until its
stream is synchronised; on the GPU with the default stream kept busy."""
import os
import shutil
import subprocess

import pytest
import torch

from conv2d_backward_implicit_bwd_gb300 import build as cbuild

HERE = os.path.dirname(os.path.abspath(__file__))


def compiled(tmp, source, *flags):
    """The test's program with one file of the library; the launches and events that create does not reach all end in one place."""
    cxx, nm = shutil.which("g++"), shutil.which("nm")
    if not cxx or not nm:
        pytest.skip("no C++ compiler")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cbuild.nvcc()))), "include")

    def call(*args):
        r = subprocess.run(args, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout
    names = {}
    for src in (os.path.join(HERE, "plan_memory.cpp"), os.path.join(cbuild.CSRC, source)):
        obj = str(tmp / (os.path.basename(src) + ".o"))
        call(cxx, "-std=c++17", "-O1", *flags, "-I", include, "-c", src, "-o", obj)
        names[obj] = [line.split()[-2:] for line in call(nm, obj).splitlines()]
    defined = {n for table in names.values() for kind, n in table if kind != "U"}
    rest = {n for table in names.values() for kind, n in table if kind == "U" and n.startswith(("_ZN3cbd", "cuda"))} - defined
    exe = str(tmp / "plan_memory")
    call(cxx, *names, "-o", exe, *(f"-Wl,--defsym={n}=not_reached" for n in sorted(rest)), "-ldl", "-lpthread")
    return exe


def run(exe, what):
    r = subprocess.run([exe, what], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr


@pytest.fixture(scope="module")
def train(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("train"), "train_capi.cpp", "-DTRAIN")


@pytest.mark.parametrize("what", ["experts", "clip", "policy"])
def test_training_plans_are_ready_when_made(train, what):
    run(train, what)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["experts", "clip", "policy"])
def test_new_plan_on_an_unordered_stream(what):
    """Made while the default stream is busy, run at once on another: the results of a plan made in quiet, bit for bit."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if what == "experts":  # one tile with its rows split over many blocks, which count their arrivals
        dy, x, o = normal(3000, 40), normal(3000, 50), torch.tensor([0, 3000], dtype=torch.int32, device="cuda")
        make, call = lambda: T.Experts(1, 50, 40, "f32"), lambda p, s: [p.backward_weight(dy, x, o, stream=s)]
    elif what == "clip":
        grads = [normal(70_000), normal(9).bfloat16(), normal(1_000_003)]
        out = [torch.zeros_like(t) for t in grads]
        make, call = lambda: T.GradClip.like(grads), lambda p, s: [*p.clip(grads, 1.0, out=out, stream=s), *out]
    else:
        z, a = normal(2000, 100), torch.randint(0, 100, (2000,), generator=g, device="cuda", dtype=torch.int32)
        adv, w = normal(2000), torch.full((2000,), 1 / 2000, device="cuda")
        make, call = lambda: T.PolicyLoss(100, "f32"), lambda p, s: p.forward(z, a, adv, w, stream=s)
    quiet = make()
    want = [t.clone() for t in call(quiet, None)]
    streams, kept = [torch.cuda.Stream() for _ in range(3)], []  # (freeing a plan would wait for the default stream)
    torch.cuda.synchronize()
    for s in streams:
        torch.cuda._sleep(100_000_000)  # some 50 ms of the default stream
        plan = make()
        kept.append(plan)
        got = call(plan, s)
        got = call(plan, s)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert plan.status(stream=s) == (0, 0)
        torch.cuda.synchronize()


@pytest.fixture(scope="module")
def conv(tmp_path_factory):
    return compiled(tmp_path_factory.mktemp("conv"), "capi.cpp")


@pytest.mark.parametrize("what", ["status", "split", "streamk"])
def test_convolution_plans_are_ready_when_made(conv, what):
    run(conv, what)


@pytest.mark.gpu
def test_new_convolution_plan_on_an_unordered_stream():
    """A contraction split over SM pairs, whose flags create clears: the same bits as a plan made in quiet."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import binding as B
    make = lambda: B.Plan(32, 512, 512, 28, 28, 3, 3, pad=(1, 1), stride=(2, 2), dil=(2, 2), layout="nhwc", dtype="bf16")  # noqa: E731
    plan = make()
    assert plan.k_splits() > 1
    g = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randn(32, plan.Ho, plan.Wo, 512, generator=g, device="cuda").bfloat16()
    w = torch.randn(512, 3, 3, 512, generator=g, device="cuda").bfloat16()
    want, dx = (torch.empty(32, 28, 28, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    plan.run(dy, w, want)
    assert torch.isfinite(want).all() and plan.status() == (0, 0)
    streams, kept = [torch.cuda.Stream() for _ in range(3)], []  # (freeing a plan would wait for the default stream)
    torch.cuda.synchronize()
    for s in streams:
        torch.cuda._sleep(100_000_000)
        plan = make()
        kept.append(plan)
        plan.run(dy, w, dx, stream=s)
        plan.run(dy, w, dx, stream=s)
        s.synchronize()
        assert torch.equal(dx, want) and plan.status(stream=s) == (0, 0)
        torch.cuda.synchronize()
        dx.zero_()
        torch.cuda.synchronize()
