"""Split tiles of the orthogonalised updates: every matrix of a batch has places of its own in the workspace.  (One may be in X's product
while another is still in a square, and a place that tiles of both have would count and hold pieces of either.)"""
import os
import shutil
import subprocess

import pytest
import torch

from conv2d_backward_implicit_bwd_gb300 import build as cbuild

HERE = os.path.dirname(os.path.abspath(__file__))


def test_places_are_apart(tmp_path):
    """The library's plans, on a host runtime."""
    cxx, nm = shutil.which("g++"), shutil.which("nm")
    if not cxx or not nm:
        pytest.skip("no C++ compiler")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cbuild.nvcc()))), "include")

    def call(*args):
        r = subprocess.run(args, capture_output=True, text=True)
        assert r.returncode == 0, r.stdout + r.stderr
        return r.stdout
    names = {}
    for src in (os.path.join(HERE, "orth_places.cpp"), os.path.join(cbuild.CSRC, "train_capi.cpp")):
        obj = str(tmp_path / (os.path.basename(src) + ".o"))
        call(cxx, "-std=c++17", "-O1", "-DTRAIN", "-I", include, "-c", src, "-o", obj)
        names[obj] = [line.split()[-2:] for line in call(nm, obj).splitlines()]
    defined = {n for table in names.values() for kind, n in table if kind != "U"}
    rest = {n for table in names.values() for kind, n in table if kind == "U" and n.startswith(("_ZN3cbd", "cuda"))} - defined
    exe = str(tmp_path / "places")
    call(cxx, *names, "-o", exe, *(f"-Wl,--defsym={n}=not_reached" for n in sorted(rest)), "-ldl", "-lpthread")
    call(exe)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 768, 768), (2, 705, 740), (2, 767, 706)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_matrices_whose_products_are_split_differently(shape, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_orth import COEF, DT, check, iterate, matrices
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
    u = matrices(shape, dtype=DT[dtype])
    plan = T.Orthogonal(*shape, dtype)
    first = plan.apply(u)
    check(first, *iterate(u, [COEF] * 5))
    for _ in range(50):
        assert torch.equal(first, plan.apply(u))
    assert plan.status() == (0, 0)
