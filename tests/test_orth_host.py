"""Refusals of the orthogonalised updates (no GPU): descriptors, arguments, tensors."""
import ctypes

import pytest
import torch

from conv2d_backward_implicit_bwd_gb300 import build as cbuild


@pytest.fixture(scope="module")
def T():
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train
    return train


def status_of(f):
    from conv2d_backward_implicit_bwd_gb300.binding import ConvBwdError
    with pytest.raises(ConvBwdError) as e:
        f()
    return e.value.status


@pytest.mark.parametrize("args,kw,status", [
    ((0, 8, 8), {}, 1), ((1, 0, 8), {}, 1), ((1, 8, -3), {}, 1), ((1, 8, 8), dict(steps=0), 1), ((1, 8, 8), dict(coefficients=(33.0, 0, 0)), 1),
    ((1, 8, 8), dict(coefficients=(1.0, float("nan"), 0)), 1), ((1, 8, 8), dict(coefficients=(1.0, 0, float("inf"))), 1), ((65536, 1, 1), {}, 2),
    ((1, 65537, 1), {}, 2), ((1, 1, 65537), {}, 2), ((5, 65536, 65536), {}, 2), ((1, 8, 8), dict(steps=65), 2)])
def test_descriptor(T, args, kw, status):
    assert status_of(lambda: T.Orthogonal(*args, **kw)) == status


def test_coefficients(T):
    T.Orthogonal(1, 8, 8, steps=2, coefficients=[(1, 2, 3), (3, 2, 1)])
    for c in ([(1, 2, 3)], (1.0, 2.0), [(1, 2), (3, 4)], []):
        with pytest.raises(ValueError):
            T.Orthogonal(1, 8, 8, steps=2, coefficients=c)


def test_unknown(T):
    with pytest.raises(ValueError):
        T.Orthogonal(1, 8, 8, "f16")
    h, c = ctypes.c_void_p(), (ctypes.c_float * 3)(1, 0, 0)
    create = T._lib.conv_bwd_orth_create
    assert create(ctypes.byref(T.OrthDesc(1, 8, 8, 7, 1, c)), ctypes.byref(h)) == 1 and not h.value
    assert create(ctypes.byref(T.OrthDesc(1, 8, 8, 0, 1, None)), ctypes.byref(h)) == 1
    assert create(None, ctypes.byref(h)) == 1 and create(None, None) == 1
    assert T._lib.conv_bwd_orth_get_status(None, None, None) == 1


def test_arguments(T):
    """Checked before the device is looked at."""
    p = T.Orthogonal(2, 10, 16, "f32")
    run, step = T._lib.conv_bwd_orth_apply, T._lib.conv_bwd_orth_update
    x, o = 1 << 20, 2 << 20
    assert run(None, x, 0, 0, o, 0, 0, None) == 1
    assert run(p._h, None, 0, 0, o, 0, 0, None) == 1 and run(p._h, x, 0, 0, None, 0, 0, None) == 1
    assert run(p._h, x, 15, 0, o, 0, 0, None) == 1 and run(p._h, x, 0, 159, o, 0, 0, None) == 1
    assert run(p._h, x, 0, 0, o, 17, 160, None) == 1
    assert run(p._h, x + 2, 0, 0, o, 0, 0, None) == 3 and run(p._h, x, 0, 0, o + 1, 0, 0, None) == 3
    assert run(p._h, x, 0, 0, x + 4, 0, 0, None) == 1 and run(p._h, x, 20, 0, x, 16, 0, None) == 1  # overlaps, not in place
    assert run(p._h, x, (1 << 31) + 1, 0, o, 0, 0, None) == 2 and run(p._h, x, 0, (1 << 40) + 1, o, 0, 0, None) == 2
    assert run(p._h, x, 1 << 62, 0, o, 0, 0, None) == 2 and run(p._h, x, 0, 0, o, 1 << 60, 0, None) == 2 and run(p._h, x, -16, 0, o, 0, 0, None) == 1
    w, g, m, c = (i << 20 for i in range(1, 5))
    good = lambda **k: step(*[{"p": p._h, "w": w, "g": g, "ldg": 0, "lsg": 0, "m": m, "c": c, "lr": .1, "beta": .9, "nes": 1, "decay": 0., "scale": 1., "s": None, **k}[n]  # noqa: E731
                              for n in ("p", "w", "g", "ldg", "lsg", "m", "c", "lr", "beta", "nes", "decay", "scale", "s")])
    for k in ("p", "w", "g", "m"):
        assert good(**{k: None}) == 1, k
    for k, v in (("w", w + 2), ("m", m + 1), ("c", c + 1), ("g", g + 2)):
        assert good(**{k: v}) == 3, k
    for k, v in (("w", g + 16), ("m", w + 640), ("c", w), ("c", m + 64), ("c", g), ("m", g)):  # overlaps
        assert good(**{k: v}) == 1, k
    nan, inf = float("nan"), float("inf")
    for k, v in (("lr", nan), ("lr", inf), ("beta", nan), ("beta", -0.1), ("beta", 1.5), ("decay", inf), ("scale", nan), ("ldg", 15), ("lsg", 100)):
        assert good(**{k: v}) == 1, (k, v)
    if not torch.cuda.is_available():
        assert run(p._h, x, 0, 0, o, 0, 0, None) == 4 and run(p._h, x, 0, 0, x, 0, 0, None) == 4 and good() == 4 and good(c=None) == 4


def test_tensors(T):
    p, z = T.Orthogonal(2, 10, 16, "f32"), torch.zeros
    with pytest.raises(ValueError, match="x"):
        p.apply(z(2, 10, 16))                  # on the CPU
    with pytest.raises(ValueError, match="x"):
        p.apply(z(2, 10, 15))
    with pytest.raises(ValueError, match="grad"):
        p.update(z(2, 10, 16), z(2, 10, 16), z(2, 10, 16), 0.1)
