"""Host-side tests of the training-step operators' C ABI and binding (no GPU):
exports, refusals, and plans without a device."""
import ctypes

import pytest
import torch

from conv2d_backward_implicit_bwd_gb300 import build as cbuild


@pytest.fixture(scope="module")
def T():
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train
    return train


def test_library_exports_every_declared_symbol(T):
    lib = ctypes.CDLL(T._b.LIB_PATH)
    for n in T.EXPORTED:
        assert hasattr(lib, n), n


def status_of(f):
    from conv2d_backward_implicit_bwd_gb300.binding import ConvBwdError
    with pytest.raises(ConvBwdError) as e:
        f()
    return e.value.status


@pytest.mark.parametrize("args,status", [
    ((0, 8, 8), 1), ((1, 0, 8), 1), ((1, 8, -1), 1), ((1025, 8, 8), 2), ((1, (1 << 20) + 1, 8), 2),
    ((1024, 1 << 20, 1 << 20), 2)])
def test_experts_descriptor(T, args, status):
    assert status_of(lambda: T.Experts(*args)) == status


def test_unknown_dtype(T):
    for make in (lambda: T.Experts(1, 8, 8, "f16"), lambda: T.PolicyLoss(8, torch.float16),
                 lambda: T.GradClip([1], ["int8"])):
        with pytest.raises(ValueError):
            make()
    lib = T._lib
    h = ctypes.c_void_p()
    assert lib.conv_bwd_experts_create(ctypes.byref(T.ExpertsDesc(1, 8, 8, 7)), ctypes.byref(h)) == 1 and not h.value
    assert lib.conv_bwd_policy_create(ctypes.byref(T.PolicyDesc(8, 7, .2, .2, 0, 1)), ctypes.byref(h)) == 1
    assert lib.conv_bwd_clip_create(1, (ctypes.c_int64 * 1)(3), (ctypes.c_int32 * 1)(7), ctypes.byref(h)) == 1
    for f in (lib.conv_bwd_experts_create, lib.conv_bwd_policy_create):
        assert f(None, ctypes.byref(h)) == 1
        assert f(None, None) == 1


@pytest.mark.parametrize("kw", [dict(vocab=0), dict(clip_low=-0.1), dict(clip_low=1.5), dict(clip_high=-1.0),
                                dict(clip_high=float("inf")), dict(kl=-1.0), dict(kl=float("nan")), dict(scale=0.0),
                                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf"))])
def test_policy_parameters(T, kw):
    assert status_of(lambda: T.PolicyLoss(**{"vocab": 8, **kw})) == 1


def test_policy_vocab_limit(T):
    assert status_of(lambda: T.PolicyLoss((1 << 30) + 1)) == 2


def test_clip_sizes(T):
    assert status_of(lambda: T.GradClip([-1], ["f32"])) == 1
    assert status_of(lambda: T.GradClip([1 << 38], ["f32"])) == 2
    assert status_of(lambda: T.GradClip([1 << 37] * 9, ["f32"] * 9)) == 2
    with pytest.raises(ValueError):
        T.GradClip([1, 2], ["f32"])


def test_run_arguments(T):
    """Checked before the device is looked at."""
    lib = T._lib
    e = T.Experts(2, 16, 8)
    run = lib.conv_bwd_experts_forward
    a, b, o, y = 1 << 20, 2 << 20, 3 << 20, 4 << 20
    assert run(None, 4, a, 0, b, o, y, 0, None) == 1
    assert run(e._h, -1, a, 0, b, o, y, 0, None) == 1
    for null in (dict(a=0), dict(b=0), dict(o=0), dict(y=0)):
        v = {"a": a, "b": b, "o": o, "y": y, **null}
        assert run(e._h, 4, v["a"], 0, v["b"], v["o"], v["y"], 0, None) == 1
    assert run(e._h, 4, a, 15, b, o, y, 0, None) == 1          # row stride shorter than a row
    assert run(e._h, 4, a, 0, b, o, y, 7, None) == 1
    assert run(e._h, 4, a, 0, b, o, a + 32, 0, None) == 1      # overlaps x
    assert run(e._h, 4, a, 0, b, o, b + 32, 0, None) == 1      # overlaps w
    assert run(e._h, 4, a, 0, b, o, o, 0, None) == 1           # overlaps offsets
    assert run(e._h, 4, a + 1, 0, b, o, y, 0, None) == 3
    assert run(e._h, 4, a, 0, b, o + 2, y, 0, None) == 3
    assert run(e._h, 1 << 31, a, 0, b, o, 1 << 50, 0, None) == 2
    wt = lib.conv_bwd_experts_weight
    assert wt(e._h, 4, a, 0, b, 0, o, None, 0, None) == 1
    assert wt(e._h, 4, a, 0, None, 0, o, y, 0, None) == 1
    assert wt(e._h, 4, a, 0, b, 15, o, y, 0, None) == 1
    assert wt(e._h, 4, a, 0, b, 0, o, y + 2, 0, None) == 3
    p = T.PolicyLoss(100, "f32")
    f = [1 << 20, 2 << 20, 3 << 20, 4 << 20, None, None, 5 << 20, 6 << 20, 7 << 20, 8 << 20]
    fwd = lib.conv_bwd_policy_forward
    assert fwd(None, 4, f[0], 0, *f[1:], None) == 1
    assert fwd(p._h, -1, f[0], 0, *f[1:], None) == 1
    assert fwd(p._h, 4, f[0], 99, *f[1:], None) == 1
    for i in (1, 2, 3, 6, 7, 8, 9):
        g = list(f)
        g[i] = None
        assert fwd(p._h, 4, g[0], 0, *g[1:], None) == 1, i
        if i != 6:
            g[i] = f[i] + 2
            assert fwd(p._h, 4, g[0], 0, *g[1:], None) == 3, i
    bwd = lib.conv_bwd_policy_backward
    assert bwd(p._h, 4, f[0], 0, f[1], f[2], f[3], None, f[0] + 8, 0, None) == 1     # overlaps, not in place
    assert bwd(p._h, 4, f[0], 128, f[1], f[2], f[3], None, f[0], 100, None) == 1     # in place with another stride
    c = T.GradClip([4, 0, 8], ["f32", "bf16", "bf16"])
    arr = ctypes.c_void_p * 3
    good = arr(1 << 20, None, 2 << 20)
    clip = lib.conv_bwd_clip_run
    n, k = 3 << 20, 4 << 20
    assert clip(c._h, good, good, float("nan"), n, k, None) == 1
    assert clip(c._h, good, good, -1.0, n, k, None) == 1
    assert clip(c._h, good, good, 1.0, None, k, None) == 1
    assert clip(c._h, good, good, 1.0, n, None, None) == 1
    assert clip(c._h, arr(None, None, 2 << 20), good, 1.0, n, k, None) == 1
    assert clip(c._h, good, arr((1 << 20) + 4, None, 2 << 20), 1.0, n, k, None) == 1
    odd = arr((1 << 20) + 2, None, 2 << 20)
    assert clip(c._h, odd, odd, 1.0, n, k, None) == 3
    assert lib.conv_bwd_clip_norm(c._h, None, n, None) == 1
    if not torch.cuda.is_available():  # plans made without a device cannot run
        assert run(e._h, 4, a, 0, b, o, y, 0, None) == 4
        assert fwd(p._h, 4, f[0], 0, *f[1:], None) == 4
        assert clip(c._h, good, good, 1.0, n, k, None) == 4
        assert e._h and T._lib.conv_bwd_experts_get_status(e._h, None, None) == 4


def test_tensor_checks(T):
    """Shapes, types and devices are refused before the library is called."""
    e = T.Experts(2, 16, 8, "f32")
    z = torch.zeros
    off = z(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="x"):
        e.forward(z(4, 16), z(2, 8, 16), off)                    # on the CPU
    with pytest.raises(ValueError, match="x"):
        e.forward(z(4, 15), z(2, 8, 16), off)
    with pytest.raises(ValueError, match="dy"):
        e.backward_weight(z(4, 16), z(4, 16), off)
    with pytest.raises(ValueError, match="logits"):
        T.PolicyLoss(9, "f32").forward(z(4, 9), None, None, None)
    c = T.GradClip.like([z(3), z(2, 2)])
    with pytest.raises(ValueError, match="2 tensors"):
        c.norm([z(3)])
    with pytest.raises(ValueError, match="grads"):
        c.norm([z(3), z(2, 2)])
    with pytest.raises(ValueError, match="max_norm"):
        c.clip([z(3), z(2, 2)], -1)
