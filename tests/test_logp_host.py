"""Refusals of the token log-probabilities (no GPU): descriptors, arguments, tensors."""
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


@pytest.mark.parametrize("kw,status", [(dict(vocab=0), 1), (dict(vocab=-5), 1), (dict(top=-1), 1), (dict(top=9), 1), (dict(scale=0.0), 1),
                                       (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(vocab=(1 << 30) + 1), 2), (dict(vocab=100, top=33), 2)])
def test_descriptor(T, kw, status):
    assert status_of(lambda: T.TokenLogp(**{"vocab": 8, **kw})) == status


def test_unknown(T):
    with pytest.raises(ValueError):
        T.TokenLogp(8, "f16")
    h = ctypes.c_void_p()
    create = T._lib.conv_bwd_logp_create
    assert create(ctypes.byref(T.LogpDesc(8, 7, 0, 1.0)), ctypes.byref(h)) == 1 and not h.value
    assert create(None, ctypes.byref(h)) == 1 and create(None, None) == 1
    assert T._lib.conv_bwd_logp_get_status(None, None, None) == 1


def test_arguments(T):
    """Checked before the device is looked at."""
    p = T.TokenLogp(100, "f32", top=3)
    fwd, bwd = T._lib.conv_bwd_logp_forward, T._lib.conv_bwd_logp_backward
    z, a, lp, h, lse, tl, tt = (i << 20 for i in range(1, 8))
    assert fwd(None, 4, z, 0, a, lp, h, lse, tl, tt, None) == 1
    assert fwd(p._h, -1, z, 0, a, lp, h, lse, tl, tt, None) == 1
    assert fwd(p._h, 4, z, 99, a, lp, h, lse, tl, tt, None) == 1
    good = [z, a, lp, h, lse, tl, tt]
    for i in range(7):  # NULL, misaligned
        g = list(good)
        g[i] = None
        assert fwd(p._h, 4, g[0], 0, *g[1:], None) == 1, i
        g[i] = good[i] + 2
        assert fwd(p._h, 4, g[0], 0, *g[1:], None) == 3, i
        if i >= 2:  # an output over the logits, the tokens, another output
            for other in (z, a, h if i != 3 else lse):
                g[i] = other
                assert fwd(p._h, 4, g[0], 0, *g[1:], None) == 1, i
    assert fwd(p._h, 1 << 31, z, 0, 1 << 50, 2 << 50, 3 << 50, 4 << 50, 5 << 50, 6 << 50, None) == 2
    args = [z, a, lse, h, lp, tl]  # logits, tokens, lse, entropy, grad_logp, grad_entropy
    out = 9 << 20
    assert bwd(None, 4, args[0], 0, *args[1:], out, 0, None) == 1
    assert bwd(p._h, 4, args[0], 0, *args[1:], None, 0, None) == 1
    assert bwd(p._h, 4, args[0], 0, *args[1:], out, 99, None) == 1
    assert bwd(p._h, 4, z, 0, a, lse, h, None, None, out, 0, None) == 1     # no gradient
    assert bwd(p._h, 4, z, 0, None, lse, h, lp, tl, out, 0, None) == 1      # a gradient of logp without tokens
    assert bwd(p._h, 4, z, 0, a, lse, None, lp, tl, out, 0, None) == 1      # of entropy without entropy
    assert bwd(p._h, 4, z, 0, a, None, h, lp, tl, out, 0, None) == 1
    assert bwd(p._h, 4, z, 0, *args[1:], z + 8, 0, None) == 1               # overlaps, not in place
    assert bwd(p._h, 4, z, 128, *args[1:], z, 100, None) == 1               # in place with another stride
    assert bwd(p._h, 4, z, 0, *args[1:], lse, 0, None) == 1                 # over an input
    assert bwd(p._h, 4, z, 0, *args[1:], out + 2, 0, None) == 3
    if not torch.cuda.is_available():
        assert fwd(p._h, 4, z, 0, a, lp, h, lse, tl, tt, None) == 4
        assert bwd(p._h, 4, z, 0, *args[1:], z, 0, None) == 4


def test_tensors(T):
    z = torch.zeros
    p = T.TokenLogp(9, "f32")
    with pytest.raises(ValueError, match="logits"):
        p.forward(z(4, 9), None)                       # on the CPU
    with pytest.raises(ValueError, match="logits"):
        p.forward(z(4, 8))
    with pytest.raises(ValueError, match="logits"):
        p.backward(z(4, 9), None, z(4), z(4), grad_entropy=z(4))
