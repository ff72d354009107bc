"""Counts that a 32-bit field does not hold are refused, not taken by their low bits (no GPU)."""
import pytest

from conv2d_backward_implicit_bwd_gb300 import build as cbuild


@pytest.fixture(scope="module")
def T():
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train
    return train


@pytest.mark.parametrize("make,status", [(lambda T: T.TokenLogp(1 << 29, top=(1 << 32) + 3), 1), (lambda T: T.TokenLogp(100, top=-(1 << 32) + 3), 1), (lambda T: T.Orthogonal(1, 8, 8, steps=(1 << 32) + 2), 2),
                                         (lambda T: T.Orthogonal(1, 8, 8, steps=1 << 40), 2), (lambda T: T.Orthogonal(1, 8, 8, steps=-(1 << 32) + 2), 1), (lambda T: T.Orthogonal(1, 8, 8, steps=65), 2)])
def test_refused(T, make, status):
    from conv2d_backward_implicit_bwd_gb300.binding import ConvBwdError
    with pytest.raises(ConvBwdError) as e:
        make(T)
    assert e.value.status == status
