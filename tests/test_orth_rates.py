"""Steps whose factors overflow are refused (no GPU)."""
import pytest

from conv2d_backward_implicit_bwd_gb300 import build as cbuild


@pytest.mark.parametrize("lr,decay,scale", [(1e30, 0.0, 1e30), (1e30, 1e30, 1.0), (-1e30, 0.0, 1e30)])
def test_products_that_overflow(lr, decay, scale):
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
    p = T.Orthogonal(2, 10, 16, "f32")
    w, g, m = (i << 20 for i in range(1, 4))
    assert T._lib.conv_bwd_orth_update(p._h, w, g, 0, 0, m, None, lr, 0.9, 1, decay, scale, None) == 1
