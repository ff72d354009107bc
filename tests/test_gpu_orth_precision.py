"""What the results of the orthogonalised updates are off by, against the iteration in 64 bits."""
import pytest
import torch
from test_gpu_orth import T, iterate, matrices  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(1, 60, 90), (3, 200, 128), (1, 1000, 1000), (2, 300, 513), (20, 512, 300), (40, 513, 520), (2, 257, 2000)])
@pytest.mark.parametrize("coef", [(1.0, 0.0, 0.0), (1.5, -0.5, 0.0)])
def test_bf16_results_are_rounded_once(T, shape, coef):  # noqa: F811
    """Of a result y off by e from the exact x, the nearest bf16 is off by |bf16(y) - x| <= |bf16(x) - y| + |x - y| <= |bf16(x) - x| + 2 e for
    every element, and so are the norms.  e is that of test_gpu_orth with four times its truncations (accumulators of eight k-blocks).
    One step on a flat spectrum, so that it is small beside the rounding: 4e-6 and 1.5e-5 of a norm of 1 and more, of which bf16
    rounds 1.6e-3; operands of 11 bits in the product would add 4.6e-5."""
    u = matrices(shape, "flat", dtype=torch.bfloat16)
    got = T.Orthogonal(*shape, "bf16", steps=1, coefficients=coef).apply(u)
    x, _ = iterate(u, [coef])
    e = coef[0] * 2.0 ** -23 + (abs(coef[0]) + 3.4 * abs(coef[1])) * 2.0 ** -18
    off, own = (torch.linalg.matrix_norm(t.double() - x) for t in (got, x.bfloat16()))
    assert (off <= own + 2 * e).all(), (off - own).max()
