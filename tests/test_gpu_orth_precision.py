"""What the results of the orthogonalised updates are off by, against the iteration in 64 bits."""
import pytest
import torch
from test_gpu_orth import COEF, DT, T, iterate, matrices  # noqa: F401

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


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1024, 2048), (1, 1024, 1024), (1, 512, 4096), (2, 2048, 300), (16, 1024, 768), (1, 100, 131), (1, 128, 2048)])
@pytest.mark.parametrize("kind", ["few directions", "flat"])
def test_five_steps(T, dtype, shape, kind):  # noqa: F811
    """What the header says of them: below 2^-14 of X's norm in plans of fp32, 2^-12 in plans of bf16, in steps on weights as in results."""
    g = torch.Generator(device="cuda").manual_seed(1)
    b, m, n = shape
    u = torch.randn(shape, generator=g, device="cuda")
    if kind == "few directions":
        u = torch.randn(b, m, 8, generator=g, device="cuda") @ torch.randn(b, 8, n, generator=g, device="cuda") + 0.01 * u
    u = u.to(DT[dtype])
    x, _ = iterate(u, [COEF] * 5)
    plan, w, mom = T.Orthogonal(*shape, dtype), torch.zeros(shape, device="cuda"), torch.zeros(shape, device="cuda")
    plan.update(w, u, mom, 1.0, beta=0.0, scale=1.0)  # w = -X
    room = {"f32": 2.0 ** -14, "bf16": 2.0 ** -12}[dtype] * torch.linalg.matrix_norm(x)
    off = torch.linalg.matrix_norm(-w.double() - x)
    assert (off <= room).all(), (off / room).max()
    if dtype == "f32":
        off = torch.linalg.matrix_norm(plan.apply(u).double() - x)
        assert (off <= room).all(), (off / room).max()
    assert plan.status() == (0, 0)
