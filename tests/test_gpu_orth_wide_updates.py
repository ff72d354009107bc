"""Updates whose tiles are 256 wide, deep contractions among them, and matrices at the ends of the sizes; tolerances as in test_gpu_orth."""
import pytest
import torch
from test_gpu_orth import COEF, DT, T, check, iterate, matrices  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(90, 300, 600), (40, 520, 513), (16, 1024, 768), (14, 700, 2050), (1, 2304, 2310), (2, 300, 2048)])
@pytest.mark.parametrize("nesterov", [True, False])
def test_update(T, dtype, shape, nesterov):  # noqa: F811
    b, m, n = shape
    g = matrices(shape, dtype=DT[dtype])
    mom, w = matrices(shape, seed=2), matrices(shape, "flat", seed=3)
    copy = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    lr, beta, decay, scale = 0.1, 0.9, 0.3, max(1.0, m / n) ** 0.5
    f = lambda v: float(torch.tensor(v))  # noqa: E731  (as the library has them)
    m1 = f(beta) * mom.double() + g.double()
    u = g.double() + f(beta) * m1 if nesterov else m1
    x, off = iterate(u, [COEF] * 5)
    off = off * (4.0 if dtype == "bf16" else 1.0)  # (accumulators of eight k-blocks)
    want = w.double() * (1 - lr * decay) - lr * scale * x
    terms = torch.linalg.matrix_norm(g.double().abs() + 2 * mom.double().abs()) / torch.linalg.matrix_norm(u)
    room = lr * scale * (off + 200 * 2.0 ** -23 * terms) + 4 * 2.0 ** -24 * (torch.linalg.matrix_norm(w.double()) + lr * scale * torch.linalg.matrix_norm(x))
    plan = T.Orthogonal(*shape, dtype)
    plan.update(w, g, mom, lr, beta=beta, nesterov=nesterov, decay=decay, copy=copy)
    assert plan.status() == (0, 0)
    assert ((mom.double() - m1).abs() <= 2.0 ** -24 * m1.abs() + 1e-45).all()
    assert (torch.linalg.matrix_norm(w.double() - want) <= room).all()
    assert torch.equal(copy, w.bfloat16())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1, 65536), (1, 65536, 1), (2, 3, 2049), (1, 60000, 2), (3, 33, 2500), (1, 2500, 128), (700, 1, 2100)])
def test_long_thin_matrices(T, dtype, shape):  # noqa: F811
    u = matrices(shape, dtype=DT[dtype])
    plan = T.Orthogonal(*shape, dtype)
    check(plan.apply(u), *iterate(u, [COEF] * 5))
    assert plan.status() == (0, 0)
