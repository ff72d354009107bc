"""Stacks of padded matrices by the C ABI: a matrix stride of 0 is that of [batch][rows][ld]."""
import ctypes

import pytest
import torch
from test_gpu_orth import DT, T, matrices  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 10, 16), (2, 200, 140), (2, 140, 300)])
@pytest.mark.parametrize("pad", [0, 3, 4])
def test_matrix_stride_of_zero(T, dtype, shape, pad):  # noqa: F811
    b, m, n = shape
    u = matrices(shape, dtype=DT[dtype])
    plan = T.Orthogonal(*shape, dtype)
    want = plan.apply(u)
    x, out = torch.zeros(b, m, n + pad, dtype=DT[dtype], device="cuda"), torch.full((b, m, n + pad), 5.0, dtype=DT[dtype], device="cuda")
    x[:, :, :n] = u
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert T._lib.conv_bwd_orth_apply(plan._h, x.data_ptr(), n + pad, 0, out.data_ptr(), n + pad, 0, stream) == 0
    assert torch.equal(out[:, :, :n], want) and (out[:, :, n:] == 5.0).all()
    sides = [[matrices(shape, seed=s) for s in (2, 3)] for _ in range(2)]  # weight, momentum
    plan.update(sides[0][0], u, sides[0][1], 0.1)
    assert T._lib.conv_bwd_orth_update(plan._h, sides[1][0].data_ptr(), x.data_ptr(), n + pad, 0, sides[1][1].data_ptr(), None, 0.1, 0.95, 1, 0.0, max(1.0, m / n) ** 0.5, stream) == 0
    assert torch.equal(sides[0][0], sides[1][0]) and torch.equal(sides[0][1], sides[1][1]) and plan.status() == (0, 0)
