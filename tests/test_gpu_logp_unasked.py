"""Arguments of the log-probabilities' gradient that no gradient asks for: whatever they hold, the result is that without them."""
import math

import pytest
import torch
from test_gpu_logp import T, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(5, 50), (3, 40001)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_entropy_without_its_gradient(T, dtype, t, v, value):  # noqa: F811
    z, a = rows_of(t, v, dtype)
    plan, g = T.TokenLogp(v, dtype), torch.ones(t, device="cuda")
    lse = plan.forward(z, a)[2]
    want = plan.backward(z, a, lse, grad_logp=g)
    assert torch.isfinite(want).all()
    assert torch.equal(plan.backward(z, a, lse, torch.full((t,), value, device="cuda"), grad_logp=g), want)
