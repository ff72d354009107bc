"""The policy loss's backward call on rows whose logits all have the type's lowest value: |dz| <= 2 |coef scale|, three roundings."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,v", [(4, 50), (3, 9001), (400, 20000)])
def test_backward_is_bounded(dtype, t, v):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_backward_implicit_bwd_gb300 import build as cbuild
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
    z = torch.full((t, v), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    a, one = torch.arange(t, dtype=torch.int32, device="cuda") % v, torch.ones(t, device="cuda")
    for scale in (1.0, 0.9, 0.8, 0.77, 0.7, 0.6, 0.55, 0.3, 0.1, 0.01):
        plan = T.PolicyLoss(v, "f32" if dtype == torch.float32 else "bf16", scale=scale)
        _, _, lse, coef = plan.forward(z, a, one, one)
        dz = plan.backward(z, a, lse, coef)
        assert plan.status() == (0, 0)
        room = 2 * scale * coef.abs() * (1 + 3 * torch.finfo(dtype).eps)
        assert (dz.float().abs() <= room[:, None]).all(), scale
