"""The one-launch form of clipping over every number of blocks: norm, coefficient and all gradients the same at every call,
and those of a norm that is taken alone (tolerances as in test_gpu_clip.py)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

NORM_TOL = 36 * 2.0 ** -24
COEF_TOL = 40 * 2.0 ** -24


@pytest.mark.parametrize("dtype,each", [(torch.float32, 8192), (torch.bfloat16, 16384)])
def test_blocks_agree_on_the_coefficient(dtype, each):
    """1 to 300 blocks of a chunk each, 20 calls without a pause: a block that took another for the last one, or scaled
    a part by another coefficient, shows in its chunk."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_backward_implicit_bwd_gb300 import build as cbuild
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
    gen = torch.Generator(device="cuda").manual_seed(1)
    for blocks in (1, 2, 3, 37, 152, 153, 300):
        g = [torch.randn(blocks * each - 3, generator=gen, device="cuda").to(dtype)]
        plan, out = T.GradClip.like(g), [torch.empty_like(g[0]) for _ in range(20)]
        alone = plan.norm(g)
        got = [plan.clip(g, 1.0, out=[o]) for o in out]
        want = math.sqrt(float((g[0].double() ** 2).sum()))
        assert abs(float(alone) - want) <= NORM_TOL * want
        assert plan.status() == (0, 0)
        for (norm, coef), o in zip(got, out):
            assert torch.equal(norm, alone) and torch.equal(coef, got[0][1])
            assert abs(float(coef) * (want + 1e-6) - 1) <= COEF_TOL
            assert torch.equal(o, (g[0].float() * coef).to(dtype))
