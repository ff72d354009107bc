"""Rows whose masked logits have the type's lowest value, against the definition in 64 bits; tolerances as in test_gpu_logp."""
import pytest
import torch
from test_gpu_logp import DT, T, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu

KINDS = {"first half": lambda v: slice(0, v // 2), "tail": lambda v: slice(v // 2, v), "all but one": lambda v: slice(0, v - 1), "every other": lambda v: slice(0, v, 2),
         "all": lambda v: slice(0, v), "all but the first of a batch": lambda v: slice(1, v)}


def statistics(z, scale):
    """log p and entropy of each row."""
    zd = z.double() * scale
    u = zd - zd.amax(1, keepdim=True)
    u = u - u.exp().sum(1, keepdim=True).log()
    return u, -torch.special.xlogy(u.exp(), u.exp()).sum(1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(3, 5), (4, 50), (4, 3000), (4, 60000), (1, 128000), (600, 9000), (2500, 5001)])
@pytest.mark.parametrize("scale", [1.0, 0.75, 3.0])
@pytest.mark.parametrize("top", [0, 4])
def test_statistics(T, dtype, t, v, scale, top):  # noqa: F811
    for kind, where in KINDS.items():
        z, a = rows_of(t, v, dtype)
        z[:, where(v)] = torch.finfo(DT[dtype]).min
        a[1::5] = -1
        plan = T.TokenLogp(v, dtype, top=top, scale=scale)
        logp, h, lse, tlp, tt = plan.forward(z, a)
        assert plan.status() == (0, 0)
        live, lowest = a >= 0, torch.finfo(torch.float32).min
        u, h_ = statistics(z, scale)
        # (what fp32 cannot hold is -inf)
        near = lambda x, y: ((x.double() - y).abs() <= 2.0 ** -19 * (1 + lse.double().abs().clamp(max=1e30) + y.abs())) | ((y < 0.999 * lowest) & (x.double() < 0.998 * lowest))  # noqa: E731
        assert ((h.double() - h_).abs() <= 2.0 ** -19 * (2 + h_))[live].all(), kind
        assert near(logp, u.gather(1, a.clamp(min=0).long()[:, None])[:, 0])[live].all(), kind
        if top:
            order = z.float().sort(dim=1, descending=True, stable=True).indices[:, :top]
            assert torch.equal(tt[live], order[live].int()), kind
            want = u.gather(1, order)
            assert ((tlp.double() - want).abs() <= 2.0 ** -19 * (1 + lse.double().abs().clamp(max=1e30)[:, None] + want.abs()))[live & (want > 0.9 * lowest).all(1)].all(), kind


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(4, 50), (3, 9001), (400, 20000)])
def test_gradients_of_rows_that_are_lowest_throughout(T, dtype, t, v):  # noqa: F811
    """lse cannot hold log v beside them, but no probability is above 1: |dz| <= scale (2 |gl| + |ge| H), and three roundings."""
    z = torch.full((t, v), torch.finfo(DT[dtype]).min, dtype=DT[dtype], device="cuda")
    a = torch.arange(t, dtype=torch.int32, device="cuda") % v
    g = torch.Generator(device="cuda").manual_seed(1)
    gl, ge = torch.randn(t, generator=g, device="cuda"), torch.randn(t, generator=g, device="cuda")
    for scale in (1.0, 0.9, 0.8, 0.77, 0.7, 0.6, 0.55, 0.3, 0.1, 0.01):
        plan = T.TokenLogp(v, dtype, scale=scale)
        _, h, lse, _, _ = plan.forward(z, a)
        dz = plan.backward(z, a, lse, h, grad_logp=gl, grad_entropy=ge)
        assert plan.status() == (0, 0)
        room = scale * (2 * gl.abs() + ge.abs() * h) * (1 + 3 * torch.finfo(DT[dtype]).eps)
        assert (dz.float().abs() <= room[:, None]).all(), scale


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(4, 50), (4, 60000), (600, 9000)])
@pytest.mark.parametrize("kind", ["first half", "tail", "all but one", "every other"])
def test_gradients_beside_lowest_values(T, dtype, t, v, kind):  # noqa: F811
    from test_gpu_logp import gradient
    z, a = rows_of(t, v, dtype)
    z[:, KINDS[kind](v)] = torch.finfo(DT[dtype]).min
    scale = torch.tensor(0.7).item()
    plan = T.TokenLogp(v, dtype, scale=0.7)
    _, h, lse, _, _ = plan.forward(z, a)
    g = torch.Generator(device="cuda").manual_seed(3)
    gl, ge = torch.randn(t, generator=g, device="cuda"), torch.randn(t, generator=g, device="cuda")
    want, size = gradient(z, a, lse, h, gl, ge, scale)
    got = plan.backward(z, a, lse, h, grad_logp=gl, grad_entropy=ge)
    # (size has 0 * inf in lowest places, where p is 0)
    assert ((got.double() - want).abs() <= size.nan_to_num(0.0) + want.abs() * torch.finfo(DT[dtype]).eps / 2 + 1e-37).all()
