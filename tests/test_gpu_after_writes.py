"""Launches begin while the kernel before them in the stream still runs: every input written just before a call, over and
over without a pause, must be read as written."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_backward_implicit_bwd_gb300 import build as cbuild
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train
    return train


def values(call, inputs, shapes):
    """The call's results for ten sets of inputs written one after the other, and the same with a pause around each call."""
    out = []
    for pause in (False, True):
        got = []
        for new in inputs:
            for t, n in zip(shapes, new):
                t.copy_(n)
            if pause:
                torch.cuda.synchronize()
            got.append([r.clone() for r in call()])
            if pause:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        out.append(got)
    return out


@pytest.mark.parametrize("dtype,experts,k,n,each", [
    ("f32", 24, 516, 260, 1), ("f32", 24, 515, 259, 3), ("f32", 3, 516, 260, 90), ("bf16", 24, 520, 264, 1), ("bf16", 96, 576, 1040, 2),
    ("bf16", 3, 520, 264, 200), ("bf16", 3, 517, 263, 90)])
@pytest.mark.parametrize("way", ["forward", "data", "weight"])
def test_experts(T, way, dtype, experts, k, n, each):
    plan, rows = T.Experts(experts, k, n, dtype), experts * each
    g = torch.Generator(device="cuda").manual_seed(1)
    a, b = {"forward": ((rows, k), (experts, n, k)), "data": ((rows, n), (experts, n, k)), "weight": ((rows, n), (rows, k))}[way]
    new = lambda s: torch.randn(*s, generator=g, device="cuda").to(plan.dtype)  # noqa: E731
    cuts = lambda i: torch.tensor([min(rows, e * each + i % 3) for e in range(experts)] + [rows], dtype=torch.int32, device="cuda")  # noqa: E731
    x, y, o = new(a), new(b), cuts(0)
    call = {"forward": plan.forward, "data": plan.backward_data, "weight": plan.backward_weight}[way]
    quick, slow = values(lambda: [call(x, y, o)], [(new(a), new(b), cuts(i)) for i in range(10)], (x, y, o))
    assert all(torch.equal(p, q) for u, v in zip(quick, slow) for p, q in zip(u, v))
    assert plan.status() == (0, 0)


@pytest.mark.parametrize("sizes", [[70_000, 9], [5_000_000, 3_000_000]])
def test_clip(T, sizes):
    g = torch.Generator(device="cuda").manual_seed(2)
    grads = [torch.zeros(s, device="cuda") for s in sizes]
    plan = T.GradClip.like(grads)
    new = [[torch.randn(s, generator=g, device="cuda") for s in sizes] for _ in range(10)]
    quick, slow = values(lambda: [*plan.clip(grads, 1.0), *grads], new, grads)
    assert all(torch.equal(p, q) for u, v in zip(quick, slow) for p, q in zip(u, v))


@pytest.mark.parametrize("vocab", [1000, 20000])
def test_policy(T, vocab):
    t, plan = 900, T.PolicyLoss(vocab, kl=0.1)
    g = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    new = lambda: (normal(t, vocab).bfloat16(), torch.randint(-1, vocab, (t,), generator=g, device="cuda", dtype=torch.int32), normal(t),  # noqa: E731
                   normal(t).relu(), normal(t) - 9, normal(t) - 9)
    state = new()

    def call():
        loss, logp, lse, coef = plan.forward(*state)
        dz = plan.backward(*state[:2], lse, coef)
        return [loss, logp, lse, coef, dz, *plan.forward_backward(*state)]
    quick, slow = values(call, [new() for _ in range(5)], state)
    assert all(torch.equal(p, q) for u, v in zip(quick, slow) for p, q in zip(u, v))
    assert plan.status() == (0, 0)
