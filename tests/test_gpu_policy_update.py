"""Token log-probabilities and orthogonalised updates in a policy step with the operators around them: the gradients against the
formulas in 64 bits, the step on the weights, a whole step captured."""
import os
import sys

import pytest
import torch
from test_gpu_orth import COEF, iterate

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def step():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_backward_implicit_bwd_gb300 import build as cbuild
    cbuild.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import expert_policy_step
    finally:
        sys.path.pop(0)
    return expert_policy_step


def test_gradients_of_a_step(step):
    """As in the plain step, with an entropy bonus: both gradients are rounded to bf16, and so is their sum.  What is left are
    roundings that fall to the other side, 2^-8 of single elements: 2^-8 of the norm at most."""
    m = step.ExpertPolicy(rows=700, seed=3, orthogonal=True, bonus=0.3)
    actions, adv, weight, old, _ = m.batch()
    loss, logp = m.gradients(actions, adv, weight, old, old)
    r = lambda t: t.bfloat16().double()  # noqa: E731
    off = m.offsets.tolist()
    a = torch.cat([m.x[s:e].double() @ m.w[0][i].double().T for i, (s, e) in enumerate(zip(off, off[1:]))])
    h = r(torch.relu(r(a)))
    z = r(h @ m.w[1][0].double().T).requires_grad_()
    u = torch.log_softmax(z, 1)
    lp = u.gather(1, actions[:, None].long())[:, 0]
    assert float((old.double() - lp.detach()).abs().max()) <= 1e-4 and float((logp - old).abs().max()) <= 1e-4  # the same policy
    ratio, d = torch.exp(lp - old.double()), old.double() - lp
    want = (weight.double() * (-torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + 0.01 * (torch.expm1(d) - d))).sum()
    policy, = torch.autograd.grad(want, z, retain_graph=True)
    entropy, = torch.autograd.grad((-0.3 * weight.double() * -(u.exp() * u).sum(1)).sum(), z)
    assert abs(float(loss) - float(want.detach())) <= 1e-5
    dz = r(r(policy) + r(entropy))
    dh = r(r(dz @ m.w[1][0].double()) * (h > 0))
    dw0 = torch.stack([dh[s:e].T @ m.x[s:e].double() for s, e in zip(off, off[1:])])
    dw1 = (dz.T @ h)[None]
    for got, ref in zip(m.grads, (dw0, dw1)):
        assert float((got.double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm())
    # the update, from the gradients as they are: clipped (2^-23), u = 1.95 times that (2^-23), X (its tolerance), the step
    grads, masters = [g.clone() for g in m.grads], [w.clone() for w in m.masters]
    norm = float(m.update())
    clip = min(1.0, m.max_norm / (norm + 1e-6))
    for g, before, after, copy, moment in zip(grads, masters, m.masters, m.w, m.momenta):
        x, off_x = iterate(g, [COEF] * 5)
        move = m.lr * max(1.0, g.shape[1] / g.shape[2]) ** 0.5
        room = move * (off_x + 400 * 2.0 ** -23) + 2.0 ** -22 * (torch.linalg.matrix_norm(before.double()) + move * torch.linalg.matrix_norm(x))
        assert (torch.linalg.matrix_norm(after.double() - (before.double() - move * x)) <= room).all()
        assert torch.equal(copy, after.bfloat16())
        assert ((moment.double() - clip * g.double()).abs() <= 2.0 ** -21 * clip * g.double().abs() + 1e-30).all()
    assert all(float(g.abs().max()) == 0 for g in m.grads)
    m.check()


def test_steps_run(step):
    m = step.ExpertPolicy(seed=1, orthogonal=True)
    for _ in range(5):
        out = m.step()
    assert all(torch.isfinite(t).all() for t in (*out.values(), *m.masters, *m.momenta))
    m.check()


def test_the_step_as_a_graph(step):
    """Gradients and update captured once and replayed: the same bits as outside."""
    m = step.ExpertPolicy(rows=500, seed=5, orthogonal=True)
    args = [t.clone() for t in m.batch()[:4]]
    state = [*m.masters, *m.w, *m.momenta, *m.grads]
    start = [t.clone() for t in state]

    def whole():
        loss, _ = m.gradients(*args, args[3])
        return [loss, m.update()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        whole()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = whole()
    seen = []
    for replay in (True, False):
        for t, x in zip(state, start):
            t.copy_(x)
        for _ in range(3):
            got = out if replay else whole()
            if replay:
                graph.replay()
        torch.cuda.synchronize()
        seen.append([t.clone() for t in (*state, *got)])
    assert all(torch.equal(x, y) for x, y in zip(*seen))
    m.check()
