"""The training-step operators together: one step's gradients against the formulas in 64 bits, and learning."""
import os
import sys

import pytest
import torch

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
    """Reference: the chain in 64 bits, rounded to bf16 where the operators round (hidden, logits, dlogits, dhidden).
    What is left are roundings that fall to the other side, 2^-8 of single elements: 2^-8 of the norm at most."""
    m = step.ExpertPolicy(rows=700, seed=3)
    actions, adv, weight, old, _ = m.batch()
    loss, logp = m.gradients(actions, adv, weight, old, old)
    r = lambda t: t.bfloat16().double()  # noqa: E731
    off = m.offsets.tolist()
    a = torch.cat([m.x[s:e].double() @ m.w[0][i].double().T for i, (s, e) in enumerate(zip(off, off[1:]))])
    h = r(torch.relu(r(a)))
    z = r(h @ m.w[1][0].double().T).requires_grad_()
    lp = torch.log_softmax(z, 1).gather(1, actions[:, None].long())[:, 0]
    ratio, d = torch.exp(lp - old.double()), old.double() - lp
    want = (weight.double() * (-torch.minimum(ratio * adv, ratio.clamp(0.8, 1.2) * adv) + 0.01 * (torch.expm1(d) - d))).sum()
    want.backward()
    assert abs(float(loss) - float(want)) <= 1e-5 and float((logp - lp).abs().max()) <= 1e-4
    dz = r(z.grad)
    dh = r(r(dz @ m.w[1][0].double()) * (h > 0))
    dw0 = torch.stack([dh[s:e].T @ m.x[s:e].double() for s, e in zip(off, off[1:])])
    dw1 = (dz.T @ h)[None]
    for got, ref in zip(m.grads, (dw0, dw1)):
        assert float((got.double() - ref).norm()) <= 2.0 ** -8 * float(ref.norm())
    norm = torch.sqrt(dw0.square().sum() + dw1.square().sum())
    assert abs(float(m.update()) - float(norm)) <= 2.0 ** -8 * float(norm)
    m.check()


def test_the_policy_learns(step):
    m = step.ExpertPolicy(seed=1)
    first = float(m.step()["reward"])
    for _ in range(100):
        last = m.step()
    assert float(last["reward"]) >= 0.15 and first <= 0.05  # 64 actions: 0.016 at random
    m.check()


def test_the_step_as_a_graph(step):
    """The gradient part captured once and replayed: the same bits as outside, on new actions."""
    m = step.ExpertPolicy(rows=500, seed=5)
    args = [t.clone() for t in m.batch()[:4]]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        m.gradients(*args, args[3])
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    for gr in m.grads:
        gr.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        loss, _ = m.gradients(*args, args[3])
    for _ in range(2):
        for t, new in zip(args, m.batch()):
            t.copy_(new)
        for gr in m.grads:
            gr.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [gr.clone() for gr in m.grads] + [loss.clone()]
        for gr in m.grads:
            gr.zero_()
        want, _ = m.gradients(*args, args[3])
        assert all(torch.equal(x, y) for x, y in zip(got, m.grads + [want]))
