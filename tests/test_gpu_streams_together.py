"""Plans of the training-step operators on streams of their own, all at once; updates on wide tiles as graphs."""
import pytest
import torch
from test_gpu_logp import T, rows_of  # noqa: F401
from test_gpu_orth import matrices

pytestmark = pytest.mark.gpu


def test_plans_on_streams_of_their_own(T):  # noqa: F811
    """The same bits as alone: rows in parts, rows of a warp, split tiles, wide tiles, clusters."""
    jobs = []
    for t, v, top in ((3, 60000, 7), (64, 128000, 5), (700, 3000, 2), (400, 20000, 0)):
        z, a = rows_of(t, v, "bf16", seed=t)
        plan, g = T.TokenLogp(v, top=top), torch.ones(t, device="cuda")

        def run(s, plan=plan, z=z, a=a, g=g):
            out = plan.forward(z, a, stream=s)
            return [*(x for x in out if x is not None), plan.backward(z, a, out[2], out[1], grad_logp=g, grad_entropy=g, stream=s)]
        jobs.append((plan, run))
    for shape, dtype in (((2, 768, 768), "f32"), ((1, 1000, 700), "bf16"), ((40, 513, 520), "bf16"), ((5, 128, 2048), "f32"), ((3, 300, 2000), "f32")):
        u, plan = matrices(shape, dtype=torch.float32 if dtype == "f32" else torch.bfloat16), T.Orthogonal(*shape, dtype)
        jobs.append((plan, lambda s, plan=plan, u=u: [plan.apply(u, stream=s)]))
    want = [[x.clone() for x in run(None)] for _, run in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(6):
        got = [[run(s) for _ in range(2)][-1] for (_, run), s in zip(jobs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for g, w in zip(got, want) for x, y in zip(g, w))
    assert all(plan.status() == (0, 0) for plan, _ in jobs)


@pytest.mark.parametrize("shape,dtype", [((16, 1024, 768), torch.bfloat16), ((40, 513, 520), torch.float32), ((2, 768, 768), torch.float32), ((4, 128, 2048), torch.float32)])
def test_updates_as_graphs(T, shape, dtype):  # noqa: F811
    plan, seen = T.Orthogonal(*shape, "bf16" if dtype == torch.bfloat16 else "f32"), []
    w, mom, g, copy = matrices(shape, seed=5), matrices(shape, seed=6), matrices(shape, seed=7, dtype=dtype), torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    start = [t.clone() for t in (w, mom, g, copy)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        plan.update(w, g, mom, 0.1, copy=copy)
    side.synchronize()
    with torch.cuda.graph(graph):
        plan.update(w, g, mom, 0.1, copy=copy)
    for replay in (True, False):
        for t, s in zip((w, mom, g, copy), start):
            t.copy_(s)
        for i in range(3):
            g.copy_(matrices(shape, seed=20 + i, dtype=dtype))
            graph.replay() if replay else plan.update(w, g, mom, 0.1, copy=copy)
        seen.append([t.clone() for t in (w, mom, copy)])
    assert all(torch.equal(a, b) for a, b in zip(*seen)) and plan.status() == (0, 0)
