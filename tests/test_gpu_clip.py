"""Global gradient norm and clipping against the definition in 64 bits.

Tolerances: a thread sums at most 68 squares in fp32 (each product and
addition rounds to 2^-24: below 70 2^-24 relative, all terms positive), then
fp64, then one fp32 rounding; the square root halves the relative error:
36 2^-24 on norm.  coef adds two roundings, out one product and its rounding."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

NORM_TOL = 36 * 2.0 ** -24
COEF_TOL = 40 * 2.0 ** -24


@pytest.fixture(scope="module")
def T():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from conv2d_backward_implicit_bwd_gb300 import build as cbuild
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train
    return train


def tensors(sizes, dtypes, scale=1.0, seed=1, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n, d in zip(sizes, dtypes):
        t = (torch.randn(n + shift, generator=g, device="cuda") * scale).to({"f32": torch.float32, "bf16": torch.bfloat16}[d])
        out.append(t[shift:])
    return out


def norm64(grads):
    return math.sqrt(sum(float((t.double() ** 2).sum()) for t in grads))


def check_clip(T, grads, max_norm, inplace, out_shift=0):
    want_norm = norm64(grads)
    want_coef = min(1.0, max_norm / (want_norm + 1e-6))
    before = [g.double() for g in grads]
    out = None
    if not inplace:
        out = [torch.full((g.numel() + out_shift,), 7.0, dtype=g.dtype, device="cuda")[out_shift:] for g in grads]
    plan = T.GradClip.like(grads)
    norm, coef = plan.clip(grads, max_norm, out=out)
    assert abs(float(norm) - want_norm) <= NORM_TOL * want_norm
    assert abs(float(coef) - want_coef) <= COEF_TOL * want_coef
    assert float(plan.norm(grads if not inplace else [b.to(g.dtype) for b, g in zip(before, grads)])) == float(norm)
    for b, o, g in zip(before, grads if inplace else out, grads):
        want = b * float(coef)
        ulp = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -23
        assert ((o.double() - want).abs() <= ulp * want.abs()).all()
        if not inplace:
            assert torch.equal(g.double(), b)
            if out_shift:
                assert (o._base[:out_shift] == 7).all()


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("sizes,dtypes", [
    ([1], ["f32"]), ([1], ["bf16"]), ([0, 5, 0], ["f32", "bf16", "bf16"]),
    ([8192, 8193, 16384, 16385, 3], ["f32", "f32", "bf16", "bf16", "f32"]),
    ([100_000, 7, 250_001, 64], ["bf16", "f32", "f32", "bf16"]),
    ([3_000_017], ["bf16"]), ([1_500_003], ["f32"]), ([9_000_001, 5, 4_000_003], ["bf16", "f32", "f32"]),
])
def test_norm_and_clip(T, sizes, dtypes, inplace):
    check_clip(T, tensors(sizes, dtypes), 0.5, inplace)


@pytest.mark.parametrize("shift,out_shift", [(1, 1), (3, 0), (0, 5), (2, 2)])
@pytest.mark.parametrize("inplace", [True, False])
def test_any_alignment(T, shift, out_shift, inplace):
    check_clip(T, tensors([9000, 17, 40_000, 1], ["f32", "bf16", "bf16", "f32"], shift=shift), 2.0, inplace, out_shift)


@pytest.mark.parametrize("out_shift", [0, 1])
def test_any_alignment_large(T, out_shift):
    """More than the SMs' registers hold: the norm and the scaling in launches of their own."""
    check_clip(T, tensors([7_000_003, 3_000_001], ["bf16", "f32"], shift=3), 2.0, False, out_shift)


def test_many_tensors(T):
    """More tensors than one launch carries."""
    n = 2503
    check_clip(T, tensors([1 + i % 77 for i in range(n)], ["f32" if i % 3 else "bf16" for i in range(n)]), 1.0, True)


def test_nothing_to_clip(T):
    g = tensors([1000, 2000], ["f32", "bf16"], scale=1e-3)
    before = [t.clone() for t in g]
    norm, coef = T.GradClip.like(g).clip(g, 100.0)
    assert float(coef) == 1.0 and all(torch.equal(a, b) for a, b in zip(g, before))
    out = [torch.zeros_like(t) for t in g]
    T.GradClip.like(g).clip(g, float("inf"), out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, before))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e30, 3e-30, 1e-38])
def test_squares_out_of_range(T, dtype, scale):
    """Gradients whose squares overflow or vanish in fp32 still have the right norm."""
    g = tensors([5000, 70_000], [dtype, dtype], scale=scale)
    g[1][::3] = 0
    want = norm64(g)
    norm = T.GradClip.like(g).norm(g)
    assert abs(float(norm) - want) <= NORM_TOL * want


def test_large_beside_small(T):
    """One tensor of huge and one of ordinary gradients: each thread falls back by itself."""
    g = tensors([5000], ["f32"], scale=1e25) + tensors([50_000], ["f32"])
    want = norm64(g)
    assert abs(float(T.GradClip.like(g).norm(g)) - want) <= NORM_TOL * want


def test_zeros(T):
    g = [torch.zeros(100, device="cuda"), torch.zeros(70_000, dtype=torch.bfloat16, device="cuda")]
    norm, coef = T.GradClip.like(g).clip(g, 1.0)
    assert float(norm) == 0 and float(coef) == 1 and (g[0] == 0).all()


def test_no_tensors(T):
    norm, coef = T.GradClip([], []).clip([], 1.0)
    assert float(norm) == 0 and float(coef) == 1


def test_max_norm_zero(T):
    g = tensors([100], ["f32"])
    _, coef = T.GradClip.like(g).clip(g, 0.0)
    assert float(coef) == 0 and (g[0] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_and_infinity(T, dtype):
    g = tensors([100, 20_000], [dtype, dtype])
    g[1][777] = float("inf")
    out = [torch.zeros_like(t) for t in g]
    norm, coef = T.GradClip.like(g).clip(g, 1.0, out=out)
    assert float(norm) == math.inf and float(coef) == 0
    assert (out[0] == 0).all() and torch.isnan(out[1][777]) and int(torch.isnan(out[1]).sum()) == 1
    g[0][3] = float("nan")
    norm, coef = T.GradClip.like(g).clip(g, 1.0, out=out)
    assert math.isnan(float(norm)) and math.isnan(float(coef)) and torch.isnan(out[0]).all()
    norm, coef = T.GradClip.like(g).clip(g, float("inf"), out=out)
    assert math.isnan(float(coef))


def test_same_bits_and_repeats(T):
    g = tensors([300_000, 41, 100_000], ["bf16", "f32", "f32"])
    plan = T.GradClip.like(g)
    first = plan.norm(g)
    for _ in range(5):
        assert torch.equal(plan.norm(g), first)
    twice = plan.clip(g, 1.0)
    again = plan.clip(g, 1.0)
    assert abs(float(again[0]) - 1.0) < 1e-2 and torch.equal(twice[0], first)


def test_side_stream_and_graph(T):
    g = tensors([50_000, 33], ["bf16", "f32"])
    out = [torch.zeros_like(t) for t in g]
    plan = T.GradClip.like(g)
    want = norm64(g)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norm = plan.norm(g, stream=s)
    s.synchronize()
    assert abs(float(norm) - want) <= NORM_TOL * want
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm, coef = plan.clip(g, 1.0, out=out)
    for k in (1.0, 3.0):
        g[0].mul_(k)
        graph.replay()
        want = norm64(g)
        assert abs(float(norm) - want) <= NORM_TOL * want
        assert abs(norm64(out) - 1.0) < 1e-2


def test_refusals(T):
    g = tensors([10, 20], ["f32", "bf16"])
    plan = T.GradClip.like(g)
    for bad in ([g[0]], [g[0], g[1][:19]], [g[0], g[1].float()], [g[0].cpu(), g[1]], [torch.zeros(20, device="cuda")[::2], g[1]]):
        with pytest.raises(ValueError):
            plan.norm(bad)
    for m in (-1.0, float("nan")):
        with pytest.raises(ValueError):
            plan.clip(g, m)
    from conv2d_backward_implicit_bwd_gb300.binding import ConvBwdError
    base = torch.zeros(12, device="cuda")
    with pytest.raises(ConvBwdError):
        plan.clip([base[:10], g[1]], 1.0, out=[base[2:], torch.zeros_like(g[1])])
