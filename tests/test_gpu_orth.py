"""Orthogonalised updates against the iteration in 64 bits.

Tolerance.  A step's products are off by less than 2^-20 of their factors' size each (operands of 22 bits, a lost third term
of 2^-24, at most 24 truncations of 2^-25 in one accumulator, fp32 sums), so X' = (a I + b A + c A^2) X by less than
(|a| + 2 |b| + 3 |c|) 2^-20 |X|_F where singular values stay below 1.3 (A below 1.7: each |A| here counts with it in the two
or three products that make it: 2 * 1.7, 3 * 2.9 at most).  A later step multiplies an error by at most
L = max |p'|, |p(s) / s| = a (p(s) = a s + b s^3 + c s^5, the usual coefficients).  So after T steps the error is below
D = sum_k L^(T-1-k) (|a| + 3.4 |b| + 8.7 |c|) 2^-20 |X_k|_F, which the test sums over the iterates in 64 bits; a result in bf16 adds half a step of each
element, the norm at the start 2^-23.  (One product of fp16 or bf16 operands each would be off by 2^8 to 2^11 times as much.)

Results in bf16 come of accumulators with 96 truncations, which is D's 2^-20 in the steps before the last 2^-18 instead, and of
a last product B X of fp16 operands alone, off by 2^-12 (|B|_F |X|_2 + |B|_2 |X|_F) < 2^-9.2 |X'|_F in the worst case (|B| < 3.5,
|X|_2 < 1.3).  They have no room of their own: rounding to the nearest bf16 is off by 0.42 half steps in the root mean square (uniform
within the half step, which is 2^-9 to 2^-8 of an element), the two together by less than 0.65 of the half step that is given.

Where the larger side is twice the smaller one, three steps are one polynomial of the Gram matrix; they are held to the D of
steps apart."""
import math

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


DT = {"f32": torch.float32, "bf16": torch.bfloat16}
COEF = (3.4445, -4.7750, 2.0315)


def matrices(shape, kind="falling", seed=1, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    b, m, n = shape
    x = torch.randn(b, m, n, generator=g, device="cuda")
    if kind == "falling":
        r = min(16, m, n)
        x = torch.bmm(torch.randn(b, m, r, generator=g, device="cuda") * torch.exp(-0.3 * torch.arange(r, device="cuda")), torch.randn(b, r, n, generator=g, device="cuda")) + 0.1 * x
    return x.to(dtype)


def iterate(u, coefs):
    """X and the tolerance D, each matrix apart."""
    x = u.double() / torch.linalg.matrix_norm(u.double())[:, None, None]
    off = torch.full((len(u),), 2.0 ** -23, dtype=torch.float64, device="cuda")
    for a, b, c in coefs:
        high = x.shape[1] > x.shape[2]
        s = x.transpose(1, 2) @ x if high else x @ x.transpose(1, 2)
        p = a * torch.eye(s.shape[1], dtype=s.dtype, device="cuda") + b * s + c * (s @ s)
        off = max(abs(a), 1.0) * off + (abs(a) + 3.4 * abs(b) + 8.7 * abs(c)) * 2.0 ** -20 * torch.linalg.matrix_norm(x)
        x = x @ p if high else p @ x
    return x, off


def check(got, x, off, what=""):
    diff = torch.linalg.matrix_norm(got.double() - x)
    room = off + (torch.finfo(got.dtype).eps / 2 * torch.linalg.matrix_norm(x))
    assert (diff <= room).all(), (what, (diff / room).max())
    return float((diff / torch.linalg.matrix_norm(x)).max())


SHAPES = [(1, 1, 1), (1, 1, 7), (2, 9, 1), (3, 8, 8), (1, 31, 33), (1, 100, 131), (2, 131, 100), (1, 256, 256), (2, 257, 300), (1, 300, 513), (5, 64, 1000),
          (3, 1000, 64), (1, 1000, 1000), (90, 40, 70), (20, 300, 512), (20, 512, 300), (1, 200, 4096), (2, 2100, 130), (40, 513, 520)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("kind", ["falling", "flat"])
def test_apply(T, dtype, shape, kind):
    u = matrices(shape, kind, dtype=DT[dtype])
    plan = T.Orthogonal(*shape, dtype)
    before = u.clone()
    got = plan.apply(u)
    assert plan.status() == (0, 0) and torch.equal(u, before)
    print(shape, dtype, kind, check(got, *iterate(u, [COEF] * 5)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 128, 256), (1, 128, 257), (3, 100, 260), (2, 17, 520), (1, 128, 1000), (2, 1, 1024), (3, 128, 2048), (2, 2048, 128), (2, 700, 33), (1, 1100, 128),
                                   (1, 129, 256), (1, 128, 2049), (200, 128, 300), (300, 20, 16)])
def test_either_side_of_the_small_kernel(T, dtype, shape):
    """Smaller sides up to 128 and larger ones up to 2048, in slices of 256 columns."""
    u = matrices(shape, dtype=DT[dtype])
    plan = T.Orthogonal(*shape, dtype)
    check(plan.apply(u), *iterate(u, [COEF] * 5))
    assert plan.status() == (0, 0)


def test_singular_values(T):
    """They come near 1 and the vectors stay: the point of it."""
    u = matrices((1, 96, 160), "flat")
    s = torch.linalg.svdvals(T.Orthogonal(1, 96, 160, "f32").apply(u)[0].double())
    assert 0.6 < float(s.min()) and float(s.max()) < 1.3


@pytest.mark.parametrize("coefs", [[(1.5, -0.5, 0.0)] * 9, [(8.2, -23.0, 16.0), (4.0, -2.9, 0.5), (1.875, -1.25, 0.375)], [(1.0, 0.0, 0.0)], [(0.0, 1.0, 0.0)], [(0.0, 0.0, 1.0)], [(-2.0, 0.5, 0.0)]])
@pytest.mark.parametrize("shape", [(2, 70, 300), (2, 300, 70)])
def test_coefficients(T, coefs, shape):
    u = matrices(shape, "flat")
    plan = T.Orthogonal(*shape, "f32", steps=len(coefs), coefficients=coefs)
    x, off = iterate(u, coefs)
    # (a later step multiplies an error by at most |a| + 3 |b| s^2 + 5 |c| s^4, s below 1.3)
    grow = max(1.0, max(abs(a) + 5.1 * abs(b) + 14.3 * abs(c) for a, b, c in coefs)) if len(coefs) == 3 else 1.0
    check(plan.apply(u), x, off * grow ** 2)


# the larger side at least twice the smaller one, or not quite
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 150, 300), (2, 150, 299), (3, 1300, 200), (1, 257, 2000), (30, 300, 1024), (30, 1100, 520), (1, 3000, 1400), (2, 130, 5000), (90, 300, 375), (90, 380, 300)])
@pytest.mark.parametrize("kind", ["falling", "flat"])
def test_steps_joined_in_one_polynomial(T, dtype, shape, kind):
    """Held to what steps apart are held to."""
    x = matrices(shape, kind, 3, DT[dtype])
    plan = T.Orthogonal(*shape, dtype)
    check(plan.apply(x), *iterate(x, [COEF] * 5), shape)
    assert plan.status() == (0, 0)


@pytest.mark.parametrize("shape", [(2, 200, 450), (1, 1500, 300), (20, 300, 700)])
@pytest.mark.parametrize("rank,noise", [(1, 0.0), (3, 0.0), (8, 1e-2), (8, 1e-3), (8, 1e-5), (2, 1e-1)])
def test_joined_steps_beside_few_directions(T, shape, rank, noise):
    """Small singular values, which the Gram matrix holds as squares."""
    g = torch.Generator(device="cuda").manual_seed(rank)
    b, m, n = shape
    u = torch.randn(b, m, rank, generator=g, device="cuda") @ torch.randn(b, rank, n, generator=g, device="cuda")
    e = torch.randn(shape, generator=g, device="cuda")
    u = u / torch.linalg.matrix_norm(u)[:, None, None] + noise * e / torch.linalg.matrix_norm(e)[:, None, None]
    check(T.Orthogonal(*shape, "f32").apply(u), *iterate(u, [COEF] * 5))
    check(T.Orthogonal(*shape, "bf16").apply(u.bfloat16()), *iterate(u.bfloat16(), [COEF] * 5))


@pytest.mark.parametrize("shape", [(2, 160, 400), (2, 700, 140), (40, 260, 530)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 7, 12])
def test_any_number_of_joined_steps(T, shape, steps):
    x = matrices(shape, "falling", 5)
    check(T.Orthogonal(*shape, "f32", steps).apply(x), *iterate(x, [COEF] * steps))


@pytest.mark.parametrize("coefs", [[(1.5, -0.5, 0.0)] * 9, [(8.2, -23.0, 16.0), (4.0, -2.9, 0.5), (1.875, -1.25, 0.375)], [(4.0, -6.0, 3.0)] * 3, [(0.0, 0.0, 6.0)] * 3, [(4.0, 6.0, 6.0), (1.0, 0.0, 0.0), (0.5, 0.0, 0.0)],
                                   [(2.0, -1.5, 0.5), (0.0, 1.0, 0.0), (-2.0, 0.5, 0.0), (3.0, -3.2, 1.2)]])
@pytest.mark.parametrize("shape", [(2, 140, 300), (2, 300, 140)])
def test_coefficients_of_joined_steps(T, coefs, shape):
    """Large ones, and ones whose products would leave the planes' range, among them: those steps go apart."""
    x = matrices(shape, "flat", 7)
    plan = T.Orthogonal(*shape, "f32", len(coefs), coefs)
    check(plan.apply(x), *iterate(x, coefs))
    assert plan.status() == (0, 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(3, 100, 132), (2, 300, 140), (1, 5, 3)])
@pytest.mark.parametrize("pad,shift", [(0, 1), (3, 0), (8, 0), (4, 4)])
def test_strides(T, dtype, shape, pad, shift):
    b, m, n = shape
    u = matrices(shape, dtype=DT[dtype])

    def padded(fill):
        flat = torch.full((b * (m + 2) * (n + pad) + shift,), fill, dtype=DT[dtype], device="cuda")
        return flat, flat[shift:].view(b, m + 2, n + pad)[:, :m, :n]
    _, x = padded(math.nan)
    x.copy_(u)
    flat, out = padded(5.0)
    plan = T.Orthogonal(*shape, dtype)
    assert plan.apply(x, out=out) is out and plan.status() == (0, 0)
    assert torch.equal(out, plan.apply(u))
    out.fill_(5.0)
    assert (flat == 5.0).all()  # nothing beside it was written
    plan.apply(x, out=x)
    assert torch.equal(x, plan.apply(u))


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-12, 1e12, 1e30, 3e36])
def test_scales(T, scale):
    """X does not depend on u's size, near the ends of fp32 either.  (Powers of two: the bits of u stay, but below 2^-126.)"""
    u = matrices((2, 60, 90), "flat").clamp(-4, 4)
    power = 2.0 ** round(math.log2(scale))
    scaled = u * power
    plan = T.Orthogonal(2, 60, 90, "f32")
    check(plan.apply(scaled), *iterate(scaled.double() / power, [COEF] * 5))


def test_zero_and_broken_matrices(T):
    u = matrices((6, 300, 200))
    plan = T.Orthogonal(6, 300, 200, "f32")
    want = plan.apply(u)
    v = u.clone()
    v[1] = 0
    v[2, 7, 9] = math.nan
    v[3, 0, 0] = math.inf
    v[4] = -0.0
    got = plan.apply(v)
    assert (got[1] == 0).all() and (got[4] == 0).all()
    assert torch.isnan(got[2]).all() and torch.isnan(got[3]).all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[5], want[5])
    assert torch.equal(plan.apply(u), want) and plan.status() == (0, 0)


def test_norm_of_equal_elements(T):
    """Squares of 1 + 0.45 * 2^-14 lose 0.45 * 2^-14 with each addition to a sum of 512 to 1024 of them, all one way: 2^-17 of the
    norm of these matrices, whose threads add 978 each.  One step with (1, 0, 0) is u / |u|; room for operands of 22 bits, the
    sum's and the root's roundings."""
    c = 1 + 0.9 * 2.0 ** -16
    u = torch.full((304, 1000, 1001), c, device="cuda")
    u[:, 1::2] = -c
    x = T.Orthogonal(304, 1000, 1001, "f32", steps=1, coefficients=(1.0, 0.0, 0.0)).apply(u)
    assert (x.abs() * 1001000 ** 0.5 - 1).abs().max() <= 2.0 ** -20


def test_low_rank(T):
    """Directions that the matrix lacks stay out of the result but for rounding."""
    g = torch.Generator(device="cuda").manual_seed(2)
    u = torch.randn(2, 200, 3, generator=g, device="cuda") @ torch.randn(2, 3, 333, generator=g, device="cuda")
    check(T.Orthogonal(2, 200, 333, "f32").apply(u), *iterate(u, [COEF] * 5))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 100, 131), (3, 300, 140), (2, 64, 1000), (90, 33, 40), (1, 7, 1)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("pad", [0, 5])
def test_update(T, dtype, shape, nesterov, pad):
    b, m, n = shape
    wide = matrices((b, m, n + pad), dtype=DT[dtype])
    g = wide[:, :, :n]
    mom, w = matrices(shape, seed=2), matrices(shape, "flat", seed=3)
    copy = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    lr, beta, decay, scale = 0.1, 0.9, 0.3, max(1.0, m / n) ** 0.5
    f = lambda v: float(torch.tensor(v))  # noqa: E731  (as the library has them)
    m1 = f(beta) * mom.double() + g.double()
    u = g.double() + f(beta) * m1 if nesterov else m1
    x, off = iterate(u, [COEF] * 5)
    want = w.double() * (1 - lr * decay) - lr * scale * x
    plan = T.Orthogonal(*shape, dtype)
    before = wide.clone()
    w0, versions = w.clone(), (w._version, mom._version, copy._version, g._version)
    assert plan.update(w, g, mom, lr, beta=beta, nesterov=nesterov, decay=decay, copy=copy) is None
    assert plan.status() == (0, 0) and torch.equal(wide, before)
    assert (w._version, mom._version, copy._version, g._version) == tuple(v + (i < 3) for i, v in enumerate(versions))
    assert ((mom.double() - m1).abs() <= 2.0 ** -24 * m1.abs() + 1e-45).all()  # one rounding
    # u is rounded once or twice (2^-24 of its terms), the factors of the step and the step itself three times
    terms = torch.linalg.matrix_norm(g.double().abs() + 2 * mom.double().abs()) / torch.linalg.matrix_norm(u)
    room = lr * scale * (off + 200 * 2.0 ** -23 * terms) + 4 * 2.0 ** -24 * (torch.linalg.matrix_norm(w0.double()) + lr * scale * torch.linalg.matrix_norm(x))
    assert (torch.linalg.matrix_norm(w.double() - want) <= room).all()
    assert torch.equal(copy, w.bfloat16())
    again = w.clone()
    plan.update(w, g, mom, 0.0)
    assert torch.equal(w, again)  # without a copy; a rate of 0 moves nothing


def test_same_bits_every_time(T):
    for shape in [(1, 1000, 700), (40, 200, 300)]:
        u, plan = matrices(shape, dtype=torch.bfloat16), T.Orthogonal(*shape)
        first = plan.apply(u)
        for _ in range(10):
            assert torch.equal(first, plan.apply(u))


def test_one_matrix_and_many(T):
    """A matrix's result is near the same in a batch of any size (other tiles add in another order)."""
    u = matrices((80, 300, 260))
    many, one = T.Orthogonal(80, 300, 260, "f32").apply(u), T.Orthogonal(1, 300, 260, "f32")
    x, off = iterate(u[:2], [COEF] * 5)
    for i in range(2):
        check(many[i:i + 1], x[i:i + 1], off[i:i + 1])
        check(one.apply(u[i:i + 1]), x[i:i + 1], off[i:i + 1])


def test_captured(T):
    shape = (2, 300, 200)
    plan, seen = T.Orthogonal(*shape), []
    w, mom, g, copy = matrices(shape, seed=5), matrices(shape, seed=6), matrices(shape, seed=7, dtype=torch.bfloat16), torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
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
        for i in range(4):
            g.copy_(matrices(shape, seed=20 + i, dtype=torch.bfloat16))
            if replay:
                graph.replay()
            else:
                plan.update(w, g, mom, 0.1, copy=copy)
        seen.append([t.clone() for t in (w, mom, copy)])
    assert all(torch.equal(a, b) for a, b in zip(*seen)) and plan.status() == (0, 0)


def test_written_just_before(T):
    shape = (2, 300, 200)
    plan = T.Orthogonal(*shape)
    sets = [matrices(shape, seed=s, dtype=torch.bfloat16) for s in range(5)]
    want = [plan.apply(u) for u in sets]
    torch.cuda.synchronize()
    x, got = torch.empty_like(sets[0]), []
    for u in sets * 4:
        x.copy_(u)
        got.append(plan.apply(x))
    assert all(torch.equal(g, want[i % 5]) for i, g in enumerate(got))


def test_two_plans_on_two_streams(T):
    shape = (3, 400, 300)
    u = matrices(shape, dtype=torch.bfloat16)
    want = T.Orthogonal(*shape).apply(u)
    torch.cuda.synchronize()
    plans, streams = [T.Orthogonal(*shape) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    got = [plan.apply(u, stream=s) for _ in range(5) for plan, s in zip(plans, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_new_plan_on_an_unordered_stream(T):
    shape = (2, 100, 90)
    u = matrices(shape, dtype=torch.bfloat16)
    want = T.Orthogonal(*shape).apply(u)
    streams, kept = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for s in streams:
        torch.cuda._sleep(100_000_000)
        plan = T.Orthogonal(*shape)
        kept.append(plan)
        got = plan.apply(u, stream=s)
        s.synchronize()
        assert torch.equal(got, want) and plan.status(stream=s) == (0, 0)
        torch.cuda.synchronize()
