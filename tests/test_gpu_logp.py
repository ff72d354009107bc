"""Token log-probabilities, entropy, alternatives and their gradients against the definition in 64 bits.

Tolerances.  A row's sums have relative errors below 2^-20: each argument c (z - m) is off by 2^-23 of itself and of |c z|
(below 256 where z c is taken first), the exponential by 2^-22, the additions of a thread's chunk and of the joins by
2^-22 on sums of one sign.  So logp and lse are off by at most E = 2^-19 (1 + |lse| + |logp|) (roundings of 2^-23 of their
size included) and H, the sum of two terms of one sign that both lie below H + 1 (the reference lies within 2^1 of the
maximum), by 2^-19 (2 + H).  In the gradient u = scale z - lse is off by 2^-23 (|lse| + 2 |u|), which p inherits relatively
beside the exponential's 2^-22: e = 2^-21 (1 + |lse| + |u|); dz is a product of p and gl + ge (u + H) plus the given token's gl,
rounded to the type (half a step, eps / 2)."""
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


def rows_of(t, v, dtype, seed=1, ld=None, shift=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or v
    flat = torch.full((t * ld + shift,), float("nan"), dtype=DT[dtype], device="cuda")
    z = flat[shift:].view(t, ld)[:, :v]
    z.copy_(torch.randn(t, v, generator=g, device="cuda") * spread)
    return z, torch.randint(0, v, (t,), generator=g, device="cuda", dtype=torch.int32)


def check_forward(plan, z, a, scale=1.0):
    logp, h, lse, tlp, tt = out = plan.forward(z, a)
    assert plan.status() == (0, 0)
    live = torch.ones(len(z), dtype=torch.bool, device="cuda") if a is None else a >= 0
    zd = z.double() * scale
    top = zd.amax(1, keepdim=True)
    lse_ = torch.logsumexp(zd - top, 1) + top[:, 0]
    u = zd - lse_[:, None]
    h_ = -torch.special.xlogy(u.exp(), u.exp()).sum(1)
    E = 2.0 ** -19 * (1 + lse_.abs())
    assert ((lse.double() - lse_).abs() <= E)[live].all()
    assert ((h.double() - h_).abs() <= 2.0 ** -19 * (2 + h_))[live].all() and (h >= 0)[live].all()
    if a is not None:
        lp = u.gather(1, a.clamp(min=0).long()[:, None])[:, 0]
        finite = torch.isfinite(lp)
        assert ((logp.double() - lp).abs() <= E + 2.0 ** -19 * lp.abs())[live & finite].all()
        assert (logp[live & ~finite] == -math.inf).all()
    else:
        assert logp is None
    if plan.top:
        order = z.float().sort(dim=1, descending=True, stable=True).indices[:, :plan.top]
        assert torch.equal(tt[live], order[live].int())
        want = u.gather(1, order)
        ok = ~torch.isfinite(want) | ((tlp.double() - want).abs() <= (E[:, None] + 2.0 ** -19 * want.abs()))
        assert ok[live].all() and torch.equal(torch.isinf(tlp)[live], torch.isinf(want)[live])
        assert (tlp[~live] == 0).all() and (tt[~live] == -1).all()
    else:
        assert tlp is None and tt is None
    for t in out[:3]:
        if t is not None:
            assert (t[~live] == 0).all()
    return out


SIZES = [(1, 1), (1, 2), (3, 7), (5, 33), (2, 100), (9, 1009), (40, 4096), (3, 8191), (2, 8192), (3, 8193), (1, 20000), (7, 40001), (1, 128000), (70, 30011), (500, 9000), (1400, 8200)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", SIZES)
@pytest.mark.parametrize("top", [0, 1, 20, 32])
def test_forward(T, dtype, t, v, top):
    top = min(top, v)
    z, a = rows_of(t, v, dtype, seed=t + v)
    a[1::5] = -1
    check_forward(T.TokenLogp(v, dtype, top=top, scale=0.7), z, a, scale=torch.tensor(0.7).item())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("v,ld,shift", [(1000, 1003, 1), (1000, 1000, 3), (9001, 9001, 5), (30000, 30001, 7), (30000, 30008, 0)])
@pytest.mark.parametrize("t", [2, 600])
def test_any_address(T, dtype, v, ld, shift, t):
    z, a = rows_of(t, v, dtype, ld=ld, shift=shift)
    check_forward(T.TokenLogp(v, dtype, top=5), z, a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(3, 50), (4, 3000), (4, 60000), (600, 9000)])
@pytest.mark.parametrize("kind", ["equal", "few values", "rising", "falling", "banned", "signed zeros", "one hot", "wide", "rising groups"])
def test_alternatives_of_hard_rows(T, dtype, t, v, kind):
    hard_rows(T, dtype, t, v, kind, 20)


# rows of up to 32 KB, of which there are enough for a warp each
MANY = [("bf16", 2500, 8200), ("bf16", 2433, 16384), ("bf16", 2500, 11003), ("f32", 2500, 5001), ("f32", 2440, 8192)]


@pytest.mark.parametrize("dtype,t,v", MANY)
@pytest.mark.parametrize("top", [0, 3, 12, 20, 32])
def test_many_rows(T, dtype, t, v, top):
    z, a = rows_of(t, v, dtype, seed=top, ld=v + top % 2, shift=top % 5)
    a[1::5] = -1
    check_forward(T.TokenLogp(v, dtype, top=top), z, a)


@pytest.mark.parametrize("dtype,t,v", MANY[1:4])
@pytest.mark.parametrize("kind", ["equal", "few values", "rising", "falling", "banned", "signed zeros", "one hot", "rising groups"])
@pytest.mark.parametrize("top", [7, 30])
def test_alternatives_of_many_hard_rows(T, dtype, t, v, kind, top):
    hard_rows(T, dtype, t, v, kind, top)


@pytest.mark.parametrize("v", [1024, 1023, 400])
@pytest.mark.parametrize("top", [9, 11, 17, 32])
def test_alternatives_of_short_hard_rows(T, v, top):
    for kind in ("few values", "rising groups", "banned"):
        hard_rows(T, "bf16", 50, v, kind, top)


def hard_rows(T, dtype, t, v, kind, top):
    z, a = rows_of(t, v, dtype)
    i = torch.arange(v, device="cuda").float()
    if kind == "equal":
        z.fill_(1.5)
    elif kind == "few values":
        z.copy_((z * 0.5).round())
    elif kind == "rising":
        z.copy_((i / v * 20).expand(t, v))
    elif kind == "falling":
        z.copy_((-i / v * 20).expand(t, v))
    elif kind == "rising groups":  # each of a block's chunks above all before it
        z.copy_((i // 64).expand(t, v) * 1e-2 + z.float() * 1e-3)
    elif kind == "banned":  # fewer logits left than alternatives
        z[:, 9:] = -math.inf
        a.fill_(3)
    elif kind == "signed zeros":
        z.zero_()
        z[:, ::2] = -0.0
    elif kind == "one hot":
        z[:, v // 2] = 60.0
    elif kind == "wide":  # scale z c above 256: differences are taken first
        z.mul_(300)
    check_forward(T.TokenLogp(v, dtype, top=top), z, a)


@pytest.mark.parametrize("v", [40, 5000, 50000])
def test_without_tokens(T, v):
    z, _ = rows_of(6, v, "bf16")
    check_forward(T.TokenLogp(v, top=4), z, None)


@pytest.mark.parametrize("v", [40, 50000])
def test_rows_that_are_not_distributions(T, v):
    z, a = rows_of(8, v, "f32")
    z[1] = -math.inf
    z[2, 3] = math.nan
    z[3, 5] = math.inf
    z[4] = math.nan
    z[4, 7] = 1.0
    z[5, :] = math.nan
    a[6], a[7] = -1, v
    z[6:] = math.nan  # masked: not read
    plan = T.TokenLogp(v, "f32", top=6)
    logp, h, lse, tlp, tt = plan.forward(z, a)
    assert plan.status()[0] == 6 and plan.status() == (0, 0)
    assert torch.isfinite(logp[0]) and torch.isfinite(h[0])
    for r in (1, 2, 3, 4, 5):
        assert torch.isnan(logp[r]) and torch.isnan(h[r]) and torch.isnan(tlp[r]).all(), r
    assert lse[1] == -math.inf and torch.isnan(lse[2:6]).all()
    assert tt[1].tolist() == [0, 1, 2, 3, 4, 5]
    order = torch.nan_to_num(z[2], nan=-math.inf, posinf=math.inf, neginf=-math.inf).sort(descending=True, stable=True).indices[:6]
    assert torch.equal(tt[2], order.int()) and tt[3, 0] == 5
    assert tt[4].tolist() == [7, -1, -1, -1, -1, -1] and (tt[5] == -1).all()
    for t in (logp, h, lse, tlp):
        assert (t[6:] == 0).all()
    assert (tt[6:] == -1).all()


def gradient(z, a, lse, h, gl, ge, scale):
    live = torch.ones(len(z), dtype=torch.bool, device="cuda") if a is None else (a >= 0) & (a < z.shape[1])
    pick = torch.zeros(z.shape, dtype=torch.float64, device="cuda")
    if a is not None:
        pick[torch.arange(len(z), device="cuda")[live], a[live].long()] = 1
    g = torch.zeros(len(z), device="cuda") if gl is None else gl
    e = torch.zeros(len(z), device="cuda") if ge is None else ge
    g, e = (g.double() * live)[:, None], (e.double() * live)[:, None]
    hd = torch.zeros_like(g) if h is None else h.double()[:, None]
    u = scale * z.double() - lse.double()[:, None]
    p = u.exp()
    u = u.clamp(min=-1e4)
    dz = scale * (g * (pick - p) - e * p * (u + hd))
    size = scale * (p * (g.abs() + e.abs() * (1 + u.abs() + hd)) * 2.0 ** -21 * (1 + lse.double().abs()[:, None] + u.abs()) + g.abs() * pick * 2.0 ** -22)
    return torch.where(live[:, None], dz, 0.0), size


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v,ld,shift", [(1, 1, 0, 0), (5, 33, 0, 0), (9, 1009, 0, 0), (40, 4096, 0, 0), (3, 8193, 0, 0), (7, 40001, 0, 0), (2, 128000, 0, 0), (600, 9000, 9003, 1), (20, 1000, 1001, 3), (2500, 8001, 8003, 1)])
@pytest.mark.parametrize("which", ["both", "logp", "entropy", "in place"])
def test_backward(T, dtype, t, v, ld, shift, which):
    plan = T.TokenLogp(v, dtype, scale=0.7)
    scale = torch.tensor(0.7).item()
    z, a = rows_of(t, v, dtype, ld=ld or None, shift=shift)
    z[:, 2::7] = -math.inf
    a[1::5] = -1
    a[::5] = 0
    _, h, lse, _, _ = plan.forward(z, a)
    g = torch.Generator(device="cuda").manual_seed(3)
    gl, ge = torch.randn(t, generator=g, device="cuda"), torch.randn(t, generator=g, device="cuda")
    gl[2::6] = ge[2::6] = 0
    if which == "logp":
        ge = None
    if which == "entropy":
        gl = None
    want, size = gradient(z, a, lse, h, gl, ge, scale)
    before = z.clone()
    got = plan.backward(z, a, lse, h, grad_logp=gl, grad_entropy=ge, out=z if which == "in place" else None)
    assert plan.status() == (0, 0)
    assert ((got.double() - want).abs() <= size + want.abs() * torch.finfo(DT[dtype]).eps / 2 + 1e-37).all()
    dead = (a < 0) | ((0 if gl is None else gl) + torch.zeros(t, device="cuda") == 0) & ((0 if ge is None else ge) + torch.zeros(t, device="cuda") == 0)
    assert (got[dead] == 0).all()
    if which != "in place":
        assert torch.equal(z, before)


def test_gradient_against_differences(T):
    v, t = 50, 4
    plan = T.TokenLogp(v, "f32", scale=0.7)
    scale = torch.tensor(0.7).item()
    z, a = rows_of(t, v, "f32", spread=1.0)
    gl, ge = torch.tensor([1.0, 0.5, 0.0, -2.0], device="cuda"), torch.tensor([0.3, 0.0, 1.0, 0.7], device="cuda")
    _, h, lse, _, _ = plan.forward(z, a)
    got = plan.backward(z, a, lse, h, grad_logp=gl, grad_entropy=ge)

    def f(zd):
        u = torch.log_softmax(scale * zd, 1)
        return (gl * u.gather(1, a.long()[:, None])[:, 0] - ge * (u.exp() * u).sum(1)).sum()
    zd, eps = z.double(), 1e-4
    for r in range(t):
        for k in range(0, v, 7):
            step = torch.zeros_like(zd)
            step[r, k] = eps
            slope = float((f(zd + step) - f(zd - step)) / (2 * eps))
            # central differences: eps^2 / 6 of the third derivative (below 10 here) and 1e-15 / eps of rounding
            assert abs(float(got[r, k]) - slope) <= 2e-7 + 2.0 ** -17 * (1 + abs(slope))


def test_same_bits_every_time(T):
    z, a = rows_of(5, 100003, "bf16")
    plan = T.TokenLogp(100003, top=20)
    first = plan.forward(z, a)
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(first, plan.forward(z, a)))


def test_empty(T):
    plan = T.TokenLogp(10, top=3)
    z, a = torch.empty(0, 10, dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    assert [tuple(t.shape) for t in plan.forward(z, a)] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    e = torch.empty(0, device="cuda")
    assert plan.backward(z, a, e, e, grad_logp=e, grad_entropy=e).shape == (0, 10)


@pytest.mark.parametrize("t,v", [(3, 60000), (20, 2000)])
def test_captured(T, t, v):
    plan = T.TokenLogp(v, top=7)
    z, a = rows_of(t, v, "bf16")
    g = torch.ones(t, device="cuda")

    def step():
        out = plan.forward(z, a)
        return [*out, plan.backward(z, a, out[2], out[1], grad_logp=g, grad_entropy=g)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (5, 6, 7):
        nz, na = rows_of(t, v, "bf16", seed=seed)
        z.copy_(nz)
        a.copy_(na)
        graph.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in out]
        assert all(torch.equal(x, y) for x, y in zip(kept, step()))
    assert plan.status() == (0, 0)


def test_written_just_before(T):
    """Launches begin while the kernel before them still runs: inputs and the plan's workspace are read as written."""
    plan = T.TokenLogp(60000, top=7)
    sets = [rows_of(3, 60000, "bf16", seed=s) for s in range(6)]
    want = [[t.clone() for t in plan.forward(z, a)] for z, a in sets]
    torch.cuda.synchronize()
    z, a = (t.clone() for t in sets[0])
    got = []
    for nz, na in sets * 4:
        z.copy_(nz)
        a.copy_(na)
        got.append(plan.forward(z, a))
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 6]))


def test_new_plan_on_an_unordered_stream(T):
    z, a = rows_of(3, 60000, "bf16")
    want = T.TokenLogp(60000, top=7).forward(z, a)
    streams, kept = [torch.cuda.Stream() for _ in range(3)], []
    torch.cuda.synchronize()
    for s in streams:
        torch.cuda._sleep(100_000_000)
        plan = T.TokenLogp(60000, top=7)
        kept.append(plan)
        for _ in range(2):
            got = plan.forward(z, a, stream=s)
        s.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and plan.status(stream=s) == (0, 0)
        torch.cuda.synchronize()


def test_versions(T):
    plan = T.TokenLogp(9, "f32")
    z, a, f = torch.ones(4, 9, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
    out = torch.empty_like(z)
    plan.forward(z, a)
    plan.backward(z, a, f, f, grad_logp=f, out=out)
    assert z._version == 0 and a._version == 0 and f._version == 0 and out._version == 1


def test_long_rows_offsets_past_32_bits(T):
    """Rows whose elements lie past 2^31."""
    v, t = 1 << 20, 2100
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("memory")
    z = torch.zeros(t, v, dtype=torch.bfloat16, device="cuda")
    z[-1, -3:] = torch.tensor([1.0, 3.0, 2.0])
    a = torch.full((t,), -1, dtype=torch.int32, device="cuda")
    a[-1] = v - 2
    out = T.TokenLogp(v, top=4).forward(z, a)
    assert out[4][-1].tolist() == [v - 2, v - 1, v - 3, 0] and (out[4][:-1] == -1).all()
    want = 3.0 - math.log(v - 3 + math.exp(1) + math.exp(3) + math.exp(2))
    assert abs(float(out[0][-1]) - want) <= 2.0 ** -19 * (1 + 2 * abs(want))
