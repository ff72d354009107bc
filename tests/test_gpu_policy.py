"""Clipped policy loss with a KL term against the definition in 64 bits.

Tolerances: a row's sum of V exponentials has a relative error below
2^-20 (each factor: argument off by |z| 2^-23, the exponential by 2^-22, the
running rescales and the additions of a thread's chunk below 2^-21 on the
positive sum), logp and lse add roundings of 2^-23 of their size: E = 2^-19 (1 +
|lse| + |logp|).  r and exp(d) inherit E relatively; dlogits are
coef scale (onehot - p): E relative to (onehot + p) plus the type's rounding."""
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
LO, HI = 0.2, 0.3


def inputs(t, v, dtype, seed=1, ld=None, shift=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld = ld or v
    flat = torch.full((t * ld + shift,), float("nan"), dtype=DT[dtype], device="cuda")
    z = flat[shift:].view(t, ld)[:, :v]
    z.copy_(torch.randn(t, v, generator=g, device="cuda") * spread)
    a = torch.randint(0, v, (t,), generator=g, device="cuda", dtype=torch.int32)
    adv = torch.randn(t, generator=g, device="cuda")
    w = torch.rand(t, generator=g, device="cuda") / max(t, 1)
    lp = torch.log_softmax(z.float(), 1).gather(1, a[:, None].long())[:, 0] if t else adv
    old = lp + 0.3 * torch.randn(t, generator=g, device="cuda")
    ref = lp + 0.3 * torch.randn(t, generator=g, device="cuda")
    return z, a, adv, w, old, ref


def reference(z, a, adv, w, old, ref, kl, scale, grad=1.0, lo=LO, hi=HI):
    z = z.double() * scale
    adv, w = adv.double(), w.double()
    top = z.amax(1, keepdim=True)
    z = z - torch.where(torch.isfinite(top), top, 0.0)  # exact for fp32 logits of any size
    lse = torch.logsumexp(z, 1)
    pick = torch.zeros_like(z)
    pick[torch.arange(len(a), device="cuda"), a.long()] = 1
    logp = z.gather(1, a[:, None].long())[:, 0] - lse
    r = torch.exp(logp - old.double()) if old is not None else torch.ones_like(logp)
    held = r.clamp(1 - lo, 1 + hi)
    free = r * adv <= held * adv
    l = -torch.where(free, r * adv, held * adv)
    c = torch.where(free, -r * adv, 0.0)
    if ref is not None:
        d = ref.double() - logp
        l = l + kl * (torch.expm1(d) - d)
        c = c - kl * torch.expm1(d)
    dz = grad * (w * c * scale)[:, None] * (pick - torch.exp(z - lse[:, None]))
    return dict(loss=(w * l).sum(), terms=(w * l).abs().sum(), logp=logp, lse=lse + torch.where(torch.isfinite(top), top, 0.0)[:, 0], coef=w * c, dz=dz, pick=pick,
                p=torch.exp(z - lse[:, None]), r=r)


def near_edge(ref, old):
    """Tokens whose ratio is within rounding of a clip bound: either branch is right."""
    r = ref["r"]
    return ((r - (1 - LO)).abs() < 1e-4) | ((r - (1 + HI)).abs() < 1e-4) if old is not None else torch.zeros_like(r, dtype=torch.bool)


def check(got, ref, kl, scale, adv, w, old, dtype, grad=1.0):
    E = 2.0 ** -19 * (1 + ref["lse"].abs() + ref["logp"].abs())
    ok = ~near_edge(ref, old)
    size = w.double() * (adv.double().abs() * ref["r"] + kl * (2 + 2 * ref["r"]) * 4)
    if "logp" in got:
        assert ((got["logp"].double() - ref["logp"]).abs() <= E).all()
    if "lse" in got:
        assert ((got["lse"].double() - ref["lse"]).abs() <= E).all()
    if "coef" in got:
        assert ((got["coef"].double() - ref["coef"]).abs() <= 2 * E * size + 1e-30)[ok].all()
    if "loss" in got:
        assert abs(float(got["loss"]) - float(ref["loss"])) <= float((2 * E * size).sum()) + 2.0 ** -22 * float(ref["terms"]) + 1e-30
    if "dz" in got:
        rnd = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22
        tol = rnd * ref["dz"].abs() + 3 * grad * scale * (E * size)[:, None] * (ref["pick"] + ref["p"]) + 1e-30
        bad = ~((got["dz"].double() - ref["dz"]).abs() <= tol) & ok[:, None]
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}"


def run_all(T, t, v, dtype, kl=0.05, scale=0.7, old=True, ref=True, ld=None, shift=0, seed=1):
    z, a, adv, w, o, f = inputs(t, v, dtype, seed=seed, ld=ld, shift=shift)
    o, f = (o if old else None), (f if ref else None)
    plan = T.PolicyLoss(v, dtype, clip_low=LO, clip_high=HI, kl=kl, scale=scale)
    want = reference(z, a, adv, w, o, f, kl, scale)
    loss, logp, lse, coef = plan.forward(z, a, adv, w, o, f)
    check(dict(loss=loss, logp=logp, lse=lse, coef=coef), want, kl, scale, adv, w, o, dtype)
    g = torch.tensor([1.5], device="cuda")
    dz = plan.backward(z, a, lse, coef, grad=g)
    want15 = reference(z, a, adv, w, o, f, kl, scale, grad=1.5)
    check(dict(dz=dz), want15, kl, scale, adv, w, o, dtype, grad=1.5)
    loss2, logp2, dz2 = plan.forward_backward(z, a, adv, w, o, f)
    assert torch.equal(loss2, loss) and torch.equal(logp2, logp)
    check(dict(dz=dz2), want, kl, scale, adv, w, o, dtype)
    assert plan.status() == (0, 0)
    return plan, (z, a, adv, w, o, f), (loss, logp, lse, coef, dz2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,v", [(1, 1), (1, 2), (5, 7), (33, 100), (300, 1000), (64, 1024), (3, 1025), (40, 4099), (17, 32000), (700, 8192)])
def test_sizes(T, dtype, t, v):
    run_all(T, t, v, dtype)


@pytest.mark.parametrize("dtype,v", [("bf16", 131073), ("f32", 100003), ("bf16", 262144)])
def test_wide_vocabularies(T, dtype, v):
    run_all(T, 3, v, dtype)


@pytest.mark.parametrize("old,ref,kl", [(False, False, 0.0), (False, True, 0.1), (True, False, 0.1), (True, True, 0.0)])
def test_left_out_terms(T, old, ref, kl):
    run_all(T, 50, 333, "f32", kl=kl, old=old, ref=ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v,ld,shift", [(1000, 1008, 0), (1000, 1001, 3), (5000, 5003, 1), (4096, 4104, 4), (20000, 20001, 0)])
def test_strides_and_alignment(T, dtype, v, ld, shift):
    """Rows that start at any element; what lies between them is not touched."""
    plan, (z, a, adv, w, o, f), (_, _, lse, coef, dz) = run_all(T, 9, v, dtype, ld=ld, shift=shift)
    out = torch.full((9, ld + 2), 7.0, dtype=DT[dtype], device="cuda")
    plan.forward_backward(z, a, adv, w, o, f, out=out[:, 1:v + 1])
    check(dict(dz=out[:, 1:v + 1]), reference(z, a, adv, w, o, f, 0.05, 0.7), 0.05, 0.7, adv, w, o, dtype)
    assert (out[:, 0] == 7).all() and (out[:, v + 1:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [100, 5001, 70000])
def test_in_place(T, dtype, v):
    plan, (z, a, adv, w, o, f), (_, _, lse, coef, dz) = run_all(T, 20, v, dtype)
    y = z.clone()
    out = plan.forward_backward(y, a, adv, w, o, f, out=y)[2]
    assert out.data_ptr() == y.data_ptr() and torch.equal(y, dz)
    y = z.clone()
    want = plan.backward(z, a, lse, coef)
    assert torch.equal(plan.backward(y, a, lse, coef, out=y), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [50, 3001])
def test_masked_tokens(T, dtype, v):
    """Weight 0 or a negative action: nothing of the row is used, not even NaN, and its outputs are 0."""
    z, a, adv, w, o, f = inputs(12, v, dtype)
    plan = T.PolicyLoss(v, dtype, clip_low=LO, clip_high=HI, kl=0.1)
    keep = torch.ones(12, dtype=torch.bool, device="cuda")
    keep[[0, 3, 7, 11]] = False
    clean = plan.forward_backward(z, a, adv, w * keep, o, f)
    w[[0, 3]] = 0
    a[[7, 11]] = -100
    for x in (z, adv, o, f):
        x[~keep] = float("nan")
    loss, logp, lse, coef = plan.forward(z, a, adv, w, o, f)
    _, logp2, dz = plan.forward_backward(z, a, adv, w, o, f)
    assert torch.equal(logp[keep], clean[1][keep]) and torch.equal(dz[keep], clean[2][keep])
    assert abs(float(loss) - float(clean[0])) <= 2.0 ** -22 * float(clean[0].abs() + 1e-3)
    for x in (logp, lse, coef, logp2, dz, plan.backward(z, a, lse, coef)):
        assert (x[~keep] == 0).all()
    assert plan.status() == (0, 0)
    w.zero_()
    loss, _, dz = plan.forward_backward(z, a, adv, w, o, f)
    assert float(loss) == 0 and (dz == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [64, 2500])
def test_masked_vocabulary(T, dtype, v):
    """-inf and the type's lowest value among the logits: probability 0 and gradient 0 there; infinite sums stay away."""
    z, a, adv, w, o, f = inputs(8, v, dtype)
    low = torch.finfo(DT[dtype]).min
    z[:, ::2] = -math.inf
    z[4:, ::2] = low
    z[2, :] = -math.inf
    z[2, 1] = 3.0                      # one entry left
    a.copy_(torch.full((8,), 1))
    plan = T.PolicyLoss(v, dtype, clip_low=LO, clip_high=HI, kl=0.1)
    o = f = torch.log_softmax(z.float(), 1)[:, 1] + 0.1
    want = reference(z, a, adv, w, o, f, 0.1, 1.0)
    want["dz"] = torch.where(torch.isnan(want["dz"]), 0.0, want["dz"])
    loss, logp, lse, coef = plan.forward(z, a, adv, w, o, f)
    check(dict(loss=loss, logp=logp, lse=lse, coef=coef), want, 0.1, 1.0, adv, w, o, dtype)
    dz = plan.forward_backward(z, a, adv, w, o, f)[2]
    check(dict(dz=dz), want, 0.1, 1.0, adv, w, o, dtype)
    check(dict(dz=plan.backward(z, a, lse, coef)), want, 0.1, 1.0, adv, w, o, dtype)
    assert (dz[:, ::2] == 0).all() and float(logp[2]) == 0


@pytest.mark.parametrize("v", [64, 2500])
def test_rows_without_a_distribution(T, v):
    """All -inf, +inf or NaN: NaN in that row's logp, in the loss and in its gradient; other rows keep theirs."""
    for bad in (-math.inf, math.inf, math.nan):
        z, a, adv, w, o, f = inputs(6, v, "f32")
        plan = T.PolicyLoss(v, "f32", clip_low=LO, clip_high=HI, kl=0.1)
        clean = plan.forward_backward(z, a, adv, w, o, f)
        z[2] = bad
        for old in (o, None):
            loss, logp, dz = plan.forward_backward(z, a, adv, w, old, f if old is not None else None)
            assert math.isnan(float(loss)) and math.isnan(float(logp[2])) and torch.isnan(dz[2]).any()
        loss, logp, dz = plan.forward_backward(z, a, adv, w, o, f)
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(logp[keep], clean[1][keep]) and torch.equal(dz[keep], clean[2][keep])


def test_large_logits(T):
    """Sums far from 0 neither overflow nor vanish."""
    for shift in (3e4, -3e4, 1e30):
        z, a, adv, w, o, f = inputs(5, 700, "f32")
        z = z + shift
        plan = T.PolicyLoss(700, "f32", clip_low=LO, clip_high=HI)
        loss, logp, lse, coef = plan.forward(z, a, adv, w)
        want = reference(z, a, adv, w, None, None, 0.0, 1.0)
        assert ((logp.double() - want["logp"]).abs() <= 2.0 ** -19 * (1 + want["logp"].abs())).all()
        assert torch.isfinite(loss).all()


@pytest.mark.parametrize("v", [30, 4000])
def test_action_out_of_range(T, v):
    from conv2d_backward_implicit_bwd_gb300 import binding as B
    z, a, adv, w, o, f = inputs(6, v, "f32")
    a[4] = v
    plan = T.PolicyLoss(v, "f32", clip_low=LO, clip_high=HI)
    loss, logp, dz = plan.forward_backward(z, a, adv, w, o, f)
    assert plan.status()[0] == B.ERR_DEVICE_FAULT and plan.status() == (0, 0)
    assert float(logp[4]) == 0 and (dz[4] == 0).all() and math.isfinite(float(loss))


def test_gradient_against_differences(T):
    """Central differences of the 64-bit loss, step 1e-5: truncation 1e-10, rounding 1e-11 relative to terms of order 1."""
    t, v, kl, scale = 6, 9, 0.3, 0.9
    z, a, adv, w, o, f = inputs(t, v, "f32", seed=4)
    plan = T.PolicyLoss(v, "f32", clip_low=LO, clip_high=HI, kl=kl, scale=scale)
    dz = plan.forward_backward(z, a, adv, w, o, f)[2].double()
    ref = reference(z, a, adv, w, o, f, kl, scale)
    assert not near_edge(ref, o).any()
    h = 1e-5
    for i in range(t):
        for j in range(v):
            up, dn = z.double(), z.double()
            up[i, j] += h
            dn[i, j] -= h
            d = (reference(up, a, adv, w, o, f, kl, scale)["loss"] - reference(dn, a, adv, w, o, f, kl, scale)["loss"]) / (2 * h)
            assert abs(float(dz[i, j] - d)) <= 1e-6


def test_no_tokens(T):
    plan = T.PolicyLoss(10, "f32")
    e = torch.empty(0, device="cuda")
    z, a = torch.empty(0, 10, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    loss, logp, dz = plan.forward_backward(z, a, e, e)
    assert float(loss) == 0 and logp.shape == (0,) and dz.shape == (0, 10)
    assert plan.backward(z, a, e, e).shape == (0, 10)


def test_same_bits_and_graph(T):
    z, a, adv, w, o, f = inputs(900, 3000, "bf16")
    plan = T.PolicyLoss(3000, clip_low=LO, clip_high=HI, kl=0.1)
    first = plan.forward_backward(z, a, adv, w, o, f)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(first, plan.forward_backward(z, a, adv, w, o, f)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = plan.forward_backward(z, a, adv, w, o, f, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(first, side))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, logp, lse, coef = plan.forward(z, a, adv, w, o, f)
        dz = plan.backward(z, a, lse, coef)
    for seed in (1, 2):
        z.copy_(inputs(900, 3000, "bf16", seed=seed)[0])
        graph.replay()
        torch.cuda.synchronize()
        want = plan.forward(z, a, adv, w, o, f)
        assert torch.equal(loss, want[0]) and torch.equal(dz, plan.backward(z, a, want[2], want[3]))


def test_refusals(T):
    z, a, adv, w, o, f = inputs(4, 20, "f32")
    plan = T.PolicyLoss(20, "f32")
    for g in (lambda: plan.forward(z[:, :19], a, adv, w), lambda: plan.forward(z.bfloat16(), a, adv, w),
              lambda: plan.forward(z, a.long(), adv, w), lambda: plan.forward(z, a[:3], adv, w),
              lambda: plan.forward(z, a, adv.double(), w), lambda: plan.forward(z, a, adv, w[:3]),
              lambda: plan.forward(z, a, adv, w, o[:2]), lambda: plan.forward(z.T.contiguous().T, a, adv, w),
              lambda: plan.backward(z, a, adv, w, out=z[:3]), lambda: plan.backward(z, a, adv, w, grad=adv)):
        with pytest.raises(ValueError):
            g()


def test_more_than_32_bit_offsets(T):
    """Logits past 2^31 elements: the last rows."""
    t, v = 34000, 65536
    z = torch.zeros(t, v, dtype=torch.bfloat16, device="cuda")
    zl, al, advl, wl, ol, fl = inputs(8, v, "bf16")
    z[-8:] = zl
    put = lambda x, fill=0.0: torch.cat([torch.full((t - 8,), fill, device="cuda"), x])  # noqa: E731
    a = torch.cat([torch.full((t - 8,), -1, dtype=torch.int32, device="cuda"), al])
    plan = T.PolicyLoss(v, clip_low=LO, clip_high=HI, kl=0.1)
    want = reference(zl, al, advl, wl, ol, fl, 0.1, 1.0)
    loss, logp, dz = plan.forward_backward(z, a, put(advl), put(wl), put(ol), put(fl))
    check(dict(loss=loss, logp=logp[-8:], dz=dz[-8:]), want, 0.1, 1.0, advl, wl, ol, "bf16")
    assert (dz[:16] == 0).all() and (dz[-16:-8] == 0).all()
