"""The policy loss on rows wider than 16 KB, which stream through a ring of buffers: masked rows between live ones, several
rows to a block (three blocks on an SM), masked vocabularies, rows without a distribution, actions out of range.  Reference
and tolerances as in test_gpu_policy.py."""
import math

import pytest
import torch

from test_gpu_policy import DT, HI, LO, T, check, inputs, reference  # noqa: F401 (T is a fixture)

pytestmark = pytest.mark.gpu


def blocks():
    return 3 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype,v", [("bf16", 8200), ("bf16", 20000), ("bf16", 32768), ("f32", 4100), ("f32", 16384), ("f32", 20000)])
@pytest.mark.parametrize("pattern", ["live masked live", "masked live", "live masked masked live live masked", "random"])
def test_masked_rows_between_live_ones(T, dtype, v, pattern):  # noqa: F811
    """A row's results do not depend on what its block did before: the live rows' bits are those of a call without masks."""
    b = blocks()
    kind = pattern.split()
    t = b * max(len(kind), 4) + 5
    z, a, adv, w, o, f = inputs(t, v, dtype, seed=3)
    w = w + 0.1 / t
    plan = T.PolicyLoss(v, dtype, clip_low=LO, clip_high=HI, kl=0.1)
    clean = plan.forward(z, a, adv, w, o, f)
    clean_dz = plan.forward_backward(z, a, adv, w, o, f)[2]
    row = torch.arange(t, device="cuda")
    if pattern == "random":
        keep = torch.rand(t, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)) < 0.5
    else:
        keep = torch.tensor([k == "live" for k in kind], device="cuda")[row // b % len(kind)]
    w[~keep & (row % 2 == 0)] = 0
    a[~keep & (row % 2 == 1)] = -1
    for x in (adv, o, f):
        x[~keep] = float("nan")
    z[~keep, :5] = float("nan")
    for _ in range(5):
        loss, logp, lse, coef = plan.forward(z, a, adv, w, o, f)
        loss2, logp2, dz = plan.forward_backward(z, a, adv, w, o, f)
        assert torch.equal(loss, loss2) and torch.equal(logp, logp2)
        for got, want in ((logp, clean[1]), (lse, clean[2]), (coef, clean[3]), (dz, clean_dz)):
            assert torch.equal(got[keep], want[keep])
            assert (got[~keep] == 0).all()
        back = plan.backward(z, a, lse, coef)
        assert (back[~keep] == 0).all()
    some = keep.nonzero()[:: max(1, int(keep.sum()) // 60), 0]
    p = lambda x: x[some]  # noqa: E731
    want = reference(p(z), p(a), p(adv), p(w), p(o), p(f), 0.1, 1.0)
    check(dict(logp=p(logp), lse=p(lse), coef=p(coef), dz=p(dz)), want, 0.1, 1.0, p(adv), p(w), p(o), dtype)
    check(dict(dz=p(back)), want, 0.1, 1.0, p(adv), p(w), p(o), dtype)
    assert plan.status() == (0, 0)


@pytest.mark.parametrize("dtype,v", [("bf16", 20000), ("f32", 9000)])
def test_masked_vocabulary(T, dtype, v):  # noqa: F811
    """-inf and the type's lowest value among the logits of wide rows."""
    z, a, adv, w, o, f = inputs(8, v, dtype)
    z[:, ::2] = -math.inf
    z[4:, ::2] = torch.finfo(DT[dtype]).min
    z[2, :] = -math.inf
    z[2, 1] = 3.0
    a.fill_(1)
    plan = T.PolicyLoss(v, dtype, clip_low=LO, clip_high=HI, kl=0.1)
    o = f = torch.log_softmax(z.float(), 1)[:, 1] + 0.1
    want = reference(z, a, adv, w, o, f, 0.1, 1.0)
    want["dz"] = torch.where(torch.isnan(want["dz"]), 0.0, want["dz"])
    loss, logp, lse, coef = plan.forward(z, a, adv, w, o, f)
    check(dict(loss=loss, logp=logp, lse=lse, coef=coef), want, 0.1, 1.0, adv, w, o, dtype)
    dz = plan.forward_backward(z, a, adv, w, o, f)[2]
    for g in (dz, plan.backward(z, a, lse, coef)):
        check(dict(dz=g), want, 0.1, 1.0, adv, w, o, dtype)
        assert (g[:, ::2] == 0).all()
    assert float(logp[2]) == 0


@pytest.mark.parametrize("dtype,v", [("bf16", 20000), ("f32", 9000)])
@pytest.mark.parametrize("bad", [-math.inf, math.inf, math.nan])
def test_rows_without_a_distribution(T, dtype, v, bad):  # noqa: F811
    z, a, adv, w, o, f = inputs(6, v, dtype)
    plan = T.PolicyLoss(v, dtype, clip_low=LO, clip_high=HI, kl=0.1)
    clean = plan.forward_backward(z, a, adv, w, o, f)
    z[2] = bad
    loss, logp, dz = plan.forward_backward(z, a, adv, w, o, f)
    keep = [0, 1, 3, 4, 5]
    assert math.isnan(float(loss)) and math.isnan(float(logp[2])) and torch.isnan(dz[2]).any()
    assert torch.equal(logp[keep], clean[1][keep]) and torch.equal(dz[keep], clean[2][keep])


@pytest.mark.parametrize("dtype,v", [("bf16", 20000), ("f32", 9000)])
def test_action_out_of_range(T, dtype, v):  # noqa: F811
    from conv2d_backward_implicit_bwd_gb300 import binding as B
    z, a, adv, w, o, f = inputs(6, v, dtype)
    a[4] = v
    plan = T.PolicyLoss(v, dtype, clip_low=LO, clip_high=HI)
    loss, logp, dz = plan.forward_backward(z, a, adv, w, o, f)
    assert plan.status()[0] == B.ERR_DEVICE_FAULT and plan.status() == (0, 0)
    assert float(logp[4]) == 0 and (dz[4] == 0).all() and math.isfinite(float(loss))


@pytest.mark.parametrize("dtype,v", [("f32", (1 << 29) - 5000), ("f32", 1 << 29), ("f32", 1 << 30), ("bf16", 1 << 30)])
def test_widest_rows(T, dtype, v):  # noqa: F811
    """Rows whose bytes reach 2^31 and 2^32.  A thread adds a sum of 16 (32) exponentials to its own v / 4096 (v / 8192) times,
    each rounding to 2^-24 of a positive sum: the row's sum, and with it lse and every probability, is off by
    v 2^-36 at most, and by what test_gpu_policy.py has for narrower rows."""
    z = torch.empty(1, v, dtype=DT[dtype], device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    for part in z[0].split(1 << 26):
        part.copy_(torch.randn(len(part), generator=g, device="cuda"))
    at = v - 7
    z[0, at] = 12.5
    a, one = torch.tensor([at], dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    lse = math.log(sum(float(part.double().exp().sum()) for part in z[0].split(1 << 26)))
    plan = T.PolicyLoss(v, dtype)
    loss, logp, got_lse, coef = plan.forward(z, a, one, one)
    rel = v * 2.0 ** -36 + 2.0 ** -19 * (1 + abs(lse) + abs(12.5 - lse))
    assert abs(float(got_lse) - lse) <= rel and abs(float(logp) - (12.5 - lse)) <= rel
    assert float(coef) == -1 and float(loss) == -1
    rnd = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -22

    def gradient(dz):
        first = 0
        for x, d in zip(z[0].split(1 << 26), dz[0].split(1 << 26)):
            p = (x.double() - lse).exp()
            want, size = p.clone(), p.clone()
            if first <= at < first + len(x):
                want[at - first] -= 1
                size[at - first] += 1
            assert ((d.double() - want).abs() <= rnd * want.abs() + 3 * rel * size).all()
            first += len(x)
    dz = plan.backward(z, a, got_lse, coef)
    gradient(dz)
    dz.fill_(7.0)
    loss2, logp2, _ = plan.forward_backward(z, a, one, one, out=dz)
    assert torch.equal(loss, loss2) and torch.equal(logp, logp2)
    gradient(dz)
    assert plan.status() == (0, 0)
