"""Products grouped by expert against the definition in 64 bits.

Tolerance per element: an fp32 sum of L products has an error of at most
(L + 1) 2^-24 sum |a b| when each addition rounds to nearest, and twice that
when additions truncate (tensor cores): L' = (L + 8) 2^-23.  bf16 results add
half a unit in the last place, 2^-9 |result|, rounded up to 2^-8 for the
rounding of a value that is off by the first term."""
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


def reference(way, a, b, off, experts, k, n, rows):
    """(result, sum of absolute products) in 64 bits; a, b as the call takes them."""
    if way == "weight":
        out = torch.zeros(experts, n, k, dtype=torch.float64, device="cuda")
    else:
        out = torch.zeros(rows, n if way == "forward" else k, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    for e in range(experts):
        s = slice(off[e], off[e + 1])
        if way == "weight":
            p, q, at = a[s].double().T, b[s].double(), e
        else:
            p, q, at = a[s].double(), b[e].double(), s
            q = q.T if way == "forward" else q
        out[at] = p @ q
        mag[at] = p.abs() @ q.abs()
    return out, mag


def check(got, want, mag, length, bf16, what=""):
    tol = (length + 8) * 2.0 ** -23 * mag + (2.0 ** -8 * want.abs() if bf16 else 0.0)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}"


def offsets(rows_of, first=0):
    o = [first]
    for r in rows_of:
        o.append(o[-1] + r)
    return o


def run_way(T, plan, way, k, n, off, rows, dtype, seed, ld_pad=0, accumulate=False, stream=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype]

    def mat(r, c):
        t = torch.empty(r, c + ld_pad, dtype=dt, device="cuda").fill_(float("nan"))
        t[:, :c] = torch.randn(r, c, generator=g, device="cuda")
        return t[:, :c]
    experts = plan.experts
    x, dy = mat(rows, k), mat(rows, n)
    w = torch.randn(experts, n, k, generator=g, device="cuda").to(dt)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    if way == "forward":
        out = torch.full((rows, n + ld_pad), float("nan"), dtype=dt, device="cuda")[:, :n]
        got = plan.forward(x, w, o, out=out)
        want, mag = reference(way, x, w, off, experts, k, n, rows)
        check(got, want, mag, k, dtype == "bf16", way)
        if ld_pad and rows:
            assert torch.isnan(out._base[:, n:]).all()
    elif way == "data":
        out = torch.full((rows, k + ld_pad), float("nan"), dtype=dt, device="cuda")[:, :k]
        got = plan.backward_data(dy, w, o, out=out)
        want, mag = reference(way, dy, w, off, experts, k, n, rows)
        check(got, want, mag, n, dtype == "bf16", way)
        if ld_pad and rows:
            assert torch.isnan(out._base[:, k:]).all()
    else:
        longest = max(b - a for a, b in zip(off, off[1:]))
        out = torch.randn(experts, n, k, generator=g, device="cuda") if accumulate else torch.full((experts, n, k), float("nan"), device="cuda")
        before = out.double()
        got = plan.backward_weight(dy, x, o, out=out, accumulate=accumulate)
        want, mag = reference(way, dy, x, off, experts, k, n, rows)
        if accumulate:
            want, mag = want + before, mag + before.abs()
        check(got, want, mag, longest, False, way)
    assert plan.status() == (0, 0)
    return got


WAYS = ("forward", "data", "weight")

# rows of each expert: one row, none, tiles that end inside, several tiles, all rows on one expert
SPLITS = {
    "one_row": [1],
    "one_expert": [130],
    "single_tokens": [0, 1, 0, 0, 1, 1, 0, 1],
    "ragged": [5, 0, 64, 63, 65, 1, 17, 128],
    "empty_ends": [0, 0, 200, 0],
    "uneven": [3, 700, 0, 257, 31],
    "none": [0, 0, 0],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("k,n", [(64, 128), (72, 200), (136, 24)])
def test_small(T, dtype, way, split, k, n):
    rows = SPLITS[split]
    off = offsets(rows)
    run_way(T, T.Experts(len(rows), k, n, dtype), way, k, n, off, off[-1], dtype, seed=k + n)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("k,n", [(256, 512), (520, 1000), (1024, 264)])
@pytest.mark.parametrize("split", [[300, 513, 0, 1024, 77], [40] * 20, [3] * 33, [1100], [25] * 16, [1] * 64,
                                   [0, 0, 150, 0, 0, 0, 0, 0, 3], [0] * 60 + [17, 16, 1, 33], [0] * 1020 + [2, 0, 0, 1]])
def test_bf16_larger(T, way, k, n, split):
    off = offsets(split)
    run_way(T, T.Experts(len(split), k, n), way, k, n, off, off[-1], "bf16", seed=n)


@pytest.mark.parametrize("dtype,k,n", [("bf16", 33, 7), ("bf16", 1, 1), ("f32", 33, 7), ("f32", 1, 3), ("bf16", 100, 131), ("f32", 100, 131)])
@pytest.mark.parametrize("way", WAYS)
def test_widths_no_tile_fits(T, way, dtype, k, n):
    rows = [0, 70, 3, 129]
    off = offsets(rows)
    run_way(T, T.Experts(len(rows), k, n, dtype), way, k, n, off, off[-1], dtype, seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("pad", [8, 3])
def test_row_strides(T, way, dtype, pad):
    """Row strides above the width: 16-byte multiples and not; what lies between the rows is neither read nor written."""
    rows = [30, 0, 100, 64]
    off = offsets(rows)
    run_way(T, T.Experts(len(rows), 128, 256, dtype), way, 128, 256, off, off[-1], dtype, seed=6, ld_pad=pad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [1, 4])
def test_pointer_alignment(T, dtype, shift):
    """Tensors that start at any element."""
    k, n, rows = 64, 64, [20, 45]
    off = offsets(rows)
    g = torch.Generator(device="cuda").manual_seed(3)

    def flat(*shape):
        t = torch.randn(math.prod(shape) + shift, generator=g, device="cuda").to(DT[dtype])
        return t[shift:].view(*shape)
    x, dy, w = flat(65, k), flat(65, n), flat(2, n, k)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    plan = T.Experts(2, k, n, dtype)
    for way, got, a, b, length in (("forward", plan.forward(x, w, o, out=flat(65, n)), x, w, k),
                                   ("data", plan.backward_data(dy, w, o, out=flat(65, k)), dy, w, n)):
        want, mag = reference(way, a, b, off, 2, k, n, 65)
        check(got, want, mag, length, dtype == "bf16", way)
    dw = torch.empty(2 * n * k + 1, device="cuda")[1:].view(2, n, k)
    want, mag = reference("weight", dy, x, off, 2, k, n, 65)
    check(plan.backward_weight(dy, x, o, out=dw), want, mag, 45, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("way", WAYS)
def test_rows_of_no_expert(T, way, dtype):
    """Rows before the first offset and past the last one give zeros, and reach no gradient, whatever they hold."""
    k, n, rows = 96, 160, [17, 0, 70]
    off, total = offsets(rows, first=5), 5 + 87 + 9
    plan = T.Experts(3, k, n, dtype)
    got = run_way(T, plan, way, k, n, off, total, dtype, seed=8)
    if way != "weight":
        assert (got[:5] == 0).all() and (got[92:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("k,n", [(128, 256), (40, 24)])
def test_experts_do_not_mix(T, dtype, bad, k, n):
    """NaN and infinity in one expert's rows, in its filter and in rows of no expert stay there."""
    rows = [37, 50, 3, 66]
    off, total = offsets(rows, first=2), 2 + 156 + 11
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(total, k, generator=g, device="cuda").to(DT[dtype])
    dy = torch.randn(total, n, generator=g, device="cuda").to(DT[dtype])
    w = torch.randn(4, n, k, generator=g, device="cuda").to(DT[dtype])
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    plan = T.Experts(4, k, n, dtype)
    clean = plan.forward(x, w, o), plan.backward_data(dy, w, o), plan.backward_weight(dy, x, o)
    for t in (x, dy):
        t[off[1]:off[2]] = bad
        t[:2] = bad
        t[off[-1]:] = bad
    w[1] = bad
    y, dx, dw = plan.forward(x, w, o), plan.backward_data(dy, w, o), plan.backward_weight(dy, x, o)
    keep = torch.ones(total, dtype=torch.bool, device="cuda")
    keep[off[1]:off[2]] = False
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])
    assert torch.equal(dw[[0, 2, 3]], clean[2][[0, 2, 3]])
    assert not torch.isfinite(y[~keep]).any() and not torch.isfinite(dw[1]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("split", ["ragged", "uneven", "none"])
def test_accumulate(T, dtype, split):
    rows = SPLITS[split]
    off = offsets(rows)
    plan = T.Experts(len(rows), 128, 264, dtype)
    run_way(T, plan, "weight", 128, 264, off, off[-1], dtype, seed=10, accumulate=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_rows(T, dtype):
    plan = T.Experts(3, 64, 32, dtype)
    o = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty(0, 64, dtype=plan.dtype, device="cuda"), torch.empty(0, 32, dtype=plan.dtype, device="cuda")
    w = torch.zeros(3, 32, 64, dtype=plan.dtype, device="cuda")
    assert plan.forward(x, w, o).shape == (0, 32)
    assert plan.backward_data(dy, w, o).shape == (0, 64)
    dw = torch.full((3, 32, 64), 2.0, device="cuda")
    assert (plan.backward_weight(dy, x, o, out=dw, accumulate=True) == 2).all()
    assert (plan.backward_weight(dy, x, o, out=dw) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", [[0, 50, 20, 60], [-3, 10, 20, 60], [0, 10, 20, 61], [0, 10, 1 << 30, 60]])
def test_broken_offsets_are_reported(T, dtype, off):
    """Offsets out of order or out of the rows: a status, nothing out of bounds, experts with good offsets computed."""
    from conv2d_backward_implicit_bwd_gb300 import binding as B
    plan = T.Experts(3, 64, 64, dtype)
    guard = torch.full((60 + 64, 64), 7.0, dtype=plan.dtype, device="cuda")
    x = torch.ones(60, 64, dtype=plan.dtype, device="cuda")
    w = torch.ones(3, 64, 64, dtype=plan.dtype, device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    y = plan.forward(x, w, o, out=guard[:60])
    assert plan.status()[0] == B.ERR_DEVICE_FAULT
    plan.backward_weight(x, x, o)
    assert plan.status()[0] == B.ERR_DEVICE_FAULT
    assert plan.status() == (0, 0)
    assert (guard[60:] == 7).all()
    if off[0] == 0 and off[1] == 10:
        assert (y[:10] == 64).all()


def test_adjoint_identities_and_differences(T):
    """<forward(x, w), dy> = <x, data(dy, w)> = <w, weight(dy, x)>; the products are bilinear, so differences are exact
    up to the rounding of three fp32 sums of L terms each, and the inner products add at most the sum's error bound."""
    rows, k, n = [33, 0, 90, 7], 100, 60
    off, total = offsets(rows), 130
    plan = T.Experts(4, k, n, "f32")
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = torch.randn(total, k, generator=g, device="cuda"), torch.randn(total, n, generator=g, device="cuda")
    w, v = torch.randn(4, n, k, generator=g, device="cuda"), torch.randn(4, n, k, generator=g, device="cuda")
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    y, dx, dw = plan.forward(x, w, o), plan.backward_data(dy, w, o), plan.backward_weight(dy, x, o)
    dot = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
    _, mag = reference("forward", x, w, off, 4, k, n, total)
    tol = (max(k, n, 90) + 8) * 2.0 ** -23 * float((mag * dy.double().abs()).sum())
    assert abs(dot(y, dy) - dot(x, dx)) <= 2 * tol
    assert abs(dot(y, dy) - dot(w, dw)) <= 2 * tol
    h = 0.5
    step = (dot(plan.forward(x, w + h * v, o), dy) - dot(plan.forward(x, w - h * v, o), dy)) / (2 * h)
    _, magv = reference("forward", x, v, off, 4, k, n, total)
    tolv = (k + 8) * 2.0 ** -23 * float(((mag + h * magv) * dy.double().abs()).sum()) / h + tol
    assert abs(step - dot(v, dw)) <= 2 * tolv


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_every_time(T, dtype):
    rows = [200, 0, 13, 411]
    off = offsets(rows)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(off[-1], 256, generator=g, device="cuda").to(DT[dtype])
    dy = torch.randn(off[-1], 320, generator=g, device="cuda").to(DT[dtype])
    w = torch.randn(4, 320, 256, generator=g, device="cuda").to(DT[dtype])
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    plan = T.Experts(4, 256, 320, dtype)
    first = plan.forward(x, w, o), plan.backward_data(dy, w, o), plan.backward_weight(dy, x, o)
    for _ in range(3):
        again = plan.forward(x, w, o), plan.backward_data(dy, w, o), plan.backward_weight(dy, x, o)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_side_stream_and_graph(T):
    """The calls run on the stream they are given and can be captured: new offsets and rows are read at each replay."""
    k, n = 128, 192
    plan = T.Experts(3, k, n)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(96, k, generator=g, device="cuda").bfloat16()
    dy = torch.randn(96, n, generator=g, device="cuda").bfloat16()
    w = torch.randn(3, n, k, generator=g, device="cuda").bfloat16()
    o = torch.tensor([0, 10, 50, 96], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = plan.forward(x, w, o, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    want, mag = reference("forward", x, w, [0, 10, 50, 96], 3, k, n, 96)
    check(y, want, mag, k, True)
    out = torch.empty(96, n, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty(96, k, dtype=torch.bfloat16, device="cuda")
    dw = torch.empty(3, n, k, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(x, w, o, out=out)
        plan.backward_data(dy, w, o, out=dx)
        plan.backward_weight(dy, x, o, out=dw)
    for off in ([0, 10, 50, 96], [0, 96, 96, 96], [0, 0, 1, 40]):
        o.copy_(torch.tensor(off, dtype=torch.int32))
        x.copy_(torch.randn(96, k, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for way, got, a, b, length in (("forward", out, x, w, k), ("data", dx, dy, w, n), ("weight", dw, dy, x, 96)):
            want, mag = reference(way, a, b, off, 3, k, n, 96)
            check(got, want, mag, length, way != "weight", way)


def test_refusals(T):
    from conv2d_backward_implicit_bwd_gb300.binding import ConvBwdError
    plan = T.Experts(2, 64, 32)
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
    x, w, o = z(8, 64), z(2, 32, 64), torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for f in (lambda: plan.forward(z(8, 63), w, o), lambda: plan.forward(x.float(), w, o), lambda: plan.forward(x, z(2, 64, 32), o),
              lambda: plan.forward(x, w, o.long()), lambda: plan.forward(x, w, o[:2]), lambda: plan.forward(x, w, o, out=z(7, 32)),
              lambda: plan.forward(z(64, 8).T, w, o), lambda: plan.forward(x[:1].expand(8, 64), w, o),
              lambda: plan.backward_data(x, w, o), lambda: plan.backward_weight(z(8, 32), z(7, 64), o),
              lambda: plan.backward_weight(z(8, 32), x, o, accumulate=True),
              lambda: plan.backward_weight(z(8, 32), x, o, out=z(2, 32, 64))):
        with pytest.raises(ValueError):
            f()
    both = z(8, 96)
    with pytest.raises(ConvBwdError) as err:
        plan.forward(both[:, :64], w, o, out=both[:, 64:])       # rows interleave: refused as overlapping
    assert err.value.status == 1


def test_more_than_32_bit_offsets(T):
    """Rows whose elements lie past 2^31: first and last rows of a tall matrix on one expert, each way."""
    k, n, rows = 1024, 16, (1 << 21) + 40
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    ends = torch.cat([torch.arange(300), torch.arange(rows - 300, rows)]).cuda()
    x[ends] = torch.randn(600, k, generator=g, device="cuda").bfloat16()
    dy = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    dy[ends] = torch.randn(600, n, generator=g, device="cuda").bfloat16()
    w = torch.randn(2, n, k, generator=g, device="cuda").bfloat16()
    off = [0, 250, rows]
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    plan = T.Experts(2, k, n)
    y, dx, dw = plan.forward(x, w, o), plan.backward_data(dy, w, o), plan.backward_weight(dy, x, o)
    e = (torch.arange(600, device="cuda") >= 250).long()
    for got, a, b, length in ((y[ends], x[ends], w.transpose(1, 2), k), (dx[ends], dy[ends], w, n)):
        want = torch.einsum("ij,ijk->ik", a.double(), b[e].double())
        check(got, want, torch.einsum("ij,ijk->ik", a.double().abs(), b[e].double().abs()), length, True)
    assert (y[300:-300] == 0).all() and (dx[300:-300] == 0).all()
    want, mag = reference("weight", dy[ends], x[ends], [0, 250, 600], 2, k, n, 600)
    check(dw, want, mag, 600, False)
    assert plan.status() == (0, 0)


def test_long_sums_keep_their_precision(T):
    """fp32 gradients over many rows: within 2^-20 of the norm, however many rows are summed (a truncating
    accumulator would lose about r 2^-30)."""
    plan = T.Experts(1, 128, 256)
    g = torch.Generator(device="cuda").manual_seed(1)
    for rows in (500, 4000, 30000):
        x = torch.randn(rows, 128, generator=g, device="cuda").bfloat16()
        dy = torch.randn(rows, 256, generator=g, device="cuda").bfloat16()
        o = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        want = dy.double().T @ x.double()
        assert float((plan.backward_weight(dy, x, o)[0].double() - want).norm() / want.norm()) <= 2.0 ** -20


# Enough tiles for the wide ones of the plain-load kernels: 128 x 128 tiles that end inside on each side; odd widths load
# single elements, even ones pairs.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("narrow,wide", [(70, 2801), (66, 2802), (131, 2564)])
@pytest.mark.parametrize("way", WAYS)
def test_plain_loads_wide(T, way, dtype, narrow, wide):
    if way == "weight":
        k, n, rows_of = wide // 2, wide // 2 - 301, [300, 95]
    else:
        (k, n), rows_of = ((narrow, wide) if way == "forward" else (wide, narrow)), [700, 3, 300]
    off = offsets(rows_of)
    plan = T.Experts(len(rows_of), k, n, dtype)
    for pad in (0, 3):
        run_way(T, plan, way, k, n, off, off[-1], dtype, 21, ld_pad=pad, accumulate=pad > 0)


# Few tiles and a long contraction: its pieces are joined, in the same order every time.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("way", WAYS)
def test_plain_loads_split(T, way, dtype):
    for k, n, rows_of in ((70, 51, [3001, 17, 0, 1]), (2003, 70, [40]), (70, 2003, [1, 0, 65]), (129, 127, [127, 128, 129, 5000])):
        off = offsets(rows_of)
        plan = T.Experts(len(rows_of), k, n, dtype)
        a = run_way(T, plan, way, k, n, off, off[-1], dtype, 22, ld_pad=1)
        b = run_way(T, plan, way, k, n, off, off[-1], dtype, 22, ld_pad=1)
        assert torch.equal(a, b)
        if way == "weight":
            run_way(T, plan, way, k, n, off, off[-1], dtype, 23, accumulate=True)


# Few rows, filters that are shallow or narrow against their other side.
@pytest.mark.parametrize("deep,wide", [(72, 4104), (512, 1000), (2056, 96), (8, 8)])
@pytest.mark.parametrize("way", ["forward", "data"])
def test_few_rows_shallow_and_narrow(T, way, deep, wide):
    k, n = (deep, wide) if way == "forward" else (wide, deep)
    experts = 160
    plan = T.Experts(experts, k, n)
    for rows_of in ([1] * experts, [0, 3] * (experts // 2), [0] * (experts - 1) + [8 * experts]):
        off = offsets(rows_of)
        run_way(T, plan, way, k, n, off, off[-1], "bf16", 24)


# Few rows and enough tiles (128 of the filter's side each) to be drawn from a counter: every tile exactly once, call after
# call, the same bits whatever block drew it.
@pytest.mark.parametrize("way", ["forward", "data"])
def test_few_rows_drawn_tiles(T, way):
    deep, wide, experts = 576, 1040, 96
    k, n = (deep, wide) if way == "forward" else (wide, deep)
    plan = T.Experts(experts, k, n)
    first = None
    for rows_of in ([1] * experts, [5, 0, 17, 1] * (experts // 4), [5, 0, 17, 1] * (experts // 4), [8 * experts] + [0] * (experts - 1)):
        off = offsets(rows_of)
        got = run_way(T, plan, way, k, n, off, off[-1], "bf16", 25)
        if rows_of[0] == 5:
            assert first is None or torch.equal(first, got)
            first = got


# fp32 with few rows: vector and single loads, groups of eight rows that end inside, narrow and wide sides.
@pytest.mark.parametrize("way", ["forward", "data"])
@pytest.mark.parametrize("k,n", [(132, 1028), (2052, 96), (33, 130), (1, 7), (131, 1), (514, 513)])
def test_few_rows_fp32(T, way, k, n):
    experts = 24
    plan = T.Experts(experts, k, n, "f32")
    for rows_of in ([1] * experts, [0, 9, 3] * (experts // 3), [0] * (experts - 1) + [8 * experts - 1]):
        off = offsets(rows_of)
        for pad in (0, 1, 4):
            run_way(T, plan, way, k, n, off, off[-1], "f32", 26, ld_pad=pad)


# Rows that no 16-byte line begins: odd and even strides and starts, tiles of one to many rows, all rows at both ends of the
# tensor; the output on lines or not.
@pytest.mark.parametrize("way", ["forward", "data"])
@pytest.mark.parametrize("k,n", [(64, 256), (200, 520), (1032, 72), (8, 8)])
def test_rows_off_the_lines(T, way, k, n):
    plan = T.Experts(6, k, n)
    for rows_of in ([1, 0, 2, 0, 0, 5], [300, 0, 64, 257, 1, 31], [0, 0, 1500, 0, 3, 0]):
        off = offsets(rows_of)
        for pad in (1, 2, 4, 17):
            run_way(T, plan, way, k, n, off, off[-1], "bf16", 27, ld_pad=pad)
    # only the input, only the output, only the first row's address
    off = offsets([70, 0, 33, 1, 0, 129])
    rows = off[-1]
    wa, wo = (k, n) if way == "forward" else (n, k)
    g = torch.Generator(device="cuda").manual_seed(28)
    w = torch.randn(6, n, k, generator=g, device="cuda").bfloat16()
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    call = plan.forward if way == "forward" else plan.backward_data
    for pad_in, pad_out, first in ((3, 0, 0), (0, 3, 0), (0, 0, 1), (0, 8, 5), (8, 2, 3)):
        flat = torch.full((first + rows * (wa + pad_in),), float("nan"), device="cuda").bfloat16()
        a = flat[first:].view(rows, wa + pad_in)[:, :wa]
        a.copy_(torch.randn(rows, wa, generator=g, device="cuda"))
        out = torch.full((rows, wo + pad_out), float("nan"), device="cuda").bfloat16()[:, :wo]
        got = call(a, w, o, out=out)
        want, mag = reference(way, a, w, off, 6, k, n, rows)
        check(got, want, mag, wa, True, f"{way} {pad_in} {pad_out} {first}")
        if pad_out:
            assert torch.isnan(out._base[:, wo:]).all()
    assert plan.status() == (0, 0)


# The same for the weight gradient: both operands, one of them, first addresses; rows that end inside a step of 16, 64 and 512.
@pytest.mark.parametrize("k,n", [(64, 256), (200, 520), (1032, 72), (8, 8)])
def test_weight_of_rows_off_the_lines(T, k, n):
    plan = T.Experts(6, k, n)
    for rows_of in ([1, 0, 2, 0, 0, 5], [300, 0, 64, 257, 1, 31], [0, 0, 1500, 0, 3, 0]):
        off = offsets(rows_of)
        for pad in (1, 2, 4, 17):
            run_way(T, plan, "weight", k, n, off, off[-1], "bf16", 29, ld_pad=pad, accumulate=pad > 2)
    off = offsets([70, 0, 33, 1, 0, 600])
    rows = off[-1]
    g = torch.Generator(device="cuda").manual_seed(30)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")

    def mat(width, pad, first):
        flat = torch.full((first + rows * (width + pad),), float("nan"), device="cuda").bfloat16()
        t = flat[first:].view(rows, width + pad)[:, :width]
        t.copy_(torch.randn(rows, width, generator=g, device="cuda"))
        return t
    for pads in ((3, 0), (0, 3), (0, 0), (8, 8)):
        for first in ((0, 1), (5, 0), (3, 7)):
            dy, x = mat(n, pads[0], first[0]), mat(k, pads[1], first[1])
            got = plan.backward_weight(dy, x, o)
            want, mag = reference("weight", dy, x, off, 6, k, n, rows)
            check(got, want, mag, 600, False, f"{pads} {first}")
    assert plan.status() == (0, 0)
