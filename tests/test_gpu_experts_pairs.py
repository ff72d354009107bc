"""Expert products on SM pairs under load: what the two CTAs of a pair hand each other.  Reference and tolerances as in
test_gpu_experts.py."""
import pytest
import torch

from test_gpu_experts import T, check, offsets, reference  # noqa: F401 (T is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("way", ["forward", "data", "weight"])
@pytest.mark.parametrize("pad", [0, 1, 17])
def test_many_tiles_every_call_the_same(T, way, pad):  # noqa: F811
    """Several rounds of tiles on every pair, rows on and off the 16-byte lines, 20 calls without a pause: a half tile that
    one CTA wrote and the other's product read too early would differ from call to call."""
    k, n, rows_of = 512, 1032, [900, 0, 257, 1300, 33, 1, 700, 2000]
    off = offsets(rows_of)
    rows = off[-1]
    g = torch.Generator(device="cuda").manual_seed(40 + pad)

    def mat(c):
        t = torch.full((rows, c + pad), float("nan"), device="cuda").bfloat16()
        t[:, :c] = torch.randn(rows, c, generator=g, device="cuda")
        return t[:, :c]
    x, dy = mat(k), mat(n)
    w = torch.randn(len(rows_of), n, k, generator=g, device="cuda").bfloat16()
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    plan = T.Experts(len(rows_of), k, n)
    call, a, b, length = {"forward": (lambda: plan.forward(x, w, o), x, w, k), "data": (lambda: plan.backward_data(dy, w, o), dy, w, n),
                          "weight": (lambda: plan.backward_weight(dy, x, o), dy, x, max(rows_of))}[way]
    got = [call() for _ in range(20)]
    assert all(torch.equal(got[0], r) for r in got[1:])
    want, mag = reference(way, a, b, off, len(rows_of), k, n, rows)
    check(got[0], want, mag, length, way != "weight", way)
    assert plan.status() == (0, 0)
