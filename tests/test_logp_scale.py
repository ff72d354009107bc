"""Scales of the log-probabilities near the ends of fp32."""
import pytest
import torch

from conv2d_backward_implicit_bwd_gb300 import build as cbuild


@pytest.mark.parametrize("scale", [2.0 ** 127 * 1.0001, 2.4e38, 3.4e38])
def test_refused(scale):
    """scale log2(e) has to be finite."""
    cbuild.build()
    from conv2d_backward_implicit_bwd_gb300 import train as T
    from conv2d_backward_implicit_bwd_gb300.binding import ConvBwdError
    with pytest.raises(ConvBwdError) as e:
        T.TokenLogp(8, scale=scale)
    assert e.value.status == 1
    for ok in (2.0 ** 127, 2.0 ** -126):
        T.TokenLogp(8, scale=ok)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("t,v", [(5, 50), (3, 40001), (2500, 5001)])
@pytest.mark.parametrize("power", [-120, -100, 100, 120, 127])
def test_powers_of_two(dtype, t, v, power):
    """Logits divided by the scale: the statistics are those of the logits themselves."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_logp import check_forward, rows_of
    from conv2d_backward_implicit_bwd_gb300 import train as T
    z, a = rows_of(t, v, dtype, spread=1.5)
    z.copy_((z.double() * 2.0 ** -power).to(z.dtype))
    a[1::5] = -1
    check_forward(T.TokenLogp(v, dtype, top=3, scale=2.0 ** power), z, a, scale=2.0 ** power)
