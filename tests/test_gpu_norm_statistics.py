"""GPU tests of the norms' statistics: what a large mean does to a layer norm.

Tolerances: a value of a row passes at most 16 additions in its thread, 6 in the
wave and 15 between waves, so that sums are off by less than 64 2^-24 of the
sum of magnitudes, a mean by its own rounding and by that much of the mean
difference to it."""
import pytest

from onnx_broadcast_matmul_amd import binding as mm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_ffn import BF16, F16, F32, rand  # noqa: E402
from test_gpu_norm import LAYER, S, mean  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    mm.lib()
    return torch.device("cuda:0")


@pytest.mark.parametrize("n", [7, 40, 513, 1000, 2047, 3000, 4099, 8192, 16384])
@pytest.mark.parametrize("dt", [BF16, F16, F32], ids=["bf16", "fp16", "fp32"])
def test_layer_norm_of_constant_rows(dt, n, dev):
    """Whatever the value and the length: the mean is the value, the result the bias."""
    m = 300
    x = (torch.linspace(-1000, 1000, m, device=dev) + rand((m,), F32, dev, 1)).to(dt)[:, None].expand(m, n).contiguous()
    b = rand((n,), dt, dev, 2)
    for kw in (dict(pre_bias=b), {}):
        y, stats = torch.empty_like(x), torch.empty(m, 4, device=dev)
        p = mm.NormPlan(m, n, mm.torch_dtype_code(dt), pre=LAYER, block=False, pre_weight=False, pre_bias=bool(kw),
                        pre_eps=1e-5, training=True)
        p.execute(x, y, stats=stats, **kw)
        assert torch.equal(stats[:, 2], x[:, 0].float())
        assert torch.equal(y, b.expand(m, n) if kw else torch.zeros_like(y))
        # the variance that is left: 2^-22 of squares of some last places of 1000
        assert bool(((stats[:, 3].double() * 1e-5 ** 0.5 - 1).abs() <= 2.0 ** -20).all())


@pytest.mark.parametrize("n", [40, 100, 1000, 2047, 4099, 8192, 16384])
def test_layer_norm_of_a_large_mean(n, dev):
    """A mean of ten thousand deviations: its own rounding is what it costs."""
    x = rand((200, n), F32, dev, 3) + 1e4
    y = torch.empty_like(x)
    mm.NormPlan(200, n, mm.FLOAT, pre=LAYER, block=False, pre_weight=False, pre_eps=1e-5).execute(x, y)
    v = x.double()
    d = v - mean(v)
    r = (mean(d * d) + 1e-5) ** -0.5
    tol = r * (S * mean(v).abs() + 64 * S * mean(d.abs())) + 64 * S * (d * r).abs()
    assert bool(((y.double() - d * r).abs() <= tol).all())
