"""GPU tests of the norms' statistics: mean and reciprocal deviation of the
block and of the sum, and what a large mean does to a layer norm.

Tolerances: a value of a row passes at most 16 additions in its thread, 6 in the
wave and 15 between waves, so that sums are off by less than 64 2^-24 of the
sum of magnitudes, a mean by its own rounding and by that much of the mean
difference to it."""
import pytest

from onnx_broadcast_matmul_amd import binding as mm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_ffn import BF16, F16, F32, TYPES, rand  # noqa: E402
from test_gpu_norm import KINDS, LAYER, S, SIZES, Case, gate_rows, mean  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    mm.lib()
    return torch.device("cuda:0")


def moments64(v, ev, kind, eps):
    """Mean and r of v (off by ev) in 64 bits, and how far they may be off."""
    if not kind:
        one = torch.ones_like(v[:, :1])
        return 0 * one, 0 * one, one, 0 * one
    m = mean(v) if kind == LAYER else 0 * v[:, :1]
    d = v - m
    em = mean(ev) + S * m.abs() + 64 * S * mean(d.abs()) if kind == LAYER else 0 * m
    var = mean(d * d)
    evar = 2 * mean(d.abs() * ev) + mean(ev * ev) + em * em + 64 * S * var
    r = (var + eps) ** -0.5
    return m, em, r, ((var - evar).clamp_min(0) + eps) ** -0.5 - r + 6 * S * r


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(SIZES)), ids=lambda i: "x".join(map(str, SIZES[i])))
def test_norm_statistics(i, dt, dev):
    """All four of a row, in every form; of a norm that is absent 0 and 1."""
    m, n = SIZES[i]
    for j, kind in enumerate(KINDS):
        c = Case(dev, m, n, TYPES[dt], seed=10 * j, gr=gate_rows(i + j, m), alpha=(1.0, -0.5)[j % 2], shift=(0.0, 5.0)[j % 2], **kind)
        stats = torch.full((m, 4), -7.0, device=dev)
        out = torch.empty_like(c.x) if c.pre else None
        c.plan.execute(c.x, out, block=c.b, gate=c.g, pre_weight=c.w2, pre_bias=c.b2, post_weight=c.w1, post_bias=c.b1,
                       stats=stats)
        b = c.x.double() if c.b is None else c.b.double()
        r, er = c.forward64()["sum"]
        want = moments64(b, 0 * b, c.post, c.eps) + moments64(r, er, c.pre, c.eps)
        for k, name in enumerate(("mean of B", "r of B", "mean of R", "r of R")):
            v, e = want[2 * k], want[2 * k + 1]
            assert bool(((stats[:, k:k + 1].double() - v).abs() <= e * (1 + 2.0 ** -10)).all()), (name, j)


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
