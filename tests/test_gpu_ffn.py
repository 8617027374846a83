"""GPU tests of the feed-forward operators (gated block with its backward pass,
INT8 product with row and column scales, row quantization) against plain forms
in 64 bits.

Tolerances are per element and follow from the arithmetic:

* an FP32 sum of n products in any order is off by at most n 2^-24 of the sum
  of magnitudes; 2 n 2^-24 is allowed;
* rounding to type t moves a value by at most ``finfo(t).eps / 2`` of it, or
  half the smallest subnormal;
* the activations and their derivatives are within 2^-16 (16-bit types: the
  hardware exponential of an argument up to 90 is off by some 90 2^-24, the
  gelu fit by 2.7e-6) or 2^-19 (FLOAT) of their magnitude, where a derivative's
  magnitude is taken as 1 + |g|;
* every activation here changes by at most 1.13 times its argument's change.
"""
import math

import numpy as np
import pytest

from onnx_broadcast_matmul_amd import binding as mm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = {"fp32": F32, "fp16": F16, "bf16": BF16}
ACTS = list(mm.ACTIVATIONS)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    mm.lib()
    return torch.device("cuda:0")


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # the smallest subnormal


def act_error(dt):
    return 2.0 ** -19 if dt == F32 else 2.0 ** -16


def act64(name, g):
    """The activation and its derivative in 64 bits."""
    if name == "relu":
        return torch.where(g > 0, g, 0 * g), (g > 0).double()
    if name == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * p, p + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    s = torch.sigmoid(g)
    return (g * s, s * (1 + g * (1 - s))) if name == "silu" else (s, s * (1 - s))


def rand(shape, dt, dev, seed, scale=1.0):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dt)


def guarded(shape, dt, dev, offset=0):
    """A dense tensor of `shape` inside a larger allocation whose other
    elements must keep their value; `offset` elements off 16-byte alignment."""
    n = math.prod(shape)
    buf = torch.full((n + 512,), -7.0 if dt.is_floating_point else -7, dtype=dt, device=dev)
    return buf[256 + offset:256 + offset + n].view(shape), buf


def check_guard(buf, t, offset=0):
    n = t.numel()
    assert bool((buf[:256 + offset] == -7).all()) and bool((buf[256 + offset + n:] == -7).all()), "wrote outside"


def within(y, want, tol, what):
    y = y.double()
    assert y.shape == want.shape
    bad = ~((y - want).abs() <= tol)
    if bool(bad.any()):
        i = int(bad.flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {y.flatten()[i].item()} "
                             f"against {want.flatten()[i].item()}, allowed {tol.expand_as(want).flatten()[i].item():.3g}")


# ---- gated block, forward


def forward64(x, wg, wu, act, dt):
    """H, G, U in 64 bits with their tolerances; weights [K, N]."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    k = x.shape[1]
    g, u = x @ wg, x @ wu
    eg, eu = (2 * k * 2.0 ** -24 * (x.abs() @ w.abs()) for w in (wg, wu))
    f, _ = act64(act, g)
    h = f * u
    u_ = half_step(dt)
    raw = 1.13 * eg * (u.abs() + eu) + f.abs() * eu + act_error(dt) * f.abs() * u.abs()
    th = raw * (1 + u_) + u_ * h.abs() + tiny(dt)
    tg, tu = (e * (1 + u_) + u_ * v.abs() + tiny(dt) for e, v in ((eg, g), (eu, u)))
    return (h, th), (g, tg), (u, tu)


def run_forward(dev, m, k, n, dt, nk, act, seed=0, keep=False, offset=0, merged=False, tile=0, algo=0, scale=1.0,
                split=0):
    x, _ = guarded((m, k), dt, dev, offset)
    x.copy_(rand((m, k), dt, dev, seed, scale))
    wide = rand((2 * n, k) if nk else (k, 2 * n), dt, dev, seed + 1, max(k, 1) ** -0.5)
    if merged:
        wg, wu = (wide[:n], wide[n:]) if nk else (wide[:, :n], wide[:, n:])
        pitch = 0 if nk else 2 * n
    else:
        wg, wu = (wide[:n].contiguous(), wide[n:].contiguous()) if nk else (wide[:, :n].contiguous(), wide[:, n:].contiguous())
        pitch = 0
        if offset:
            ws = []
            for w in (wg, wu):
                t, _ = guarded(w.shape, dt, dev, offset)
                t.copy_(w)
                ws.append(t)
            wg, wu = ws
    plan = mm.GluPlan(m, k, n, mm.torch_dtype_code(dt), activation=mm.ACTIVATIONS[act], trans_w=nk, w_pitch=pitch,
                      force_algo=algo, tile=tile, split_k=split)
    outs = [guarded((m, n), dt, dev, offset) for _ in range(3 if keep else 1)]
    plan.execute(x, wg, wu, *(t for t, _ in outs))
    torch.cuda.synchronize()
    want = forward64(x, wg.t() if nk else wg, wu.t() if nk else wu, act, dt)
    for (t, buf), (w, tol), name in zip(outs, want, "HGU"):
        within(t, w, tol, f"{name} {m}x{k}x{n}")
        check_guard(buf, t, offset)
    return plan


SIZES = [(1, 1, 1), (1, 64, 16), (1, 2048, 520), (3, 7, 5), (5, 72, 33), (16, 256, 160), (17, 264, 40), (32, 129, 96),
         (33, 200, 72), (64, 77, 55), (130, 136, 264), (257, 72, 131), (300, 512, 300)]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(SIZES)), ids=lambda i: "x".join(map(str, SIZES[i])))
def test_glu_forward(i, dt, nk, dev):
    run_forward(dev, *SIZES[i], TYPES[dt], nk, ACTS[i % len(ACTS)], seed=10 + i, keep=i % 2 == 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_glu_activations_over_a_wide_range(act, dt, dev):
    """Gate values to about +-40, where every tail is reached, on the tiles
    and on the few-row kernel."""
    run_forward(dev, 200, 64, 96, TYPES[dt], True, act, seed=40, keep=True, scale=10.0)
    run_forward(dev, 9, 64, 96, TYPES[dt], True, act, seed=41, keep=True, scale=10.0)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt,tile", [(d, t) for d in TYPES for t in ((2, 3, 4) if d == "fp32" else (1, 2, 3, 4, 5))])
def test_glu_every_tile(tile, nk, dt, dev):
    """Aligned and odd sizes over several tiles with a ragged edge, K of one
    stage, of less, and of many."""
    for j, (m, k, n) in enumerate(((530, 328, 400), (270, 16, 136), (300, 701, 281), (2, 35, 9))):
        run_forward(dev, m, k, n, TYPES[dt], nk, "silu", seed=50 + j, tile=tile, algo=mm.ALGO_GENERAL, keep=j == 0)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt,tile", [(d, t) for d in TYPES for t in ((2, 3, 4) if d == "fp32" else (2, 3, 4, 5))])
def test_glu_split(tile, nk, dt, dev):
    for j, (m, k, n, split) in enumerate(((270, 1040, 136, 3), (50, 701, 281, 1000), (2, 35, 9, 2))):
        p = run_forward(dev, m, k, n, TYPES[dt], nk, ACTS[j], seed=55 + j, tile=tile, split=split, keep=j != 1)
        assert j == 2 or p.info()["algo_name"] == "split_k"


@pytest.mark.parametrize("m", [1, 16, 17, 32])
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_glu_few_rows(m, nk, dt, dev):
    for j, (k, n) in enumerate(((4096, 48), (1000, 33), (3, 2), (130, 515))):
        run_forward(dev, m, k, n, TYPES[dt], nk, "gelu", seed=60 + j, algo=mm.ALGO_SKINNY_M, keep=j == 1)


@pytest.mark.parametrize("m", [1, 13, 32])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_glu_few_rows_off_dword_alignment(m, dt, dev):
    """Rows of every alignment (odd K) and a base off a dword (even K), blocks
    of K whole and partial, few columns and more than 512 workgroups."""
    for j, (k, n, offset) in enumerate(((1301, 35, 0), (64, 20, 1), (1300, 40, 1), (67, 8209, 0))):
        run_forward(dev, m, k, n, TYPES[dt], True, "silu", seed=90 + j, algo=mm.ALGO_SKINNY_M, offset=offset, keep=j == 0)


@pytest.mark.parametrize("m", [4, 150])
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_glu_unaligned_and_merged_operands(m, nk, dev):
    run_forward(dev, m, 64, 96, BF16, nk, "silu", seed=70, offset=1, keep=True)
    run_forward(dev, m, 64, 96, BF16, nk, "silu", seed=71, merged=True)
    run_forward(dev, m, 65, 97, F16, nk, "silu", seed=72, merged=True)
    run_forward(dev, m, 64, 96, F32, nk, "silu", seed=73, offset=1)


@pytest.mark.parametrize("m", [3, 200])
def test_glu_empty_reduction_and_nan_rows(m, dev):
    p = mm.GluPlan(m, 0, 40, mm.BFLOAT16, activation=mm.ACT_SIGMOID)
    h = torch.full((m, 40), 5.0, dtype=BF16, device=dev)
    e = torch.empty(m, 0, dtype=BF16, device=dev), torch.empty(0, 40, dtype=BF16, device=dev)
    p.execute(e[0], e[1], e[1], h)
    assert bool((h == 0).all())
    # a NaN and an infinity stay in their rows
    x, w = rand((m, 64), BF16, dev, 80), rand((40, 64), BF16, dev, 81, 0.1)
    p = mm.GluPlan(m, 64, 40, mm.BFLOAT16, trans_w=True)
    clean, dirty = torch.empty(m, 40, dtype=BF16, device=dev), torch.empty(m, 40, dtype=BF16, device=dev)
    p.execute(x, w, w, clean)
    x2 = x.clone()
    x2[1, 5] = float("nan")
    x2[2, 6] = float("inf")
    p.execute(x2, w, w, dirty)
    assert bool(dirty[1].isnan().all()) and not bool(dirty[2].isfinite().all())
    keep = [r for r in range(m) if r not in (1, 2)]
    assert torch.equal(clean[keep], dirty[keep])


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("keep", [False, True], ids=["h", "hgu"])
def test_glu_more_large_tiles_than_cus(nk, keep, dev):
    """Workgroups that walk several 256 x 256 tiles: ragged edges, K of the
    fewest stages that they take, of a part of one more, and of a few."""
    for j, (m, k, n) in enumerate(((4300, 128, 2312), (2900, 136, 3592), (4500, 328, 4104))):
        run_forward(dev, m, k, n, (BF16, F16)[j % 2], nk, ACTS[(j + 2 * keep) % 5], seed=90 + j, tile=1,
                    algo=mm.ALGO_GENERAL, keep=keep)


# ---- gated block, backward


def backward64(x, wg, wu, g, u, dh, act, dt):
    """dX, dWg, dWu (weights [K, N]) in 64 bits from the given G and U."""
    x, wg, wu, g, u, dh = (t.double() for t in (x, wg, wu, g, u, dh))
    m, k, n = x.shape[0], x.shape[1], g.shape[1]
    f, d = act64(act, g)
    dg, du = dh * u * d, dh * f
    u_, e = half_step(dt), act_error(dt)
    eg = u_ * dg.abs() + e * (dh * u).abs() * (1 + g.abs()) + tiny(dt)
    eu = u_ * du.abs() + e * du.abs() + tiny(dt)
    dx = dg @ wg.t() + du @ wu.t()
    s = 2.0 ** -24
    tx = eg @ wg.abs().t() + eu @ wu.abs().t() + 4 * n * s * (dg.abs() @ wg.abs().t() + du.abs() @ wu.abs().t())
    out = [(dx, tx * (1 + u_) + u_ * dx.abs() + tiny(dt))]
    for v, ev in ((dg, eg), (du, eu)):
        dw = x.t() @ v
        tw = x.abs().t() @ ev + 2 * m * s * (x.abs().t() @ v.abs())
        out.append((dw, tw * (1 + u_) + u_ * dw.abs() + tiny(dt)))
    return out


def run_backward(dev, m, k, n, dt, nk, act, seed=0, want="xw", offset=0, merged=False):
    x, g, u, dh = (rand(s, dt, dev, seed + i, c) for i, (s, c) in
                   enumerate((((m, k), 1.0), ((m, n), 1.5), ((m, n), 1.0), ((m, n), 0.5))))
    pitch = 0 if nk or not merged else 2 * n
    shape = (n, k) if nk else (k, n)

    def weight(s):
        w = rand(shape, dt, dev, s, 0.2)
        if not merged:
            return w
        wide = torch.full((2 * n, k) if nk else (k, 2 * n), -7.0, dtype=dt, device=dev)
        half = wide[:n] if nk else wide[:, :n]
        half.copy_(w)
        return half

    wg, wu = weight(seed + 5), weight(seed + 6)
    dwg, dwu = weight(seed + 7), weight(seed + 8)
    plan = mm.GluPlan(m, k, n, mm.torch_dtype_code(dt), activation=mm.ACTIVATIONS[act], trans_w=nk, training=True,
                      w_pitch=pitch)
    dx, buf = guarded((m, k), dt, dev, offset)
    plan.backward(x, wg, wu, g, u, dh, dx if "x" in want else None, dwg if "w" in want else None,
                  dwu if "w" in want else None)
    torch.cuda.synchronize()
    ref = backward64(x, wg.t() if nk else wg, wu.t() if nk else wu, g, u, dh, act, dt)
    if "x" in want:
        within(dx, *ref[0], f"dX {m}x{k}x{n}")
    else:
        assert bool((dx == -7).all())
    check_guard(buf, dx, offset)
    if "w" in want:
        within(dwg.t() if nk else dwg, *ref[1], f"dWg {m}x{k}x{n}")
        within(dwu.t() if nk else dwu, *ref[2], f"dWu {m}x{k}x{n}")
        if merged and not nk:  # the other half of every row
            for t in (dwg, dwu):
                rest = torch.as_strided(t, (k, n), (2 * n, 1), t.storage_offset() + n)
                assert bool((rest == -7).all()), "wrote between the rows"


BSIZES = [(1, 1, 1), (1, 64, 48), (2, 9, 3), (16, 128, 96), (33, 40, 72), (44, 882, 309), (130, 136, 264),
          (257, 71, 131), (300, 512, 364), (1200, 64, 72), (5000, 35, 42)]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(BSIZES)), ids=lambda i: "x".join(map(str, BSIZES[i])))
def test_glu_backward(i, dt, nk, dev):
    run_backward(dev, *BSIZES[i], TYPES[dt], nk, ACTS[i % len(ACTS)], seed=100 + 10 * i)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_glu_backward_activations(act, dt, dev):
    run_backward(dev, 70, 40, 56, TYPES[dt], True, act, seed=300)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_glu_backward_variants(nk, dev):
    run_backward(dev, 600, 544, 520, BF16, nk, "silu", seed=400)  # large tiles
    run_backward(dev, 40, 64, 96, F16, nk, "silu", seed=410, want="x")
    run_backward(dev, 40, 64, 96, F16, nk, "silu", seed=420, want="w")
    run_backward(dev, 40, 64, 96, BF16, nk, "silu", seed=430, offset=1)
    run_backward(dev, 40, 64, 96, BF16, nk, "silu", seed=440, merged=True)
    run_backward(dev, 41, 63, 95, F32, nk, "silu", seed=450, merged=True)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_glu_backward_more_large_tiles_than_cus(nk, dev):
    run_backward(dev, 4360, 4616, 264, BF16, nk, "silu", seed=460)  # dX: 342 large tiles
    run_backward(dev, 520, 4616, 2360, F16, nk, "gelu", seed=470)  # dW: 2 x 190


def test_glu_backward_empty(dev):
    for dt in (F32, BF16):
        code = mm.torch_dtype_code(dt)
        e = lambda *s: torch.full(s, 3.0, dtype=dt, device=dev)  # noqa: E731
        # no rows: zero weight gradients
        p = mm.GluPlan(0, 24, 40, code, training=True)
        dwg, dwu = e(24, 40), e(24, 40)
        p.backward(e(0, 24), e(24, 40), e(24, 40), e(0, 40), e(0, 40), e(0, 40), e(0, 24), dwg, dwu)
        assert bool((dwg == 0).all()) and bool((dwu == 0).all())
        # no hidden features: zero input gradient
        p = mm.GluPlan(7, 24, 0, code, training=True)
        dx = e(7, 24)
        p.backward(e(7, 24), e(24, 0), e(24, 0), e(7, 0), e(7, 0), e(7, 0), dx, e(24, 0), e(24, 0))
        assert bool((dx == 0).all())


@pytest.mark.parametrize("act", [a for a in ACTS if a != "relu"])
def test_glu_gradients_against_differences(act, dev):
    """The FLOAT gradients along random directions against central
    differences of the 64-bit loss sum(H * R).  With step h the difference is
    off by h^2 / 6 times the third derivative (below 1e2 here, so under 2e-7 at
    h = 1e-4) and the 64-bit loss's rounding over h (1e-11); the gradients by
    their tolerance along the direction."""
    m, k, n, h = 12, 20, 28, 1e-4
    x, wg, wu, r = (rand(s, F32, dev, 500 + i, c) for i, (s, c) in
                    enumerate((((m, k), 1.0), ((k, n), 0.3), ((k, n), 0.3), ((m, n), 1.0))))
    plan = mm.GluPlan(m, k, n, mm.FLOAT, activation=mm.ACTIVATIONS[act], training=True)
    H, G, U = (torch.empty(m, n, device=dev) for _ in range(3))
    plan.execute(x, wg, wu, H, G, U)
    grads = [torch.empty_like(t) for t in (x, wg, wu)]
    plan.backward(x, wg, wu, G, U, r, *grads)

    def loss(x, wg, wu):
        return float((act64(act, x @ wg)[0] * (x @ wu) * r.double()).sum())

    at = [t.double() for t in (x, wg, wu)]
    for i in range(3):
        for j in range(3):
            v = rand(at[i].shape, torch.float64, dev, 520 + 3 * i + j)
            v = v / v.norm()
            up, down = [t.clone() for t in at], [t.clone() for t in at]
            up[i] += h * v
            down[i] -= h * v
            diff = (loss(*up) - loss(*down)) / (2 * h)
            got = float((grads[i].double() * v).sum())
            # gradient entries: FP32 sums of at most 2 * 28 terms over FP32 G, U
            # of 20 terms, all below about 1e2 in magnitude sum
            scale = float((grads[i].double().abs() * v.abs()).sum()) + 10.0
            assert abs(got - diff) <= 1e-5 * scale, (i, j, got, diff)


# ---- row quantization


def quantize64(x):
    """The rule with every operation rounded to 32 bits (numpy)."""
    x = x.float().cpu().numpy()
    top = np.abs(x).max(axis=-1, initial=0.0)
    bad = ~np.isfinite(top)
    amax = np.maximum(np.where(bad, 1.0, top), np.float32(2.0 ** -100)).astype(np.float32)
    scale = (amax / np.float32(127)).astype(np.float32)
    r = (np.float32(127) / amax).astype(np.float32)
    with np.errstate(invalid="ignore"):
        q = np.rint((x * r[..., None]).astype(np.float32))
    q = np.where(bad[..., None], 0, q).astype(np.int8)
    return q, np.where(bad, np.float32("nan"), scale)


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 100), (4, 1024), (7, 1025), (2, 4097), (3, 11008),
                                       (2, 40000), (1, 131071), (1001, 33)])
def test_quantize_rows(rows, cols, dt, dev):
    x = rand((rows, cols), TYPES[dt], dev, rows + cols)
    x[0, cols // 2] *= 50
    q, buf = guarded((rows, cols), torch.int8, dev, 1)
    q, s = mm.quantize_rows(x, q)
    wq, ws = quantize64(x)
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
    check_guard(buf, q, 1)


@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_quantize_rows_special_values(dt, dev):
    t = TYPES[dt]
    big, small = torch.finfo(t).max, tiny(t)
    rows = [[0.0] * 9, [-0.0] * 9, [small] + [0.0] * 8, [big, -big] + [1.0] * 7, [float("inf")] + [1.0] * 8,
            [1.0] * 8 + [float("nan")], [-float("inf"), float("nan")] + [0.0] * 7, [127.0, 0.5, 1.5, -0.5, -1.5, 2.5, 1, 2, 3],
            [2.0 ** -14] * 9]
    x = torch.tensor(rows, dtype=t, device=dev)
    q, s = mm.quantize_rows(x)
    wq, ws = quantize64(x)
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    e, z = mm.quantize_rows(torch.empty(3, 0, dtype=t, device=dev))
    assert e.shape == (3, 0) and np.array_equal(z.cpu().numpy(), np.full(3, np.float32(2.0 ** -100) / np.float32(127)))
    assert mm.quantize_rows(torch.empty(0, 5, dtype=t, device=dev))[1].shape == (0,)


def test_quantize_more_rows_than_one_grid_dimension_covers(dev):
    """2^26 rows and some: more than 2^32 threads."""
    n = (1 << 26) // 7 + 3
    x = torch.tensor([[0.0], [1.0], [-2.5], [float("inf")], [0.1], [-100.0], [2.0 ** -14]], dtype=F16, device=dev)
    q, s = mm.quantize_rows(x)
    many_q, many_s = mm.quantize_rows(x.repeat(n, 1))
    assert torch.equal(many_q, q.repeat(n, 1)) and torch.equal(many_s.view(torch.int32), s.view(torch.int32).repeat(n))


# ---- scaled INT8 product


def ints(shape, dev, seed):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return torch.randint(-128, 128, shape, generator=gen, device=dev, dtype=torch.int8)


def scales(shape, dev, seed):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return torch.rand(shape, generator=gen, device=dev) * 0.01 + 1e-3


def run_scaled(dev, sa, sb, dt, nk=False, bias=False, seed=0, offset=0, **kw):
    """sb is the [.., K, N] shape; nk stores it [.., N, K]."""
    b = ints(sb, dev, seed + 1)
    stored = b.transpose(-1, -2).contiguous() if nk else b
    a, bt = guarded(sa, torch.int8, dev, offset)[0], guarded(stored.shape, torch.int8, dev, offset)[0]
    a.copy_(ints(sa, dev, seed))
    bt.copy_(stored)
    plan = mm.ScaledIntPlan(sa, stored.shape, mm.torch_dtype_code(dt), trans_b=nk, bias=bias, **kw)
    asc, bsc = scales(plan.a_scale_shape, dev, seed + 2), scales(plan.b_scale_shape, dev, seed + 3)
    n = 1 if len(sb) == 1 else sb[-1]
    bv = rand((n,), dt, dev, seed + 4) if bias else None
    y, buf = guarded(plan.output_shape, dt, dev, offset)
    plan.execute(a, bt, y, a_scale=asc, b_scale=bsc, bias=bv)
    torch.cuda.synchronize()
    check_guard(buf, y, offset)
    if len(sa) == 2 and len(sb) == 2:
        total, av, bvv = a.double() @ b.double(), asc.double(), bsc.double()
    else:  # batched products of 64-bit operands on the CPU
        total = torch.matmul(a.cpu().double(), b.cpu().double()).to(dev)
        av, bvv = asc.double(), bsc.double()
    if len(sa) > 1:
        av = av.unsqueeze(-1) if len(sb) > 1 else av
    want = total * av * (bvv.unsqueeze(-2) if len(sa) > 1 and len(sb) > 1 else bvv)
    t = 4 * 2.0 ** -24 * want.abs()
    if bias:
        off = bv.double()
        want = want + (off if len(sb) > 1 else off.reshape(()))
        t = t + 2.0 ** -23 * (want.abs() + off.abs().max())
    tol = t * (1 + half_step(dt)) + half_step(dt) * want.abs() + tiny(dt)
    within(y, want, tol, f"{sa} x {sb}")
    return plan, y


SSIZES = [(1, 1, 1), (1, 64, 16), (1, 11008, 96), (3, 7, 5), (16, 256, 160), (24, 1000, 130), (32, 130, 33),
          (33, 200, 72), (64, 77, 55), (130, 144, 272), (257, 64, 131), (333, 1000, 301), (100, 8192, 128)]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("i", range(len(SSIZES)), ids=lambda i: "x".join(map(str, SSIZES[i])))
def test_scaled(i, nk, dev):
    m, k, n = SSIZES[i]
    run_scaled(dev, (m, k), (k, n), list(TYPES.values())[i % 3], nk, bias=i % 2 == 0, seed=600 + 5 * i)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("m", [1, 16, 29])
def test_scaled_few_rows_of_any_alignment_and_width(m, nk, dev):
    """Row lengths and bases off 4-byte alignment, and column counts on both
    sides of each width of the few-row kernel's workgroups."""
    for j, (k, n, offset) in enumerate(((1301, 35, 0), (1302, 16, 0), (1303, 4097, 0), (256, 40, 1), (1024, 24, 2),
                                        (260, 4096, 3), (515, 8192, 0), (300, 8193, 0), (257, 8208, 1))):
        run_scaled(dev, (m, k), (k, n), BF16, nk, bias=j % 2 == 0, seed=760 + 5 * j, offset=offset,
                   force_algo=mm.ALGO_SKINNY_M)


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_scaled_every_kernel_gives_the_same_bits(nk, dt, dev):
    """Tiles, splits and the few-row kernel, aligned and odd, over one product."""
    for m, k, n in ((20, 1168, 304), (20, 1111, 301)):
        got = []
        for kw in (dict(force_algo=mm.ALGO_SKINNY_M), dict(tile=1), dict(tile=2), dict(tile=3), dict(tile=4), dict(tile=5),
                       dict(tile=5, split_k=2),
                   dict(tile=2, split_k=3), dict(tile=3, split_k=2), dict(tile=4, split_k=5),
                   dict(tile=4, split_k=1000), dict(force_algo=mm.ALGO_GENERAL)):
            got.append(run_scaled(dev, (m, k), (k, n), TYPES[dt], nk, bias=True, seed=700, **kw)[1])
        for y in got[1:]:
            assert torch.equal(y.view(torch.uint8), got[0].view(torch.uint8))


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_scaled_more_large_tiles_than_cus(dt, nk, dev):
    run_scaled(dev, (4360, 272), (272, 4624), TYPES[dt], nk, bias=True, seed=705, tile=1)
    run_scaled(dev, (3, 1400, 320), (3, 320, 4112), TYPES[dt], nk, seed=706, tile=1)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_scaled_broadcast_shapes(nk, dev):
    run_scaled(dev, (2, 1, 40, 64), (3, 64, 48), F32, nk, bias=True, seed=720)
    run_scaled(dev, (2, 3, 5, 64), (64, 48), BF16, nk, bias=True, seed=730)  # folds into the rows
    run_scaled(dev, (5, 65), (4, 65, 33), F16, nk, seed=740)
    run_scaled(dev, (2, 9, 1024), (2, 1024, 40), F32, nk, seed=750, split_k=4)
    run_scaled(dev, (64,), (64, 48), F32, nk, seed=760)
    run_scaled(dev, (3, 64, 32), (3, 32, 16), F32, nk, seed=790, offset=1)
    if not nk:
        run_scaled(dev, (6, 64), (64,), F32, bias=True, seed=770)
        run_scaled(dev, (64,), (64,), F32, seed=780)


def test_scaled_extreme_sums(dev):
    """The largest magnitude INT32 has to hold, on every kind of kernel."""
    k = 131071
    for m, n, kw in ((1, 3, {}), (2, 2, dict(force_algo=mm.ALGO_GENERAL)), (2, 2, dict(split_k=7))):
        for nk in (True, False):
            a = torch.full((m, k), -128, dtype=torch.int8, device=dev)
            b = torch.full((n, k) if nk else (k, n), -128, dtype=torch.int8, device=dev)
            p = mm.ScaledIntPlan((m, k), b.shape, mm.FLOAT, trans_b=nk, **kw)
            y = torch.empty(m, n, device=dev)
            one = torch.ones(max(m, n), device=dev)
            p.execute(a, b, y, a_scale=one[:m], b_scale=one[:n])
            assert bool((y == float(np.float32(k * 16384))).all())


def test_scaled_empty_and_nan_scales(dev):
    for kw in ({}, dict(force_algo=mm.ALGO_GENERAL)):
        p = mm.ScaledIntPlan((5, 0), (0, 24), mm.BFLOAT16, bias=True, **kw)
        y = torch.empty(5, 24, dtype=BF16, device=dev)
        bias = rand((24,), BF16, dev, 800)
        z = torch.ones(24, device=dev)
        p.execute(torch.empty(5, 0, dtype=torch.int8, device=dev), torch.empty(0, 24, dtype=torch.int8, device=dev), y,
                  a_scale=z[:5], b_scale=z, bias=bias)
        assert torch.equal(y, bias.expand(5, 24))
    for m in (6, 60):
        p = mm.ScaledIntPlan((m, 64), (64, 24), mm.FLOAT)
        sa, sb = scales((m,), dev, 1), scales((24,), dev, 2)
        a, b = ints((m, 64), dev, 3), ints((64, 24), dev, 4)
        clean, y = torch.empty(m, 24, device=dev), torch.empty(m, 24, device=dev)
        p.execute(a, b, clean, a_scale=sa, b_scale=sb)
        sa[2] = float("nan")
        sb[7] = float("inf")
        p.execute(a, b, y, a_scale=sa, b_scale=sb)
        assert bool(y[2].isnan().all()) and not bool(y[:, 7].isfinite().any())
        rest = [[r for r in range(m) if r != 2], [c for c in range(24) if c != 7]]
        assert torch.equal(y[rest[0]][:, rest[1]], clean[rest[0]][:, rest[1]])


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_dynamic_product_is_quantization_then_product(nk, dt, dev):
    """A plan that quantizes A gives the bits of the two calls: the few-row
    kernel that does it itself, rows quantized before it, tiles, splits,
    batches, another output type."""
    t = TYPES[dt]
    other = F32 if t != F32 else BF16
    for j, (sa, sb, out) in enumerate((((1, 2048), (2048, 96), t), ((4, 100), (100, 33), t), ((4, 1), (1, 3), t),
                                       ((9, 2000), (2000, 64), t), ((7, 1030), (1030, 70), t),
                                       ((3, 9000), (9000, 20), t), ((4, 1301), (1301, 70), t), ((2, 1303), (1303, 8300), t), ((4, 260), (260, 8300), t), ((1, 64), (64, 48), other), ((200, 72), (72, 130), t),
                                       ((130, 77), (77, 55), t), ((2, 3, 40, 65), (65, 48), t),
                                       ((2, 1, 40, 65), (3, 65, 33), t), ((64,), (64, 48), t), ((3, 0), (0, 9), t))):
        x = rand(sa, t, dev, 820 + j)
        if x.numel() > 64:
            x.view(-1)[5] = 40.0
        b = ints(sb, dev, 840 + j)
        stored = b.transpose(-1, -2).contiguous() if nk else b
        dyn = mm.ScaledIntPlan(sa, stored.shape, mm.torch_dtype_code(out), a_type=mm.torch_dtype_code(t), trans_b=nk, bias=True)
        two = mm.ScaledIntPlan(sa, stored.shape, mm.torch_dtype_code(out), trans_b=nk, bias=True)
        sbv, bias = scales(dyn.b_scale_shape, dev, 860 + j), rand((sb[-1],), out, dev, 870 + j)
        y1, buf = guarded(dyn.output_shape, out, dev)
        y2 = torch.empty(dyn.output_shape, dtype=out, device=dev)
        dyn.execute(x, stored, y1, b_scale=sbv, bias=bias)
        q, s = mm.quantize_rows(x)
        two.execute(q, stored, y2, a_scale=s, b_scale=sbv, bias=bias)
        torch.cuda.synchronize()
        assert torch.equal(y1.view(torch.uint8), y2.view(torch.uint8)), (sa, sb)
        check_guard(buf, y1)


def test_dynamic_product_of_rows_without_a_scale(dev):
    for m in (2, 60):
        x = rand((m, 64), BF16, dev, 900)
        x[1, 3] = float("inf")
        b = ints((24, 64), dev, 901)
        p = mm.ScaledIntPlan((m, 64), (24, 64), mm.BFLOAT16, a_type=mm.BFLOAT16, trans_b=True)
        y = torch.empty(m, 24, dtype=BF16, device=dev)
        p.execute(x, b, y, b_scale=scales((24,), dev, 902))
        assert bool(y[1].isnan().all()) and bool(y[0].isfinite().all())


# ---- together, and the ways they are called


def ffn_calls(dev, m=40, d=64, hid=96):
    """A served block with an 8-bit last layer and a training step, as a list
    of (call, outputs)."""
    x, dh = rand((m, d), BF16, dev, 910), rand((m, hid), BF16, dev, 911)
    wg, wu = rand((hid, d), BF16, dev, 912, d ** -0.5), rand((hid, d), BF16, dev, 913, d ** -0.5)
    wd, sd = mm.quantize_rows(rand((d, hid), BF16, dev, 914, hid ** -0.5))
    glu = mm.GluPlan(m, d, hid, mm.BFLOAT16, trans_w=True, training=True)
    down = mm.ScaledIntPlan((m, hid), (d, hid), mm.BFLOAT16, a_type=mm.BFLOAT16, trans_b=True)
    split = mm.ScaledIntPlan((m, hid), (d, hid), mm.BFLOAT16, trans_b=True, split_k=2)
    e = lambda *s: torch.zeros(s, dtype=BF16, device=dev)  # noqa: E731
    h, g, u, y, y2, dx, dwg, dwu = e(m, hid), e(m, hid), e(m, hid), e(m, d), e(m, d), e(m, d), e(hid, d), e(hid, d)
    q, s = torch.zeros(m, hid, dtype=torch.int8, device=dev), torch.zeros(m, device=dev)

    def call():
        glu.execute(x, wg, wu, h, g, u)
        down.execute(h, wd, y, b_scale=sd)
        mm.quantize_rows(h, q, s)
        split.execute(q, wd, y2, a_scale=s, b_scale=sd)
        glu.backward(x, wg, wu, g, u, dh, dx, dwg, dwu)

    return call, [h, g, u, y, y2, q, s, dx, dwg, dwu], (x, wg, wu, wd, sd, dh)


@pytest.mark.parametrize("m", [2, 40, 700])
def test_served_block_and_training_step(m, dev):
    call, outs, (x, wg, wu, wd, sd, dh) = ffn_calls(dev, m)
    call()
    torch.cuda.synchronize()
    h, g, u, y, y2, q, s, dx, dwg, dwu = outs
    (wh, th), (w1, t1), (w2, t2) = forward64(x, wg.t(), wu.t(), "silu", BF16)
    within(h, wh, th, "H")
    within(g, w1, t1, "G")
    within(u, w2, t2, "U")
    wq, ws = quantize64(h)
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
    want = (q.double() @ wd.double().t()) * s.double()[:, None] * sd.double()
    within(y, want, (4 * 2.0 ** -24 + half_step(BF16)) * want.abs() + tiny(BF16), "Y")
    assert torch.equal(y, y2)
    for t, (w, tol), name in zip((dx, dwg.t(), dwu.t()), backward64(x, wg.t(), wu.t(), g, u, dh, "silu", BF16), ("dX", "dWg", "dWu")):
        within(t, w, tol, name)


@pytest.mark.parametrize("m", [2, 40, 700])
def test_graph_replays_match_eager(m, dev):
    call, outs, _ = ffn_calls(dev, m)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(4):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
        call()  # eager work between the replays
        torch.cuda.synchronize()


def test_two_streams_at_once(dev):
    """Unsplit forward passes of one plan overlap freely; the rest takes a plan
    per stream."""
    sets = [ffn_calls(dev, 300, 256, 512) for _ in range(2)]
    for call, _, _ in sets:
        call()
    torch.cuda.synchronize()
    want = [[t.clone() for t in outs] for _, outs, _ in sets]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for st, (call, outs, _) in zip(streams, sets):
            with torch.cuda.stream(st):
                for t in outs:
                    t.zero_()
                call()
    torch.cuda.synchronize()
    for (_, outs, _), w in zip(sets, want):
        for t, v in zip(outs, w):
            assert torch.equal(t.view(torch.uint8), v.view(torch.uint8))
    x, w = rand((300, 256), BF16, dev, 1), rand((512, 256), BF16, dev, 2, 0.1)
    plan = mm.GluPlan(300, 256, 512, mm.BFLOAT16, trans_w=True)
    assert plan.workspace_bytes == 0
    hs = [torch.empty(300, 512, dtype=BF16, device=dev) for _ in range(2)]
    torch.cuda.synchronize()
    for st, h in zip(streams, hs):
        plan.execute(x, w, w, h, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(hs[0], hs[1])


def test_same_weight_twice_and_repeated_calls(dev):
    """Wg and Wu may be one tensor; the same call gives the same bits."""
    for m in (3, 200):
        x, w = rand((m, 96), F16, dev, 3), rand((96, 72), F16, dev, 4, 0.1)
        p = mm.GluPlan(m, 96, 72, mm.FLOAT16)
        h1, h2 = torch.empty(m, 72, dtype=F16, device=dev), torch.empty(m, 72, dtype=F16, device=dev)
        p.execute(x, w, w, h1)
        p.execute(x, w, w, h2)
        assert torch.equal(h1, h2)
        (want, tol), _, _ = forward64(x, w, w, "silu", F16)
        within(h1, want, tol, "H")


def test_binding_checks(dev):
    x, w, h = rand((4, 64), BF16, dev, 1), rand((64, 32), BF16, dev, 2), torch.empty(4, 32, dtype=BF16, device=dev)
    p = mm.GluPlan(4, 64, 32, mm.BFLOAT16)
    for bad in ((x.float(), w, w, h), (x, w.t(), w, h), (x, w, w[:, :16], h), (x, w, w, h[:2]),
                (x.cpu(), w, w, h), (x, w.t().contiguous().t(), w, h), (x.t().contiguous().t(), w, w, h)):
        with pytest.raises(ValueError):
            p.execute(*bad)
    with pytest.raises(mm.MMError):
        p.backward(x, w, w, h, h, h, x)


def test_offsets_past_32_bits(dev):
    """Operands and outputs of more than 2^31 elements: the last rows are
    those of the same rows alone."""
    m, k, n = 70000, 16, 32768
    x, w = rand((m, k), BF16, dev, 5), rand((n, k), BF16, dev, 6)
    h = torch.empty(m, n, dtype=BF16, device=dev)
    mm.GluPlan(m, k, n, mm.BFLOAT16, trans_w=True).execute(x, w, w, h)
    few = torch.empty(40, n, dtype=BF16, device=dev)
    mm.GluPlan(40, k, n, mm.BFLOAT16, trans_w=True).execute(x[-40:].contiguous(), w, w, few)
    (want, tol), _, _ = forward64(x[-40:], w.t(), w.t(), "silu", BF16)
    within(h[-40:], want, tol, "H")
    within(few, want, tol, "few H")
    # rows of 32768, quantized past 2^31 elements, then multiplied
    q, s = mm.quantize_rows(h)
    q1, s1 = mm.quantize_rows(h[-7:].contiguous())
    assert torch.equal(q[-7:], q1) and torch.equal(s[-7:], s1)
    b = ints((24, n), dev, 7)
    sb = scales((24,), dev, 8)
    y = torch.empty(m, 24, dtype=BF16, device=dev)
    mm.ScaledIntPlan((m, n), (24, n), mm.BFLOAT16, trans_b=True).execute(q, b, y, a_scale=s, b_scale=sb)
    want = (q[-40:].double() @ b.double().t()) * s[-40:].double()[:, None] * sb.double()
    within(y[-40:], want, (4 * 2.0 ** -24 + half_step(BF16)) * want.abs() + tiny(BF16), "Y")
    del q, y
    # the gradients of the last rows
    g, dh = h, torch.ones_like(h)
    dx = torch.empty_like(x)
    plan = mm.GluPlan(m, k, n, mm.BFLOAT16, trans_w=True, training=True)
    plan.backward(x, w, w, g, g, dh, dx)
    wx, tx = backward64(x[-9:], w.t(), w.t(), g[-9:], g[-9:], dh[-9:], "silu", BF16)[0]
    within(dx[-9:], wx, tx, "dX")


# ---- empty reductions, rounding, far ends of the activations


@pytest.mark.parametrize("bias", [False, True], ids=["plain", "bias"])
@pytest.mark.parametrize("a_type", ["int8", "quantized"])
def test_scaled_empty_reduction_takes_no_scales(a_type, bias, dev):
    """K == 0 gives the bias or zeros, whatever the scales hold: few rows,
    tiles, and batches with scales of their own."""
    for j, (sa, sb, kw) in enumerate((((5, 0), (0, 24), dict(force_algo=mm.ALGO_SKINNY_M)), ((5, 0), (0, 24), {}),
                                      ((70, 0), (0, 33), {}), ((3, 5, 0), (3, 0, 24), {}),
                                      ((2, 1, 40, 0), (3, 0, 24), {}), ((0,), (0,), {}))):
        dt = list(TYPES.values())[j % 3]
        at = torch.int8 if a_type == "int8" else dt
        p = mm.ScaledIntPlan(sa, sb, mm.torch_dtype_code(dt), a_type=mm.torch_dtype_code(dt) if a_type != "int8" else mm.INT8,
                             bias=bias, **kw)
        asc, bsc = torch.ones(p.a_scale_shape, device=dev), torch.ones(p.b_scale_shape, device=dev)
        asc.view(-1)[-1] = float("nan")
        bsc.view(-1)[0] = float("inf")
        bv = rand((1 if len(sb) == 1 else sb[-1],), dt, dev, 1000 + j) if bias else None
        y, buf = guarded(p.output_shape, dt, dev)
        p.execute(torch.empty(sa, dtype=at, device=dev), torch.empty(sb, dtype=torch.int8, device=dev), y,
                  a_scale=asc if a_type == "int8" else None, b_scale=bsc, bias=bv)
        torch.cuda.synchronize()
        want = torch.zeros((), dtype=dt, device=dev) if bv is None else bv if len(sb) > 1 else bv[0]
        assert torch.equal(y, want.expand(y.shape)), (sa, sb)
        check_guard(buf, y)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_glu_gradient_of_far_finite_gates(act, dt, dev):
    """f' of finite gates up to the type's largest is its limit: 1 above and 0
    below, 0 on both sides for the sigmoid.  Wg is the identity, Wu zero and U
    one, so that dX is dH f'(G) itself."""
    t = TYPES[dt]
    top = torch.finfo(t).max
    row = [v for a in (200.0, 6.0e4, 1.0e13, 1.0e19, 3.0e19, 1.0e25, 1.0e38, top) if a <= top for v in (a, -a)]
    n = len(row)
    g = torch.tensor(row, dtype=t, device=dev).repeat(5, 1)
    u, dh = torch.ones_like(g), torch.full_like(g, 0.5)
    wg, wu = torch.eye(n, dtype=t, device=dev), torch.zeros(n, n, dtype=t, device=dev)
    dx = torch.empty(5, n, dtype=t, device=dev)
    p = mm.GluPlan(5, n, n, mm.torch_dtype_code(t), activation=mm.ACTIVATIONS[act], training=True)
    p.backward(torch.zeros_like(dx), wg, wu, g, u, dh, dx)
    want = dh * ((g > 0) & (act != "sigmoid")).to(t)
    assert torch.equal(dx, want), dx[0]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_glu_forced_split_of_one_partition(nk, dev):
    for j, (m, k, n) in enumerate(((300, 64, 64), (2, 35, 9), (40, 264, 130))):
        p = run_forward(dev, m, k, n, list(TYPES.values())[j], nk, "silu", seed=1100 + j, algo=mm.ALGO_SPLIT_K, split=1,
                        keep=j != 1)
        assert p.info()["algo_name"] == "split_k" and p.info()["split_k"] == 1


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_scaled_column_scale_and_bias_round_once(nk, dev):
    """(sum sa) is rounded, then sb times it and the bias together: with sum 1,
    both scales 1 + 2^-23 and the bias -(1 + 2^-22) that leaves 2^-46, where a
    rounded product would leave 0."""
    s = 1.0 + 2.0 ** -23
    for m, kw in ((3, dict(force_algo=mm.ALGO_SKINNY_M)), (50, dict(tile=3)), (50, dict(tile=4, split_k=2))):
        a, b = torch.ones(m, 512, dtype=torch.int8, device=dev), torch.zeros(512, 24, dtype=torch.int8, device=dev)
        b[77] = 1
        b = b.t().contiguous() if nk else b
        p = mm.ScaledIntPlan(a.shape, b.shape, mm.FLOAT, trans_b=nk, bias=True, **kw)
        y = torch.empty(m, 24, device=dev)
        p.execute(a, b, y, a_scale=torch.full((m,), s, device=dev), b_scale=torch.full((24,), s, device=dev),
                  bias=torch.full((24,), -1.0 - 2.0 ** -22, device=dev))
        assert bool((y == 2.0 ** -46).all())


# ---- operands of any place, every entry of the backward products


def placed(values, offset=0, gap=0, fill=float("nan")):
    """A copy of the matrix `values` with rows `gap` elements apart, `offset`
    elements off 16-byte alignment, and a check that nothing around it changed
    (`fill` everywhere: a value read from there would spoil the result)."""
    r, c = values.shape
    buf = torch.full((256 + offset + r * (c + gap) + 256,), fill, dtype=values.dtype, device=values.device)
    at = ((r, c), (c + gap, 1), 256 + offset)
    view = buf.as_strided(*at)
    view.copy_(values)
    rest = torch.ones_like(buf, dtype=torch.bool)
    rest.as_strided(*at).fill_(False)
    before = buf[rest].clone().view(torch.uint8)

    def check(what):
        assert torch.equal(buf[rest].view(torch.uint8), before), f"wrote outside {what}"

    return view, check


def run_step(dev, m, k, n, dt, nk, act, seed=0, offset=0, gap=0, forward=True, kept=None, **options):
    """A training step whose eleven operands all lie at `offset`, the weights
    and their gradients with rows `gap` apart, G and U of type `kept`, compared
    with 64 bits."""
    kept = kept or dt
    shape = (n, k) if nk else (k, n)
    values = {"x": rand((m, k), dt, dev, seed), "dh": rand((m, n), dt, dev, seed + 1, 0.5)}
    for i, w in enumerate(("wg", "wu", "dwg", "dwu")):
        values[w] = rand(shape, dt, dev, seed + 2 + i, 0.2)
    for i, name in enumerate(("h", "g", "u")):
        values[name] = rand((m, n), dt if name == "h" else kept, dev, seed + 6 + i, 1.5)
    values["dx"] = rand((m, k), dt, dev, seed + 9)
    t, checks = {}, []
    for name, v in values.items():
        t[name], check = placed(v, offset, gap if "w" in name else 0)
        checks.append((name, check))
    plan = mm.GluPlan(m, k, n, mm.torch_dtype_code(dt), activation=mm.ACTIVATIONS[act], trans_w=nk, training=True,
                      w_pitch=shape[1] + gap if gap else 0, kept_type=mm.torch_dtype_code(kept), **options)
    w = [t[i].t() if nk else t[i] for i in ("wg", "wu")]
    if forward:
        plan.execute(t["x"], t["wg"], t["wu"], t["h"], t["g"], t["u"])
        torch.cuda.synchronize()
        for name, (want, tol) in zip("hgu", forward64(t["x"], *w, act, dt)[:1] + forward64(t["x"], *w, act, kept)[1:]):
            within(t[name], want, tol, f"{name} {m}x{k}x{n}")
    plan.backward(t["x"], t["wg"], t["wu"], t["g"], t["u"], t["dh"], t["dx"], t["dwg"], t["dwu"])
    torch.cuda.synchronize()
    for name, (want, tol) in zip(("dx", "dwg", "dwu"), backward64(t["x"], *w, t["g"], t["u"], t["dh"], act, dt)):
        within(t[name].t() if nk and "w" in name else t[name], want, tol, f"{name} {m}x{k}x{n}")
    for name, check in checks:
        check(name)
    return plan


@pytest.mark.parametrize("offset,gap", [(0, 0), (0, 16), (0, 3), (1, 0), (1, 16), (3, 5)])
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_glu_step_on_operands_of_any_place(dt, nk, offset, gap, dev):
    """Bases and pitches on and off 16-byte alignment, aligned and odd sizes,
    on the few-row kernel and the tiles."""
    for j, (m, k, n) in enumerate(((5, 64, 96), (3, 65, 33), (150, 64, 96), (150, 65, 97), (300, 200, 136))):
        run_step(dev, m, k, n, TYPES[dt], nk, ACTS[j], seed=1200 + 10 * j, offset=offset, gap=gap)


BACK_TILES = [(d, t) for d in TYPES for t in ((2, 3, 4) if d == "fp32" else (1, 2, 3, 4, 5))]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt,tile", BACK_TILES)
def test_glu_backward_every_tile(tile, nk, dt, dev):
    """dX and the pair dWg, dWu on each entry, whole and split K, over several
    tiles with a ragged edge: aligned and odd sizes, operands off alignment,
    reductions of many stages, of part of one and of one element."""
    dw = tile if dt == "fp32" or tile != 4 else 3  # dW of 16-bit types has no entry 4
    for split in (1, 3) if tile > 1 else (1,):
        for j, (m, k, n, offset, gap) in enumerate(((530, 328, 400, 0, 0), (300, 701, 281, 0, 0), (270, 136, 16, 0, 8),
                                                    (16, 264, 530, 1, 0), (2, 35, 9, 0, 0), (1, 300, 1, 0, 1))):
            p = run_step(dev, m, k, n, TYPES[dt], nk, ACTS[j % 5], seed=1300 + 10 * j, offset=offset, gap=gap,
                         forward=False, dx_tile=tile, dw_tile=dw, dx_split_k=split, dw_split_k=split)
            i = p.options()
            assert (i["dx_tile"], i["dw_tile"]) == (tile, dw)
            assert j > 1 or (i["dx_split_k"] == split and i["dw_split_k"] in (2, split))


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_glu_backward_more_tiles_of_each_large_entry_than_cus(dt, nk, dev):
    """dX of the first size has 18 x 19 tiles of 256 x 256, dW of the second twice
    10 x 19; with 256 x 128 about twice as many."""
    for tile in (1, 5):
        for j, (m, k, n) in enumerate(((4360, 4616, 264), (520, 4616, 2360))):
            p = run_step(dev, m, k, n, TYPES[dt], nk, "silu", seed=1400 + 10 * j, forward=False, dx_tile=tile, dw_tile=tile,
                         dx_split_k=1, dw_split_k=1)
            assert p.options() == {"kept_type": mm.torch_dtype_code(TYPES[dt]), "dx_tile": tile, "dx_split_k": 1,
                                   "dw_tile": tile, "dw_split_k": 1}


def test_quantize_rows_makes_its_results_on_its_stream(dev):
    """Memory freed on the current stream, whose queued work may still use it,
    is not what a call on another stream writes to."""
    x = rand((700, 3001), BF16, dev, 1500)
    wq, ws = quantize64(x)
    side = torch.cuda.Stream()
    old = [torch.empty(700, 3001, dtype=torch.int8, device=dev), torch.empty(700, device=dev)]
    at = {t.data_ptr() for t in old}
    torch.cuda.synchronize()
    del old
    q, s = mm.quantize_rows(x, stream=side)
    torch.cuda.synchronize()
    assert q.data_ptr() not in at and s.data_ptr() not in at
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


# ---- G and U kept in FP32


@pytest.mark.parametrize("offset,gap", [(0, 0), (1, 5)])
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_glu_step_with_g_and_u_in_fp32(dt, nk, offset, gap, dev):
    """The few-row kernel, every tile, whole and split K, aligned and odd."""
    t = TYPES[dt]
    for j, (m, k, n) in enumerate(((1, 64, 96), (3, 65, 33), (20, 264, 130), (150, 65, 97), (300, 200, 136))):
        run_step(dev, m, k, n, t, nk, ACTS[j], seed=1600 + 10 * j, offset=offset, gap=gap, kept=F32)
    for tile in (2, 3, 4) if dt == "fp32" else (1, 2, 3, 4, 5):
        for split in (1, 2) if tile > 1 else (1,):
            for j, (m, k, n) in enumerate(((270, 528, 136), (300, 701, 281), (2, 35, 9))):
                run_step(dev, m, k, n, t, nk, ACTS[(tile + j) % 5], seed=1650 + 10 * j, offset=offset, gap=gap, kept=F32,
                         tile=tile, split_k=split)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_glu_gradients_round_twice_when_g_and_u_are_fp32(act, dt, dev):
    """From X and the weights to the gradients, dG and dU and the results are
    the only values rounded to 16 bits: the error is that of 64-bit gradients
    with these two roundings, to 2 %.  (dG and dU are off by some 2^-16 of
    theirs before they are rounded, which moves one in a hundred over a tie,
    where either neighbour is half a step off: the norm of the error keeps.)"""
    t = TYPES[dt]
    m, k, n = 700, 192, 320
    x, dh = rand((m, k), t, dev, 1700), rand((m, n), t, dev, 1701, 0.1)
    wg, wu = rand((n, k), t, dev, 1702, k ** -0.5), rand((n, k), t, dev, 1703, k ** -0.5)
    p = mm.GluPlan(m, k, n, mm.torch_dtype_code(t), activation=mm.ACTIVATIONS[act], trans_w=True, training=True,
                   kept_type=mm.FLOAT)
    h, g, u = torch.empty(m, n, dtype=t, device=dev), torch.empty(m, n, device=dev), torch.empty(m, n, device=dev)
    got = [torch.empty_like(v) for v in (x, wg, wu)]
    p.execute(x, wg, wu, h, g, u)
    p.backward(x, wg, wu, g, u, dh, *got)
    x, wg, wu, dh = (v.double() for v in (x, wg, wu, dh))
    f, d = act64(act, x @ wg.t())
    dg, du = dh * (x @ wu.t()) * d, dh * f
    products = lambda a, b: (a @ wg + b @ wu, a.t() @ x, b.t() @ x)  # noqa: E731
    for v, exact, two in zip(got, products(dg, du), products(dg.to(t).double(), du.to(t).double())):
        error, least = (float((w.double() - exact).norm() / exact.norm()) for w in (v, two.to(t)))
        assert error <= 1.02 * least, (error, least)


def test_glu_fp32_g_and_u_replayed_from_a_graph(dev):
    m, k, n = 300, 128, 200
    x, dh = rand((m, k), BF16, dev, 1800), rand((m, n), BF16, dev, 1801)
    wg, wu = rand((n, k), BF16, dev, 1802, 0.1), rand((n, k), BF16, dev, 1803, 0.1)
    p = mm.GluPlan(m, k, n, mm.BFLOAT16, trans_w=True, training=True, split_k=2, kept_type=mm.FLOAT)
    outs = [torch.zeros(m, n, dtype=BF16, device=dev), torch.zeros(m, n, device=dev), torch.zeros(m, n, device=dev),
            torch.zeros_like(x), torch.zeros_like(wg), torch.zeros_like(wu)]

    def call():
        p.execute(x, wg, wu, *outs[:3])
        p.backward(x, wg, wu, outs[1], outs[2], dh, *outs[3:])

    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t.view(torch.uint8), w.view(torch.uint8)) for t, w in zip(outs, want))
        call()
        torch.cuda.synchronize()
    with pytest.raises(ValueError):  # G and U of the plan's type, where it keeps FP32
        p.execute(x, wg, wu, outs[0], outs[1].to(BF16), outs[2].to(BF16))


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("kept", ["same", "fp32"])
def test_glu_gradients_into_the_halves_of_one_matrix(kept, nk, dev):
    """Weights and gradients as gate and up halves of merged matrices, on a
    stream of the caller's."""
    for j, (m, k, n, dt) in enumerate(((40, 64, 96, BF16), (150, 65, 97, F16), (33, 31, 7, BF16), (70, 40, 33, F32))):
        x, dh = rand((m, k), dt, dev, 1900 + j), rand((m, n), dt, dev, 1910 + j, 0.5)
        w = rand((2 * n, k) if nk else (k, 2 * n), dt, dev, 1920 + j, 0.2)
        dw = torch.full_like(w, -7.0)
        halves = lambda t: (t[:n], t[n:]) if nk else (t[:, :n], t[:, n:])  # noqa: E731
        kt = F32 if kept == "fp32" else dt
        p = mm.GluPlan(m, k, n, mm.torch_dtype_code(dt), trans_w=nk, training=True, w_pitch=0 if nk else 2 * n,
                       kept_type=mm.torch_dtype_code(kt))
        h, g, u, dx = (torch.empty(s, dtype=t, device=dev) for s, t in (((m, n), dt), ((m, n), kt), ((m, n), kt), ((m, k), dt)))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        p.execute(x, *halves(w), h, g, u, stream=side)
        p.backward(x, *halves(w), g, u, dh, dx, *halves(dw), stream=side)
        torch.cuda.synchronize()
        wg, wu = (t.t() if nk else t for t in halves(w))
        within(h, *forward64(x, wg, wu, "silu", dt)[0], "H")
        ref = backward64(x, wg, wu, g, u, dh, "silu", dt)
        for t, r, name in zip((dx, *(v.t() if nk else v for v in halves(dw))), ref, ("dX", "dWg", "dWu")):
            within(t, *r, f"{name} {m}x{k}x{n}")
