"""GPU tests of the linear layer with its epilogue and backward pass and of the
8-bit activation checkpoints, against plain forms in 64 bits.

Tolerances are those of the feed-forward operators' tests (per element, from
the arithmetic: FP32 sums of n products within 2 n 2^-24 of the sum of
magnitudes, one rounding of half a step to the result's type, activations
within 2^-16 or 2^-19 of their magnitude).  Checkpoints are exact.
"""
import math

import numpy as np
import pytest

from onnx_broadcast_matmul_amd import binding as mm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_ffn import (BF16, F16, F32, TYPES, act64, act_error, check_guard, guarded, half_step, rand,  # noqa: E402
                          tiny, within)

ACTS = ["none"] + list(mm.ACTIVATIONS)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    mm.lib()
    return torch.device("cuda:0")


def code(act):
    return 0 if act == "none" else mm.ACTIVATIONS[act]


def f64(act, z):
    return (z, torch.ones_like(z)) if act == "none" else act64(act, z)


def act_e(act, dt):
    return 0.0 if act in ("none", "relu") else act_error(dt)


# ---- checkpoints


def pack64(x):
    """q and scale bytes of a tensor's rows, from the format's definition."""
    x = x.double().cpu().numpy()
    rows, cols = x.shape
    nb = -(-cols // 32)
    p = np.zeros((rows, nb * 32))
    p[:, :cols] = x
    p = p.reshape(rows, nb, 32)
    bad = ~np.isfinite(p).all(2)
    top = np.maximum(np.abs(np.where(np.isfinite(p), p, 0)).max(2), 2.0 ** -100)
    e = np.frexp(top)[1] - 1
    s = np.ldexp(1.0, e - 6)
    with np.errstate(invalid="ignore"):
        q = np.clip(np.rint(p / s[..., None]), -127, 127)
    q[bad] = 0
    v = q * s[..., None]
    v[bad] = np.nan
    cut = lambda a: np.ascontiguousarray(a.reshape(rows, nb * 32)[:, :cols])  # noqa: E731
    return cut(q).astype(np.int8), np.where(bad, 255, e + 127).astype(np.uint8), cut(v)


def hard_rows(rows, cols, dt, dev, seed):
    """Rows of every kind: magnitudes over the type's range, zeros, ties,
    values at a power of two's upper end, subnormals, infinities and NaN."""
    x = rand((rows, cols), F32, dev, seed)
    scale = torch.exp2(torch.linspace(-30, 15, rows, device=dev)) if dt == F16 else \
        torch.exp2(torch.linspace(-140, 127, rows, device=dev))
    x = (x.clamp(-1.9, 1.9) / 2 * scale[:, None]).to(dt)
    if rows > 8:
        x[1] = 0
        x[2] = torch.arange(cols, device=dev).to(dt) * 0.5 % 64  # halves: ties
        x[3] = torch.finfo(dt).max
        x[4] = -torch.finfo(dt).max
        x[5] = tiny(dt)
        x[6, cols // 2] = float("inf")
        x[7, cols - 1] = float("nan")
        x[8, 0] = -float("inf")
    return x


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols,offset", [(1, 1, 0), (3, 31, 1), (40, 32, 0), (33, 33, 3), (7, 127, 0), (64, 1000, 0),
                                              (19, 4099, 1), (300, 8, 0), (1, 70001, 0)])
def test_checkpoint(rows, cols, offset, dt, dev):
    t = TYPES[dt]
    x, _ = guarded((rows, cols), t, dev, offset)
    x.copy_(hard_rows(rows, cols, t, dev, 5))
    q, qbuf = guarded((rows, cols), torch.int8, dev, offset)
    s = torch.full((rows, mm.checkpoint_blocks(cols)), 99, dtype=torch.uint8, device=dev)
    back, bbuf = guarded((rows, cols), t, dev, offset)
    mm.checkpoint_pack(x, q, s)
    mm.checkpoint_unpack(q, s, back)
    torch.cuda.synchronize()
    wq, ws, wv = pack64(x)
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(back.double().cpu().numpy(), wv, equal_nan=True)
    check_guard(qbuf, q, offset)
    check_guard(bbuf, back, offset)
    # in FP32 too, and by results that the calls make
    q2, s2 = mm.checkpoint_pack(x)
    assert torch.equal(q2, q) and torch.equal(s2, s)
    assert np.array_equal(mm.checkpoint_unpack(q2, s2, F32).double().cpu().numpy(), wv, equal_nan=True)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_checkpoint_read_into_a_narrower_type(dt, dev):
    """Values of an FP32 tensor's checkpoint, rounded once to nearest even."""
    x = hard_rows(50, 100, F32, dev, 6)
    q, s = mm.checkpoint_pack(x)
    want = torch.from_numpy(pack64(x)[2]).to(F32).to(TYPES[dt])
    got = mm.checkpoint_unpack(q, s, TYPES[dt]).cpu()
    assert torch.equal(torch.nan_to_num(got.float(), 7.0, 8.0, 9.0), torch.nan_to_num(want.float(), 7.0, 8.0, 9.0))


def test_checkpoint_of_more_dimensions_and_none(dev):
    x = rand((3, 5, 70), BF16, dev, 7)
    q, s = mm.checkpoint_pack(x)
    assert q.shape == x.shape and s.shape == (3, 5, 3)
    q2, s2 = mm.checkpoint_pack(x.view(15, 70))
    assert torch.equal(q.view(15, 70), q2) and torch.equal(s.view(15, 3), s2)
    for shape in ((0, 40), (4, 0)):
        e = torch.empty(shape, dtype=BF16, device=dev)
        q, s = mm.checkpoint_pack(e)
        assert mm.checkpoint_unpack(q, s, BF16).shape == e.shape


# ---- linear layer, forward


def linear64(x, w, b, r, act, dt):
    """Y and Z in 64 bits with their tolerances, weights [K, N]; Z's own
    tolerance is that of its FP32 sum."""
    x, w = x.double(), w.double()
    z = x @ w
    ez = 2 * (x.shape[1] + 1) * 2.0 ** -24 * (x.abs() @ w.abs() + (0 if b is None else b.double().abs()))
    if b is not None:
        z = z + b.double()
    f, _ = f64(act, z)
    y = f if r is None else f + r.double()
    u = half_step(dt)
    # the sum with the residual is an FP32 operation of its own
    raw = 1.13 * ez + act_e(act, dt) * f.abs() + (0 if r is None else 2.0 ** -24 * y.abs())
    return (y, raw * (1 + u) + u * y.abs() + tiny(dt)), (z, ez)


def check_z8(z8, zs, z, ez):
    """Z's checkpoint: each value within half a step of Z, a step where the
    number is at its limit; the step from a block's largest magnitude."""
    s = torch.exp2(zs.double() - 133).repeat_interleave(32, dim=1)[:, :z.shape[1]]
    off = (z8.double() * s - z).abs() - ez
    limit = torch.where(z.abs() + ez > 127.5 * s, s, s / 2)
    assert bool((off <= limit).all()), f"Z off by {float((off - limit).max())} more than its step allows"
    pad = (0, -z.shape[1] % 32)
    blocks = lambda v: torch.nn.functional.pad(v, pad).reshape(z.shape[0], -1, 32).amax(2)  # noqa: E731
    top, e = blocks(z.abs()), blocks(ez)
    step = torch.exp2(zs.double() - 133)
    assert bool((step * 64 <= (top + e).clamp_min(2.0 ** -100)).all()) and bool((step * 128 > top - e).all())


def weight(k, n, dt, dev, nk, seed, pitched=False, offset=0, fill=None):
    """A weight and its pitch: dense, or the first part of wider rows."""
    shape = (n, k) if nk else (k, n)
    w = rand(shape, dt, dev, seed, max(k, 1) ** -0.5) if fill is None else torch.full(shape, fill, dtype=dt, device=dev)
    if pitched:
        wide = torch.full((shape[0], shape[1] + 24), -7.0, dtype=dt, device=dev)
        wide[:, :shape[1]] = w
        return wide[:, :shape[1]], shape[1] + 24
    if offset:
        t, _ = guarded(shape, dt, dev, offset)
        t.copy_(w)
        return t, 0
    return w, 0


def run_forward(dev, m, k, n, dt, nk, act, seed=0, bias=True, residual=True, z=None, offset=0, pitched=False, tile=0,
                algo=0, split=0, scale=1.0, inplace=False):
    x, _ = guarded((m, k), dt, dev, offset)
    x.copy_(rand((m, k), dt, dev, seed, scale))
    w, pitch = weight(k, n, dt, dev, nk, seed + 1, pitched, offset)
    b = rand((n,), dt, dev, seed + 2) if bias else None
    r = None
    y, buf = guarded((m, n), dt, dev, offset)
    if residual:
        r, _ = guarded((m, n), dt, dev, offset)
        r.copy_(rand((m, n), dt, dev, seed + 3))
    want, (z64, ez) = linear64(x, w.t() if nk else w, b, r, act, dt)
    if inplace:
        y.copy_(r)
        r = y
    keep = z is not None and act != "none"
    plan = mm.LinearPlan(m, k, n, mm.torch_dtype_code(dt), activation=code(act), trans_w=nk, bias=bias,
                         residual=residual, training=keep, z_type=(z or 0) if keep else 0, w_pitch=pitch,
                         force_algo=algo, tile=tile, split_k=split)
    kw = {}
    if keep:
        zt = {0: dt, mm.FLOAT: F32, mm.INT8: torch.int8}[z]
        kw["Z"], zbuf = guarded((m, n), zt, dev, offset)
        if z == mm.INT8:
            kw["z_scale"] = torch.zeros(m, mm.checkpoint_blocks(n), dtype=torch.uint8, device=dev)
    plan.execute(x, w, y, bias=b, residual=r, **kw)
    torch.cuda.synchronize()
    within(y, *want, f"Y {m}x{k}x{n}")
    check_guard(buf, y, offset)
    if keep:
        if z == mm.INT8:
            check_z8(kw["Z"], kw["z_scale"], z64, ez)
        else:
            u = half_step(zt)
            within(kw["Z"], z64, ez * (1 + u) + u * z64.abs() + tiny(zt), f"Z {m}x{k}x{n}")
        check_guard(zbuf, kw["Z"], offset)
    return plan


SIZES = [(1, 1, 1), (1, 64, 16), (1, 2048, 520), (3, 7, 5), (5, 72, 33), (16, 256, 160), (17, 264, 40), (32, 129, 96),
         (33, 200, 72), (64, 77, 55), (130, 136, 264), (257, 72, 131), (300, 512, 300), (40, 3000, 70)]
KEEP = [None, 0, mm.FLOAT, mm.INT8]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(SIZES)), ids=lambda i: "x".join(map(str, SIZES[i])))
def test_linear_forward(i, dt, nk, dev):
    run_forward(dev, *SIZES[i], TYPES[dt], nk, ACTS[i % 6], seed=10 + i, bias=i % 2 == 0, residual=i % 3 != 0,
                z=KEEP[i % 4])
    run_forward(dev, *SIZES[i], TYPES[dt], nk, ACTS[(i + 3) % 6], seed=30 + i, bias=i % 2 == 1, residual=i % 3 == 0,
                z=KEEP[(i + 2) % 4])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_linear_activations_over_a_wide_range(act, dt, dev):
    for m in (200, 9):
        run_forward(dev, m, 64, 96, TYPES[dt], True, act, seed=40, scale=10.0, z=mm.FLOAT)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("z", KEEP)
@pytest.mark.parametrize("dt,tile", [(d, t) for d in TYPES for t in ((2, 3, 4) if d == "fp32" else (1, 2, 3, 4, 5))])
def test_linear_every_tile(tile, z, nk, dt, dev):
    for j, (m, k, n) in enumerate(((530, 328, 400), (270, 16, 136), (300, 701, 281), (2, 35, 9))):
        if not (tile == 4 and z == mm.INT8):
            run_forward(dev, m, k, n, TYPES[dt], nk, "silu", seed=50 + j, tile=tile, algo=mm.ALGO_GENERAL, z=z)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt,tile", [(d, t) for d in TYPES for t in ((2, 3, 4) if d == "fp32" else (2, 3, 4, 5))])
def test_linear_split(tile, nk, dt, dev):
    for j, (m, k, n, split) in enumerate(((270, 1040, 136, 3), (50, 701, 281, 1000), (2, 35, 9, 2), (3, 2000, 61, 5))):
        p = run_forward(dev, m, k, n, TYPES[dt], nk, ACTS[j + 1], seed=55 + j, tile=tile, split=split, z=KEEP[3 - j])
        assert j == 2 or p.info()["algo_name"] == "split_k"


@pytest.mark.parametrize("m", [1, 16, 17, 32])
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_linear_few_rows(m, nk, dt, dev):
    for j, (k, n) in enumerate(((4096, 48), (1000, 33), (3, 2), (130, 515), (64, 20000))):
        run_forward(dev, m, k, n, TYPES[dt], nk, ACTS[j], seed=60 + j, algo=mm.ALGO_SKINNY_M, z=KEEP[j % 3])


@pytest.mark.parametrize("m", [1, 13, 32])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_linear_few_rows_off_dword_alignment(m, dt, dev):
    for j, (k, n, offset) in enumerate(((1301, 35, 0), (64, 20, 1), (1300, 40, 1), (67, 8209, 0))):
        run_forward(dev, m, k, n, TYPES[dt], True, "silu", seed=90 + j, algo=mm.ALGO_SKINNY_M, offset=offset)


@pytest.mark.parametrize("m", [4, 150])
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_linear_unaligned_pitched_and_in_place(m, nk, dev):
    run_forward(dev, m, 64, 96, BF16, nk, "gelu", seed=70, offset=1, z=mm.INT8)
    run_forward(dev, m, 64, 96, BF16, nk, "gelu", seed=71, offset=1, z=0)
    run_forward(dev, m, 64, 96, BF16, nk, "silu", seed=72, pitched=True)
    run_forward(dev, m, 65, 97, F16, nk, "silu", seed=73, pitched=True)
    run_forward(dev, m, 64, 96, F32, nk, "silu", seed=74, offset=1)
    for tile, split in ((0, 0), (2, 0), (3, 2), (4, 0)):
        run_forward(dev, m, 640, 100, BF16, nk, "relu", seed=75, inplace=True, tile=tile, split=split)


@pytest.mark.parametrize("m", [3, 200])
@pytest.mark.parametrize("z", [mm.FLOAT, mm.INT8])
def test_linear_empty_reduction_and_bad_rows(m, z, dev):
    b, r = rand((40,), BF16, dev, 1), rand((m, 40), BF16, dev, 2)
    p = mm.LinearPlan(m, 0, 40, mm.BFLOAT16, activation=mm.ACT_RELU, bias=True, residual=True)
    y = torch.full((m, 40), 5.0, dtype=BF16, device=dev)
    p.execute(torch.empty(m, 0, dtype=BF16, device=dev), torch.empty(0, 40, dtype=BF16, device=dev), y, b, r)
    assert torch.equal(y, (b.float().clamp_min(0) + r.float()).to(BF16))
    # a NaN and an infinity stay in their rows, in Z's checkpoint too
    x, w = rand((m, 64), BF16, dev, 80), rand((40, 64), BF16, dev, 81, 0.1)
    p = mm.LinearPlan(m, 64, 40, mm.BFLOAT16, activation=mm.ACT_SILU, trans_w=True, training=True, z_type=z)
    outs = []
    for bad in (False, True):
        if bad:
            x = x.clone()
            x[1, 5], x[2, 6] = float("nan"), float("inf")
        y = torch.empty(m, 40, dtype=BF16, device=dev)
        q = torch.empty(m, 40, dtype=torch.int8 if z == mm.INT8 else F32, device=dev)
        s = torch.empty(m, 2, dtype=torch.uint8, device=dev) if z == mm.INT8 else None
        p.execute(x, w, y, Z=q, z_scale=s)
        outs.append((y, q, s))
    (y0, q0, s0), (y1, q1, s1) = outs
    assert bool(y1[1].isnan().all()) and not bool(y1[2].isfinite().all())
    keep = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(y0[keep], y1[keep]) and torch.equal(q0[keep], q1[keep])
    if z == mm.INT8:
        assert torch.equal(s0[keep], s1[keep]) and bool((s1[1] == 255).all()) and bool((s1[2] == 255).all())


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("z", [None, mm.INT8])
def test_linear_more_large_tiles_than_cus(nk, z, dev):
    for j, (m, k, n) in enumerate(((4300, 128, 4624), (4500, 328, 4104))):
        run_forward(dev, m, k, n, (BF16, F16)[j], nk, "gelu_tanh", seed=95 + j, tile=1, algo=mm.ALGO_GENERAL, z=z)


LARGE = [(256, 64, 256), (1, 8, 8), (257, 72, 264), (300, 128, 520), (513, 136, 248), (255, 200, 1032), (40, 192, 40),
         (700, 1000, 72)]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("tile", [1, 5])
@pytest.mark.parametrize("i", range(len(LARGE)), ids=lambda i: "x".join(map(str, LARGE[i])))
def test_linear_large_tiles(i, tile, dt, nk, dev):
    """One stage of K and many, whole and in part, each kind of epilogue."""
    for j in range(4):
        p = run_forward(dev, *LARGE[i], TYPES[dt], nk, ACTS[(i + j) % 6], seed=900 + 10 * i + j, bias=j % 2 == 0,
                        residual=(i + j) % 3 != 0, z=KEEP[(i + j) % 4], tile=tile, algo=mm.ALGO_GENERAL)
        assert p.info()["tile"] == tile
    run_forward(dev, *LARGE[i], TYPES[dt], nk, "gelu", seed=990 + i, tile=tile, algo=mm.ALGO_GENERAL, inplace=True)


@pytest.mark.parametrize("z", KEEP)
@pytest.mark.parametrize("tile", [1, 5])
def test_linear_large_tiles_of_odd_columns(tile, z, dev):
    """Rows of X and W are whole 16-byte chunks, those of Y, Z and R are not."""
    for j, (m, k, n) in enumerate(((300, 128, 281), (520, 64, 515), (258, 264, 12), (3, 72, 1))):
        run_forward(dev, m, k, n, (BF16, F16)[j % 2], True, ACTS[1 + j], seed=930 + j, z=z, tile=tile, algo=mm.ALGO_GENERAL)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("z", KEEP)
def test_linear_whole_rounds_and_a_rest(nk, z, dev):
    """Two launches over the columns; every tensor starts anew at the second's."""
    for j, (m, k, n) in enumerate(((4100, 512, 5000), (4344, 520, 5016))):
        p = run_forward(dev, m, k, n, (BF16, F16)[j], nk, ("silu", "gelu_tanh")[j], seed=960 + j, z=z)
        assert 0 < p.info()["tail_col"] < n


@pytest.mark.parametrize("n,pitch", [(256, 4190000), (8, 1 << 22)])
def test_linear_rows_far_apart(n, pitch, dev):
    """A large tile's rows within 2^31 bytes of each other, and farther (other entries then)."""
    m, k = 300, 72
    wide = torch.empty(n, pitch, dtype=BF16, device=dev)
    w = wide[:, :k]
    w.copy_(rand((n, k), BF16, dev, 1, k ** -0.5))
    x, dy = rand((m, k), BF16, dev, 2), rand((m, n), BF16, dev, 3)
    for tile in (1, 5):
        p = mm.LinearPlan(m, k, n, mm.BFLOAT16, trans_w=True, training=True, w_pitch=pitch, force_algo=mm.ALGO_GENERAL,
                          tile=tile, dx_tile=tile, dw_tile=tile)
        y, dx = torch.empty(m, n, dtype=BF16, device=dev), torch.empty(m, k, dtype=BF16, device=dev)
        p.execute(x, w, y)
        within(y, *linear64(x, w.t(), None, None, "none", BF16)[0], "Y")
        p.backward(x, w, dy, dX=dx)
        within(dx, *backward64(x, torch.zeros_like(x).double(), w.t(), None, dy, "none", BF16)[0], "dX")


# ---- linear layer, backward


def backward64(x, ex, w, z, dy, act, dt):
    """dX, dW (weights [K, N]) and dbias in 64 bits from the given X (off by ex)
    and Z."""
    x, w, dy = x.double(), w.double(), dy.double()
    m, n = dy.shape
    d = torch.ones_like(dy) if act == "none" else f64(act, z.double())[1]
    dz = dy * d
    u, s = half_step(dt), 2.0 ** -24
    e0 = torch.zeros_like(dz) if act == "none" else act_e(act, dt) * dy.abs() * (1 + z.double().abs()) + 2 * s * dz.abs()
    e = e0 if act == "none" else e0 + u * dz.abs() + tiny(dt)
    narrow = lambda v, t: (v, t * (1 + u) + u * v.abs() + tiny(dt))  # noqa: E731
    dx = narrow(dz @ w.t(), e @ w.abs().t() + 2 * n * s * (dz.abs() @ w.abs().t()))
    dw = narrow(x.t() @ dz, x.abs().t() @ e + ex.t() @ (dz.abs() + e) + 2 * m * s * (x.abs().t() @ dz.abs()))
    db = narrow(dz.sum(0), e0.sum(0) + 2 * m * s * dz.abs().sum(0))
    return dx, dw, db


def run_backward(dev, m, k, n, dt, nk, act, seed=0, want="xwb", z=0, x8=False, x_act="none", offset=0, pitched=False,
                 **tiles):
    xv = rand((m, k), dt, dev, seed)
    zv = rand((m, n), F32, dev, seed + 1, 1.5)
    dy, _ = guarded((m, n), dt, dev, offset)
    dy.copy_(rand((m, n), dt, dev, seed + 2, 0.5))
    w, pitch = weight(k, n, dt, dev, nk, seed + 3, pitched, offset)
    dw, _ = weight(k, n, dt, dev, nk, seed + 4, pitched, offset, fill=-7.0)
    kw = {}
    x, ex = xv, torch.zeros(m, k, dtype=torch.float64, device=dev)
    given = xv
    if x8:
        given, kw["x_scale"] = mm.checkpoint_pack(xv)
        x = f64(x_act, torch.from_numpy(pack64(xv)[2]).to(dev))[0]
        if x_act != "none":
            ex = (act_e(x_act, dt) + half_step(dt)) * x.abs() + tiny(dt)
    zt = None
    if act != "none":
        if z == mm.INT8:
            kw["Z"], kw["z_scale"] = mm.checkpoint_pack(zv)
            zt = torch.from_numpy(pack64(zv)[2]).to(dev)
        else:
            kw["Z"] = zt = zv.to(F32 if z == mm.FLOAT else dt)
    plan = mm.LinearPlan(m, k, n, mm.torch_dtype_code(dt), activation=code(act), trans_w=nk, bias=True, training=True,
                         z_type=z if act != "none" else 0, x_type=mm.INT8 if x8 else 0, x_activation=code(x_act),
                         w_pitch=pitch, **tiles)
    dx, buf = guarded((m, k), dt, dev, offset)
    db, bbuf = guarded((n,), dt, dev, offset)
    plan.backward(given, w, dy, dX=dx if "x" in want else None, dW=dw if "w" in want else None,
                  dbias=db if "b" in want else None, **kw)
    torch.cuda.synchronize()
    ref = backward64(x, ex, w.t() if nk else w, zt, dy, act, dt)
    for name, t, r in (("x", dx, ref[0]), ("w", dw.t() if nk else dw, ref[1]), ("b", db, ref[2])):
        if name in want:
            within(t, *r, f"d{name} {m}x{k}x{n}")
        else:
            assert bool((t == -7).all())
    check_guard(buf, dx, offset)
    check_guard(bbuf, db, offset)
    if pitched:
        rest = torch.as_strided(dw, (dw.shape[0], 24), (dw.stride(0), 1), dw.storage_offset() + dw.shape[1])
        assert bool((rest == -7).all()), "wrote between the rows"
    return plan


BSIZES = [(1, 1, 1), (1, 64, 48), (2, 9, 3), (16, 128, 96), (33, 40, 72), (44, 882, 309), (130, 136, 264),
          (257, 71, 131), (300, 512, 364), (1200, 64, 72), (5000, 35, 42)]


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(BSIZES)), ids=lambda i: "x".join(map(str, BSIZES[i])))
def test_linear_backward(i, dt, nk, dev):
    run_backward(dev, *BSIZES[i], TYPES[dt], nk, ACTS[i % 6], seed=100 + 10 * i, z=KEEP[1 + i % 3], x8=i % 2 == 0)
    run_backward(dev, *BSIZES[i], TYPES[dt], nk, ACTS[(i + 3) % 6], seed=105 + 10 * i, z=KEEP[1 + (i + 1) % 3],
                 x8=i % 2 == 1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("z", [0, mm.FLOAT, mm.INT8])
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_linear_backward_activations(act, z, dt, dev):
    run_backward(dev, 70, 40, 56, TYPES[dt], True, act, seed=300, z=z, x8=True, x_act=act)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_linear_backward_variants(nk, dev):
    run_backward(dev, 600, 1040, 1032, BF16, nk, "silu", seed=400, z=mm.INT8, x8=True)  # large tiles
    for want in ("x", "w", "b", "wb", "xb"):
        run_backward(dev, 40, 64, 96, F16, nk, "silu", seed=410, want=want)
        run_backward(dev, 40, 64, 96, F16, nk, "none", seed=411, want=want, x8=True)
    run_backward(dev, 40, 64, 96, BF16, nk, "silu", seed=430, offset=1, z=mm.FLOAT)
    run_backward(dev, 40, 64, 96, BF16, nk, "none", seed=431, offset=1)
    run_backward(dev, 40, 64, 96, BF16, nk, "silu", seed=440, pitched=True)
    run_backward(dev, 41, 63, 95, F32, nk, "silu", seed=450, pitched=True, x8=True)
    run_backward(dev, 4360, 4616, 264, BF16, nk, "none", seed=460)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_linear_backward_every_entry(dt, nk, dev):
    for tile in (2, 3, 4) if dt == "fp32" else (1, 2, 3, 4, 5):
        dw = tile if not (tile == 4 and dt != "fp32") else 3
        for split in (0, 1) if tile == 1 else (0, 1, 3):
            p = run_backward(dev, 310, 296, 808, TYPES[dt], nk, "silu", seed=470, dx_tile=tile, dw_tile=dw,
                             dx_split_k=split, dw_split_k=split)
            d = p.desc()
            assert (d["dx_tile"], d["dw_tile"]) == (tile, dw)
            assert split == 0 or (d["dx_split_k"] == split and d["dw_split_k"] == split)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("tile", [1, 5])
def test_linear_backward_large_tiles(tile, dt, nk, dev):
    for j, (m, k, n) in enumerate(((1, 8, 8), (63, 264, 72), (64, 256, 256), (65, 40, 520), (130, 776, 264),
                                   (1000, 136, 328))):
        p = run_backward(dev, m, k, n, TYPES[dt], nk, ACTS[j], seed=940 + 10 * j, z=KEEP[1 + j % 3], x8=j % 2 == 0,
                         pitched=j == 3, dx_tile=tile, dw_tile=tile)
        d = p.desc()
        assert (d["dx_tile"], d["dw_tile"]) == (tile, tile)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_linear_backward_whole_rounds_and_a_rest(dt, nk, dev):
    """Sizes whose forward product runs so: dX's of the first, dW's of the others."""
    for j, (m, k, n) in enumerate(((4104, 5000, 512), (512, 5000, 4104), (512, 4104, 5000))):
        run_backward(dev, m, k, n, TYPES[dt], nk, "silu", seed=980 + j, z=mm.INT8, x8=j == 2)


def test_linear_backward_without_rows_or_features(dev):
    w = torch.zeros(24, 40, dtype=BF16, device=dev)
    dw, db = torch.full_like(w, 3.0), torch.full((40,), 3.0, dtype=BF16, device=dev)
    p = mm.LinearPlan(0, 24, 40, mm.BFLOAT16, activation=mm.ACT_SILU, bias=True, training=True, z_type=mm.INT8,
                      x_type=mm.INT8)
    e = lambda *s, t=BF16: torch.empty(*s, dtype=t, device=dev)  # noqa: E731
    p.backward(e(0, 24, t=torch.int8), w, e(0, 40), Z=e(0, 40, t=torch.int8), z_scale=e(0, 2, t=torch.uint8),
               x_scale=e(0, 1, t=torch.uint8), dX=e(0, 24), dW=dw, dbias=db)
    assert not bool(dw.any()) and not bool(db.any())
    dx = torch.full((5, 24), 3.0, dtype=BF16, device=dev)
    p = mm.LinearPlan(5, 24, 0, mm.BFLOAT16, training=True)
    p.backward(e(5, 24), e(24, 0), e(5, 0), dX=dx, dW=e(24, 0))
    assert not bool(dx.any())
    p = mm.LinearPlan(5, 0, 40, mm.BFLOAT16, bias=True, training=True)
    dy = rand((5, 40), BF16, dev, 3)
    p.backward(e(5, 0), e(0, 40), dy, dX=e(5, 0), dW=e(0, 40), dbias=db)
    within(db, dy.double().sum(0), 2.0 ** -8 * dy.double().sum(0).abs() + 1e-5, "dbias")


def test_linear_gradients_against_differences(dev):
    """FP32 gradients against central differences of the layer itself, in 64
    bits: (L(p + h d) - L(p - h d)) / 2 h for random directions d."""
    m, k, n, h = 12, 40, 33, 1e-4
    x, w, b, r = (rand(s, F32, dev, 500 + i) for i, s in enumerate(((m, k), (k, n), (n,), (m, n))))
    c = rand((m, n), F32, dev, 510)
    p = mm.LinearPlan(m, k, n, mm.FLOAT, activation=mm.ACT_GELU, bias=True, residual=True, training=True)
    y, z = torch.empty(m, n, device=dev), torch.empty(m, n, device=dev)
    p.execute(x, w, y, b, r, Z=z)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    p.backward(x, w, c, Z=z, dX=dx, dW=dw, dbias=db)
    loss = lambda x, w, b: (c.double() * (act64("gelu", x @ w + b)[0] + r.double())).sum()  # noqa: E731
    args = [t.double() for t in (x, w, b)]
    for i, g in enumerate((dx, dw, db)):
        d = rand(g.shape, F32, dev, 520 + i).double()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # the difference's own error is of the order h^2 times third
        # derivatives, which are a few times the gradient's scale
        scale = (g.double() * d).abs().sum()
        assert abs(float((g.double() * d).sum() - diff)) <= 1e-5 * float(scale), i


def test_linear_same_bits_every_time(dev):
    m, k, n = 700, 520, 328
    x, w, dy = rand((m, k), BF16, dev, 1), rand((n, k), BF16, dev, 2, 0.05), rand((m, n), BF16, dev, 3)
    b = rand((n,), BF16, dev, 4)
    outs = []
    p = mm.LinearPlan(m, k, n, mm.BFLOAT16, activation=mm.ACT_GELU, trans_w=True, bias=True, training=True,
                      z_type=mm.INT8, x_type=mm.INT8, dx_split_k=3, dw_split_k=4, dx_tile=2, dw_tile=2)
    xq, xs = mm.checkpoint_pack(x)
    for _ in range(3):
        y, dx, dw, db = torch.empty(m, n, dtype=BF16, device=dev), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
        z, zs = torch.empty(m, n, dtype=torch.int8, device=dev), torch.empty(m, 11, dtype=torch.uint8, device=dev)
        p.execute(x, w, y, b, Z=z, z_scale=zs)
        p.backward(xq, w, dy, Z=z, z_scale=zs, x_scale=xs, dX=dx, dW=dw, dbias=db)
        outs.append((y, z, zs, dx, dw, db))
    for o in outs[1:]:
        assert all(torch.equal(u, v) for u, v in zip(outs[0], o))


def test_linear_in_a_graph_and_on_another_stream(dev):
    """Forward and backward captured and replayed, eager work between, against
    eager results; then the same on a stream of its own."""
    m, k, n = 96, 128, 72
    w, b = rand((k, n), BF16, dev, 2, 0.1), rand((n,), BF16, dev, 4)
    p = mm.LinearPlan(m, k, n, mm.BFLOAT16, activation=mm.ACT_GELU, bias=True, training=True, z_type=mm.INT8,
                      x_type=mm.INT8, split_k=2, dx_split_k=2, dw_split_k=2)
    x, dy = rand((m, k), BF16, dev, 5), rand((m, n), BF16, dev, 6)
    xq, xs = mm.checkpoint_pack(x)
    z, zs = torch.empty(m, n, dtype=torch.int8, device=dev), torch.empty(m, 3, dtype=torch.uint8, device=dev)
    y, dx, dw, db = torch.empty(m, n, dtype=BF16, device=dev), torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)

    def step(stream=None):
        mm.checkpoint_pack(x, xq, xs, stream=stream)
        p.execute(x, w, y, b, Z=z, z_scale=zs, stream=stream)
        p.backward(xq, w, dy, Z=z, z_scale=zs, x_scale=xs, dX=dx, dW=dw, dbias=db, stream=stream)

    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    step()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        x.copy_(rand((m, k), BF16, dev, 20 + i))
        dy.copy_(rand((m, n), BF16, dev, 30 + i))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, z, zs, dx, dw, db)]
        for t in (y, z, zs, dx, dw, db):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, t) for a, t in zip(want, (y, z, zs, dx, dw, db))), i
        for t in (y, z, zs, dx, dw, db):
            t.zero_()
        side.wait_stream(torch.cuda.current_stream())
        step(side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, t) for a, t in zip(want, (y, z, zs, dx, dw, db))), i


def test_two_layers_from_checkpoints(dev):
    """Y = f(X W1 + b1) W2 + b2 + X as a training step uses the calls: only the
    checkpoints of X and of Z1 are kept, the second layer's X is f(Z1)."""
    m, k, n = 200, 96, 264
    for dt in (BF16, F32):
        c = mm.torch_dtype_code(dt)
        x, dy = rand((m, k), dt, dev, 1), rand((m, k), dt, dev, 2, 0.3)
        w1, w2 = rand((n, k), dt, dev, 3, k ** -0.5), rand((k, n), dt, dev, 4, n ** -0.5)
        b1, b2 = rand((n,), dt, dev, 5, 0.1), rand((k,), dt, dev, 6, 0.1)
        up = mm.LinearPlan(m, k, n, c, activation=mm.ACT_GELU_TANH, trans_w=True, bias=True, training=True,
                           z_type=mm.INT8, x_type=mm.INT8)
        down = mm.LinearPlan(m, n, k, c, trans_w=True, bias=True, residual=True, training=True, x_type=mm.INT8,
                             x_activation=mm.ACT_GELU_TANH)
        h, y = torch.empty(m, n, dtype=dt, device=dev), torch.empty(m, k, dtype=dt, device=dev)
        z, zs = torch.empty(m, n, dtype=torch.int8, device=dev), torch.empty(m, mm.checkpoint_blocks(n), dtype=torch.uint8, device=dev)
        xq, xs = mm.checkpoint_pack(x)
        up.execute(x, w1, h, b1, Z=z, z_scale=zs)
        down.execute(h, w2, y, b2, x)
        dh, dx = torch.empty_like(h), torch.empty_like(x)
        dw1, dw2, db1, db2 = (torch.empty_like(t) for t in (w1, w2, b1, b2))
        down.backward(z, w2, dy, x_scale=zs, dX=dh, dW=dw2, dbias=db2)
        up.backward(xq, w1, dh, Z=z, z_scale=zs, x_scale=xs, dX=dx, dW=dw1, dbias=db1)
        torch.cuda.synchronize()
        z64 = x.double() @ w1.double().t() + b1.double()
        y64 = act64("gelu_tanh", z64)[0] @ w2.double().t() + b2.double() + x.double()
        rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
        u = half_step(dt)
        assert rel(y, y64) < 4 * u + 1e-6  # H and Y rounded
        # gradients from the values that the checkpoints hold
        zv, xv = (mm.checkpoint_unpack(q, s, F32).double() for q, s in ((z, zs), (xq, xs)))
        f, d = act64("gelu_tanh", zv)
        dz = dh.double() * d
        for got, want in ((dh, dy.double() @ w2.double()), (dw2, dy.double().t() @ f), (db2, dy.double().sum(0)),
                          (dx, dz @ w1.double()), (dw1, dz.t() @ xv), (db1, dz.sum(0))):
            assert rel(got, want) < 3 * u + 1e-6
        # and those near the exact ones: 8 bits of a block of 32 are off by 2^-7
        # of its largest element at most, some 2^-7 of the norm
        f, d = act64("gelu_tanh", z64)
        dz = (dy.double() @ w2.double()) * d
        for got, want in ((dw2, dy.double().t() @ f), (dw1, dz.t() @ x.double()), (dx, dz @ w1.double())):
            assert rel(got, want) < 2.0 ** -6 + 4 * u
