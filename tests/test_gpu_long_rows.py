"""Rows of the operators around a residual block past 2^32 bytes and near the
limits of their sizes.

Tensors repeat a pattern of P values, P prime, so that an offset which wraps
reads other values.  Checkpoints and products by powers of two are exact.
"""
import numpy as np
import pytest

from onnx_broadcast_matmul_amd import binding as mm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_ffn import BF16, F16, F32, check_guard, guarded, rand  # noqa: E402
from test_gpu_linear import pack64  # noqa: E402

P = 1_000_003
FAR = 1 << 30  # FP32 elements in 2^32 bytes


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    mm.lib()
    return torch.device("cuda:0")


@pytest.fixture(autouse=True)
def empty():
    yield
    torch.cuda.empty_cache()


def fill(t, seed):
    """The pattern over a dense tensor: blocks of many magnitudes."""
    one = rand((P,), F32, t.device, seed) * torch.exp2(torch.arange(P, device=t.device) // 32 % 40 - 20.0)
    flat, one = t.view(-1), one.to(t.dtype)
    whole = flat.numel() // P * P
    flat[:whole].view(-1, P).copy_(one)
    flat[whole:].copy_(one[:flat.numel() - whole])
    return t


def signs(seed, shape, dt, dev):
    """The pattern of -1, 0 and 1."""
    n = int(np.prod(shape))
    one = (rand((P,), F32, dev, seed) * 1.5).round().clamp(-1, 1).to(dt)
    return one.repeat(-(-n // P))[:n].view(shape)


def blocks_to_check(cols):
    nb, rng = -(-cols // 32), np.random.default_rng(3)
    near = [0, 1, FAR // 32 - 1, FAR // 32, FAR // 32 + 1, nb - 3, nb - 2, nb - 1]
    return sorted(b for b in {*near, *rng.integers(0, nb, 20).tolist()} if 0 <= b < nb)


def check_checkpoint(x, q, s, back):
    cols = x.shape[1]
    for b in blocks_to_check(cols):
        at = slice(32 * b, min(32 * b + 32, cols))
        wq, ws, wv = pack64(x[:, at])
        assert np.array_equal(q[:, at].cpu().numpy(), wq) and np.array_equal(s[:, b:b + 1].cpu().numpy(), ws), b
        assert np.array_equal(back[:, at].double().cpu().numpy(), wv), b


def test_checkpoint_of_an_fp32_row_past_4gib(dev):
    cols = FAR + 69
    x = fill(torch.empty(1, cols, device=dev), 1)
    q, s = mm.checkpoint_pack(x)
    check_checkpoint(x, q, s, mm.checkpoint_unpack(q, s, F32))


def test_linear_backward_of_fp32_rows_past_4gib(dev):
    """One token, one input feature: dW = x dY where Z > 0."""
    n = FAR + 69
    p = mm.LinearPlan(1, 1, n, mm.FLOAT, activation=mm.ACT_RELU, training=True, force_algo=mm.ALGO_GENERAL, tile=2,
                      dx_tile=2, dw_tile=2)
    dy, z = fill(torch.empty(1, n, device=dev), 2), fill(torch.empty(1, n, device=dev), 3)
    dw = torch.empty(1, n, device=dev)
    p.backward(torch.full((1, 1), 2.0, device=dev), None, dy, Z=z, dW=dw)
    for i in range(0, n, 1 << 28):
        at = slice(i, min(i + (1 << 28), n))
        assert torch.equal(dw[:, at], torch.where(z[:, at] > 0, 2.0 * dy[:, at], 0.0)), i


@pytest.mark.parametrize("dt", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cols", [(1 << 31) - 1, (1 << 31) - 7, (1 << 31) - 31])
def test_checkpoint_of_the_longest_rows(cols, dt, dev):
    """The last piece ends at the row's last element: nothing behind it is
    written, and nothing behind it is read into the last block."""
    x, _ = guarded((1, cols), dt, dev)
    fill(x, 4)
    q, qbuf = guarded((1, cols), torch.int8, dev)
    s = torch.empty(1, mm.checkpoint_blocks(cols), dtype=torch.uint8, device=dev)
    mm.checkpoint_pack(x, q, s)
    back, bbuf = guarded((1, cols), dt, dev)
    mm.checkpoint_unpack(q, s, back)
    check_checkpoint(x, q, s, back)
    check_guard(qbuf, q)
    check_guard(bbuf, back)


def test_norm_of_as_many_rows_as_there_may_be(dev):
    """Rows of one column: the step behind the last ones passes 2^31.  With eps 1
    and r = 1 / sqrt(x^2 + 1), y = x r and dX = dsum + dout r^3."""
    m = (1 << 31) - 65
    p = mm.NormPlan(m, 1, mm.BFLOAT16, block=False, pre_weight=False, pre_eps=1.0, training=True)
    x, xbuf = guarded((m, 1), BF16, dev)
    flat = x.view(-1)
    one = (rand((P,), F32, dev, 5) * 3).to(BF16)
    whole = m // P * P
    flat[:whole].view(-1, P).copy_(one)
    flat[whole:].copy_(one[:m - whole])
    y, ybuf = guarded((m, 1), BF16, dev)
    stats = torch.empty(m, 4, device=dev)
    p.execute(x, y, stats=stats)
    dx, dbuf = guarded((m, 1), BF16, dev)
    p.backward(stats, sum=x, dout=y, dsum=x, dX=dx)
    torch.cuda.synchronize()
    for buf, t in ((xbuf, x), (ybuf, y), (dbuf, dx)):
        check_guard(buf, t)
    size = 1 << 26
    for i in sorted({*range(0, m, 7 * size), m - size}):
        at = slice(i, min(i + size, m))
        v = x[at].double()
        r = (v * v + 1) ** -0.5
        # a rounding to BF16, and some FP32 operations on values below 1
        assert bool(((y[at].double() - v * r).abs() <= 2.0 ** -8 * (v * r).abs() + 2.0 ** -21).all()), i
        want = v + y[at].double() * r ** 3
        assert bool(((dx[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * (1 + v.abs())).all()), i
        assert bool(((stats[at, 3].double() - r[:, 0]).abs() <= 2.0 ** -21 * r[:, 0]).all()), i


def test_linear_bias_gradient_of_many_columns(dev):
    """More columns than one dimension of a grid has threads for: of one row, dbias is dY."""
    n = (1 << 29) + 71
    p = mm.LinearPlan(1, 8, n, mm.BFLOAT16, bias=True, training=True, force_algo=mm.ALGO_GENERAL, tile=2)
    dy = fill(torch.empty(1, n, dtype=BF16, device=dev), 6)
    db, buf = guarded((n,), BF16, dev)
    p.backward(None, None, dy, dbias=db)
    torch.cuda.synchronize()
    assert torch.equal(db, dy[0])
    check_guard(buf, db)


@pytest.mark.parametrize("dt,nk", [(BF16, True), (F16, False)], ids=["bf16-nk", "fp16-kn"])
def test_linear_of_5gb_activations(dt, nk, dev):
    """Y, the residual, dY and the workspace's dZ past 2^32 bytes, Z's checkpoint
    past 2^31.  Whole numbers, so that sums are exact and results rounded once."""
    m, k, n = 65600, 64, 40008
    whole = lambda seed, *shape: signs(seed, shape, dt, dev)  # noqa: E731
    x, w, b = whole(1, m, k), whole(2, *((n, k) if nk else (k, n))), whole(3, n)
    r, dy = whole(4, m, n), whole(5, m, n)
    p = mm.LinearPlan(m, k, n, mm.torch_dtype_code(dt), activation=mm.ACT_RELU, trans_w=nk, bias=True, residual=True,
                      training=True, z_type=mm.INT8, x_type=mm.INT8)
    z, zs = torch.empty(m, n, dtype=torch.int8, device=dev), torch.empty(m, mm.checkpoint_blocks(n), dtype=torch.uint8, device=dev)
    y = torch.empty_like(r)
    p.execute(x, w, y, bias=b, residual=r, Z=z, z_scale=zs)
    xq, xs = mm.checkpoint_pack(x)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    p.backward(xq, w, dy, Z=z, z_scale=zs, x_scale=xs, dX=dx, dW=dw, dbias=db)
    wf = (w.t() if nk else w).float()
    sw, sb = torch.zeros(k, n, device=dev), torch.zeros(n, device=dev)
    for i in range(0, m, 8200):
        at = slice(i, i + 8200)
        z32 = x[at].float() @ wf + b.float()
        assert torch.equal(y[at].float(), z32.clamp_min(0) + r[at].float()), i
        assert torch.equal(mm.checkpoint_unpack(z[at], zs[at], F32), z32), i
        dz = dy[at].float() * (z32 > 0)
        assert torch.equal(dx[at], (dz @ wf.t()).to(dt)), i
        sw += x[at].float().t() @ dz
        sb += dz.sum(0)
    assert torch.equal(dw, (sw.t() if nk else sw).to(dt)) and torch.equal(db, sb.to(dt))


@pytest.mark.parametrize("algo", [0, mm.ALGO_GENERAL], ids=["few-rows", "tiles"])
@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
def test_linear_of_5gb_weights(nk, algo, dev):
    """W and dW past 2^32 bytes, of four rows.  Whole numbers as above."""
    m, k, n, dt = 4, 33000, 72008, BF16
    x, w, dy = signs(1, (m, k), dt, dev), signs(2, (n, k) if nk else (k, n), dt, dev), signs(3, (m, n), dt, dev)
    p = mm.LinearPlan(m, k, n, mm.BFLOAT16, trans_w=nk, training=True, force_algo=algo)
    assert mm.ALGO_NAMES[p.algo] == ("general" if algo else "skinny_m")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    p.execute(x, w, y)
    p.backward(x, w, dy, dX=dx, dW=dw)
    sums = torch.zeros(m, k, device=dev)
    for i in range(0, n, 9001):  # output features
        at = slice(i, i + 9001)
        part = (w[at].t() if nk else w[:, at]).float()
        assert torch.equal(y[:, at], (x.float() @ part).to(dt)), i
        sums += dy[:, at].float() @ part.t()
        assert torch.equal((dw[at].t() if nk else dw[:, at]).float(), x.float().t() @ dy[:, at].float()), i
    assert torch.equal(dx, sums.to(dt))
