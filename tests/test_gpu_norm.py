"""GPU tests of the norms around a block (residual, gate, residual scale) and
of their backward pass, against the formulas in 64 bits.

Tolerances follow the errors through the formulas: an FP32 operation is off by
2^-24 of its result, a sum of n terms by at most 2 n 2^-24 of the sum of their
magnitudes, and a result is rounded once to its type (half a step)."""
import numpy as np
import pytest

from onnx_broadcast_matmul_amd import binding as mm

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_ffn import BF16, F16, F32, TYPES, check_guard, guarded, half_step, rand, tiny, within  # noqa: E402
from test_gpu_linear import pack64  # noqa: E402

S = 2.0 ** -24
RMS, LAYER, NONE = mm.NORM_RMS, mm.NORM_LAYER, mm.NORM_NONE


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    mm.lib()
    return torch.device("cuda:0")


def mean(v):
    return v.mean(dim=1, keepdim=True)


def norm64(v, ev, kind, eps):
    """The normalised rows of v (off by ev), mean and r, and how far the first
    may be off."""
    n = v.shape[1]
    m = mean(v) if kind == LAYER else torch.zeros_like(v[:, :1])
    em = mean(ev) + 2 * n * S * mean(v.abs()) if kind == LAYER else 0 * m
    d = v - m
    ed = ev + em + S * (v.abs() + m.abs())
    var = mean(d * d)
    evar = 2 * mean(d.abs() * ed) + mean(ed * ed) + 2 * (n + 2) * S * var
    r = (var + eps) ** -0.5
    er = ((var - evar).clamp_min(0) + eps) ** -0.5 - r + 6 * S * r
    hat = d * r
    return hat, m, r, ed * (r + er) + d.abs() * er + 3 * S * hat.abs()


def narrow(v, e, dt):
    u = half_step(dt)
    return v, e * (1 + u) + u * v.abs() + tiny(dt)


def rows_of(gate, gr, m):
    return gate[torch.arange(m, device=gate.device) // gr]


class Case:
    """A plan with its operands."""

    def __init__(self, dev, m, n, dt, pre=RMS, post=NONE, block=True, pw=True, pb=False, qw=True, qb=False, gr=0,
                 alpha=1.0, kept=0, training=True, seed=0, offset=0, eps=1e-5, shift=0.0):
        self.dev, self.m, self.n, self.dt, self.offset, self.eps = dev, m, n, dt, offset, eps
        self.pre, self.post, self.kept, self.alpha, self.gr = pre, post, kept, alpha, gr if block else 0
        if not block:
            self.post = post = NONE
        if pre == NONE and self.post == NONE:
            self.pre = pre = LAYER

        def make(i, *shape, scale=1.0, add=0.0):
            t, _ = guarded(shape, dt, dev, offset)
            return t.copy_(rand(shape, F32, dev, seed + i, scale) + add)

        self.x = make(0, m, n, add=shift)
        self.b = make(1, m, n, scale=2.0, add=shift) if block else None
        self.g = make(2, -(-m // gr), n) if self.gr else None
        self.w1 = make(3, n) if post and qw else None
        self.b1 = make(4, n) if post and qb else None
        self.w2 = make(5, n) if pre and pw else None
        self.b2 = make(6, n) if pre and pb else None
        self.dy = make(7, m, n, scale=0.5) if pre else None
        self.ds = make(8, m, n, scale=0.5)
        self.plan = mm.NormPlan(m, n, mm.torch_dtype_code(dt), pre=pre, post=post, block=block,
                                pre_weight=self.w2 is not None, pre_bias=self.b2 is not None,
                                post_weight=self.w1 is not None, post_bias=self.b1 is not None, gate_rows=self.gr,
                                residual_scale=alpha, pre_eps=eps, post_eps=eps, training=training,
                                kept_type=kept if training else 0)

    def fresh(self, *shape, dt=None, fill=None):
        return guarded(shape, dt or self.dt, self.dev, self.offset)

    def forward64(self):
        f = lambda t: None if t is None else t.double()  # noqa: E731
        x, b = f(self.x), f(self.b)
        zero = torch.zeros_like(x)
        m1, r1 = zero[:, :1], zero[:, :1] + 1
        if b is None:
            r, er = x, zero
        else:
            n1, e = b, zero
            if self.post:
                n1, m1, r1, e = norm64(b, zero, self.post, self.eps)
                if self.w1 is not None:
                    n1, e = n1 * f(self.w1), e * f(self.w1).abs()
                if self.b1 is not None:
                    e = e + 2 * S * (n1.abs() + f(self.b1).abs())
                    n1 = n1 + f(self.b1)
                e = e + S * n1.abs()
            c = self.alpha * (rows_of(f(self.g), self.gr, self.m) if self.gr else torch.ones_like(x))
            r = x + c * n1
            er = c.abs() * e + 3 * S * ((c * n1).abs() + x.abs())
        out = {"sum": (r, er)}
        m2, r2 = zero[:, :1], zero[:, :1] + 1
        if self.pre:
            y, m2, r2, e = norm64(r, er, self.pre, self.eps)
            if self.w2 is not None:
                y, e = y * f(self.w2), e * f(self.w2).abs()
            if self.b2 is not None:
                e = e + 2 * S * (y.abs() + f(self.b2).abs())
                y = y + f(self.b2)
            out["out"] = (y, e + S * y.abs())
        out["stats"] = torch.cat([m1, r1, m2, r2], dim=1)
        return out

    def check_forward(self, checkpoints=True, inplace=False):
        m, n, dt = self.m, self.n, self.dt
        want = self.forward64()
        train = self.plan.training
        r, rbuf = self.fresh(m, n)
        y, ybuf = self.fresh(m, n) if self.pre else (None, None)
        kw, cks = {}, {}
        if train:
            kw["stats"] = torch.full((m, 4), -7.0, device=self.dev)
            if self.kept == mm.FLOAT:
                kw["sum_f32"], fbuf = self.fresh(m, n, dt=F32)
            if checkpoints:
                for name in ("sum", "block", "out"):
                    if (name == "block" and self.b is None) or (name == "out" and not self.pre):
                        continue
                    q, qbuf = self.fresh(m, n, dt=torch.int8)
                    s = torch.zeros(m, mm.checkpoint_blocks(n), dtype=torch.uint8, device=self.dev)
                    cks[name] = (q, s, qbuf)
                    kw[name + "_checkpoint"] = (q, s)
        x, b = self.x, self.b
        if inplace:
            r.copy_(x)
            x = r
            if y is not None and b is not None:
                y.copy_(b)
                b = y
        self.plan.execute(x, y, block=b, sum=r, gate=self.g, pre_weight=self.w2, pre_bias=self.b2, post_weight=self.w1,
                          post_bias=self.b1, **kw)
        torch.cuda.synchronize()
        within(r, *narrow(*want["sum"], dt), f"sum {m}x{n}")
        check_guard(rbuf, r, self.offset)
        if self.pre:
            within(y, *narrow(*want["out"], dt), f"out {m}x{n}")
            check_guard(ybuf, y, self.offset)
        for name, (q, s, qbuf) in cks.items():
            of = {"sum": r, "block": self.b, "out": y}[name]
            wq, ws, _ = pack64(of)
            assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws), name
            check_guard(qbuf, q, self.offset)
        if train:
            st = kw["stats"].double()
            scale = torch.cat([mean(self.b.double().abs()) if self.b is not None else 0 * st[:, :1] + 1, st[:, 1:2].abs(),
                               mean(r.double().abs()), st[:, 3:].abs()], dim=1)
            # means within 2 n 2^-24 of the mean magnitude; r as the rows it makes
            assert bool(((st - want["stats"]).abs()[:, 0::2] <= (4 * n + 8) * S * scale[:, 0::2] + 1e-30).all())
            if self.kept == mm.FLOAT:
                within(kw["sum_f32"], want["sum"][0], want["sum"][1] + tiny(F32), "sum_f32")
                check_guard(fbuf, kw["sum_f32"], self.offset)
        return r, y, kw

    def backward64(self, r, b, st):
        """The gradients from the given R, B (64 bits) and statistics."""
        f = lambda t: None if t is None else t.double()  # noqa: E731
        m, n = self.m, self.n
        m1, r1, m2, r2 = (st.double()[:, i:i + 1] for i in range(4))
        ds = f(self.ds) if self.ds is not None else torch.zeros(m, n, dtype=torch.float64, device=self.dev)
        out = {}

        def through(d, ed, x, ex, rr, kind):
            p, ep = mean(d * x), (2 * n + 4) * S * mean((d * x).abs()) + mean(d.abs() * ex + ed * (x.abs() + ex))
            q, eq = (mean(d), 2 * n * S * mean(d.abs()) + mean(ed)) if kind == LAYER else (0 * p, 0 * p)
            v = d - q - x * p
            return rr * v, rr * (ed + eq + x.abs() * ep + ex * (p.abs() + ep) + 4 * S * (d.abs() + q.abs() + (x * p).abs()))

        def column(v, ev):
            return v.sum(0), ev.sum(0) + 2 * v.shape[0] * S * v.abs().sum(0)

        if self.pre:
            x2 = (r - m2) * r2
            ex2 = 3 * S * (r.abs() + m2.abs()) * r2
            dy = f(self.dy)
            d2 = dy * f(self.w2) if self.w2 is not None else dy
            v, e = through(d2, S * d2.abs(), x2, ex2, r2, self.pre)
            dr, edr = ds + v, e + 2 * S * (v.abs() + ds.abs())
            out["dpre_weight"] = column(dy * x2, dy.abs() * ex2 + S * (dy * x2).abs())
            out["dpre_bias"] = column(dy, 0 * dy)
        else:
            dr, edr = ds, 0 * ds
        out["dX"] = (dr, edr)
        if self.b is not None:
            c = self.alpha * (rows_of(f(self.g), self.gr, m) if self.gr else torch.ones_like(dr))
            dn, edn = c * dr, c.abs() * edr + 2 * S * (c * dr).abs()
            x1, ex1 = (b - m1) * r1, 3 * S * (b.abs() + m1.abs()) * r1
            if not self.post:
                x1, ex1 = b, 0 * b
            n1, en1 = x1, ex1
            if self.w1 is not None:
                n1, en1 = n1 * f(self.w1), en1 * f(self.w1).abs() + S * (n1 * f(self.w1)).abs()
            if self.b1 is not None:
                en1 = en1 + 2 * S * (n1.abs() + f(self.b1).abs())
                n1 = n1 + f(self.b1)
            if self.gr:
                v = self.alpha * dr * n1
                ev = abs(self.alpha) * (edr * (n1.abs() + en1) + dr.abs() * en1) + 3 * S * v.abs()
                owner = torch.arange(m, device=self.dev) // self.gr
                add = lambda t: torch.zeros(self.g.shape, dtype=torch.float64, device=self.dev).index_add_(0, owner, t)  # noqa: E731
                out["dgate"] = (add(v), add(ev) + 2 * self.gr * S * add(v.abs()))
            if self.post:
                out["dpost_weight"] = column(dn * x1, edn * (x1.abs() + ex1) + dn.abs() * ex1 + S * (dn * x1).abs())
                out["dpost_bias"] = column(dn, edn)
                d1 = dn * f(self.w1) if self.w1 is not None else dn
                e1 = (edn * f(self.w1).abs() if self.w1 is not None else edn) + S * d1.abs()
                out["dblock"] = through(d1, e1, x1, ex1, r1, self.post)
            else:
                out["dblock"] = (dn, edn)
        return out

    def results(self):
        """Buffers for every gradient that the plan has."""
        have = {"dX": self.x, "dblock": self.b, "dgate": self.g, "dpre_weight": self.w2, "dpre_bias": self.b2,
                "dpost_weight": self.w1, "dpost_bias": self.b1}
        return {k: self.fresh(*t.shape) for k, t in have.items() if t is not None}

    def check_backward(self, want=None, seed=50, inplace=False):
        """want: the names of the gradients that are asked for (None: all)."""
        m, n, dt = self.m, self.n, self.dt
        # R and B as the backward pass is given them: of their own, so that
        # only this pass is tested
        r = rand((m, n), F32, self.dev, seed, 1.7)
        r = r if self.kept == mm.FLOAT else r.to(dt)
        b = self.b
        st = torch.cat([t.float() for t in (0.1 * rand((m, 1), F32, self.dev, seed + 1), 0.5 + rand((m, 1), F32, self.dev, seed + 2).abs(),
                                            0.1 * rand((m, 1), F32, self.dev, seed + 3), 0.5 + rand((m, 1), F32, self.dev, seed + 4).abs())], dim=1).contiguous()
        give_r, give_b, rv, bv = r, b, r.double(), None if b is None else b.double()
        if self.kept == mm.INT8:
            give_r, rv = mm.checkpoint_pack(r), torch.from_numpy(pack64(r)[2]).to(self.dev)
            if b is not None:
                give_b, bv = mm.checkpoint_pack(b), torch.from_numpy(pack64(b)[2]).to(self.dev)
        res = self.results()
        dy, ds = self.dy, self.ds
        if inplace:
            res["dX"][0].copy_(ds)
            ds = res["dX"][0]
            if dy is not None and "dblock" in res:
                res["dblock"][0].copy_(dy)
                dy = res["dblock"][0]
        asked = {k: v[0] for k, v in res.items() if want is None or k in want}
        self.plan.backward(st, sum=give_r if self.pre else None, block=give_b, dout=dy, dsum=ds, gate=self.g,
                           pre_weight=self.w2, post_weight=self.w1, post_bias=self.b1, **asked)
        torch.cuda.synchronize()
        ref = self.backward64(rv, bv, st)
        for k, (t, buf) in res.items():
            if k in asked:
                within(t, *narrow(*ref[k], dt), f"{k} {m}x{n}")
            else:
                assert bool((t == -7).all()), k
            check_guard(buf, t, self.offset)


SIZES = [(1, 1), (1, 64), (3, 33), (4, 512), (5, 513), (130, 1000), (33, 1024), (17, 1025), (9, 2048), (7, 4096), (6, 4099),
         (5, 8192), (4, 8200), (3, 16384), (1000, 40), (2600, 72), (700, 2056)]
KINDS = [dict(pre=RMS), dict(pre=LAYER, pb=True), dict(pre=RMS, block=False), dict(pre=LAYER, block=False, pw=False),
         dict(pre=RMS, post=RMS), dict(pre=LAYER, post=LAYER, qb=True, pb=True), dict(pre=NONE, post=RMS),
         dict(pre=NONE, post=LAYER, qw=False, qb=True), dict(pre=RMS, post=LAYER, qw=False, pw=False)]


def gate_rows(j, m):
    return (0, m, 1, max(1, m // 3), 7)[j % 5]


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(SIZES)), ids=lambda i: "x".join(map(str, SIZES[i])))
def test_norm_forward(i, dt, dev):
    m, n = SIZES[i]
    for j, kind in enumerate(KINDS):
        Case(dev, m, n, TYPES[dt], seed=10 * j, gr=gate_rows(i + j, m), alpha=(1.0, -0.5)[j % 2], training=j % 3 != 0,
             kept=(0, mm.FLOAT, mm.INT8)[(i + j) % 3], **kind).check_forward()


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(SIZES)), ids=lambda i: "x".join(map(str, SIZES[i])))
def test_norm_backward(i, dt, dev):
    m, n = SIZES[i]
    for j, kind in enumerate(KINDS):
        Case(dev, m, n, TYPES[dt], seed=10 * j, gr=gate_rows(i + j, m), alpha=(1.0, -0.5)[j % 2],
             kept=(0, mm.INT8, mm.FLOAT)[(i + j) % 3], **kind).check_backward()


@pytest.mark.parametrize("dt", TYPES, ids=str)
@pytest.mark.parametrize("offset", [1, 3])
def test_norm_off_alignment(offset, dt, dev):
    for m, n in ((5, 64), (9, 1001), (3, 4096)):
        for kept in (0, mm.INT8, mm.FLOAT):
            c = Case(dev, m, n, TYPES[dt], pre=LAYER, post=RMS, pb=True, qb=True, gr=2, kept=kept, offset=offset)
            c.check_forward()
            c.check_backward()


@pytest.mark.parametrize("gr", [1, 2, 3, 5, 8, 13, 64, 299, 300, 100000])
@pytest.mark.parametrize("m,n", [(300, 40), (2600, 72), (1030, 1040), (600, 4096)])
def test_norm_gates_of_every_length(gr, m, n, dev):
    """Groups that are whole within a worker, that end inside one, that several
    share; the last one short."""
    Case(dev, m, n, BF16, post=RMS, gr=gr, alpha=0.7).check_forward(checkpoints=False)
    Case(dev, m, n, BF16, post=RMS, gr=gr, alpha=0.7).check_backward()


@pytest.mark.parametrize("kept", [0, mm.INT8])
def test_norm_some_gradients(kept, dev):
    names = ["dX", "dblock", "dgate", "dpre_weight", "dpre_bias", "dpost_weight", "dpost_bias"]
    for want in [[k] for k in names] + [names[:1] + names[3:4], names[1:3], names[2:]]:
        Case(dev, 70, 200, F16, pre=LAYER, post=LAYER, pb=True, qb=True, gr=9, kept=kept).check_backward(want)
        Case(dev, 70, 200, F16, pre=RMS, gr=9, kept=kept).check_backward([k for k in want if k in ("dX", "dblock", "dgate", "dpre_weight")])


@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_norm_in_place(dt, dev):
    for m, n in ((70, 200), (5, 4099), (40, 1000)):
        for kind in (dict(pre=RMS), dict(pre=LAYER, post=RMS, gr=3)):
            Case(dev, m, n, TYPES[dt], **kind).check_forward(inplace=True)
            Case(dev, m, n, TYPES[dt], **kind).check_backward(inplace=True)


@pytest.mark.parametrize("dt", TYPES, ids=str)
def test_norm_without_the_residual_gradient(dt, dev):
    c = Case(dev, 33, 700, TYPES[dt], post=RMS)
    c.ds = None
    c.check_backward()


def test_norm_of_a_large_mean_and_of_constant_rows(dev):
    """A layer norm's variance is a sum of differences: a mean of a thousand
    deviations costs no digits; a constant row is 0 times 1 / sqrt(eps)."""
    Case(dev, 20, 1000, F32, pre=LAYER, shift=1000.0).check_forward()
    Case(dev, 20, 5000, F32, pre=LAYER, post=LAYER, shift=300.0).check_forward()
    for n in (64, 1000, 5000):
        x = torch.full((3, n), 2.5, dtype=BF16, device=dev)
        y = torch.empty_like(x)
        mm.NormPlan(3, n, mm.BFLOAT16, pre=LAYER, block=False, pre_weight=False).execute(x, y)
        assert not bool(y.any())
        x.zero_()
        mm.NormPlan(3, n, mm.BFLOAT16, pre=RMS, block=False, pre_weight=False).execute(x, y)
        assert not bool(y.any())


def test_norm_bad_rows_stay_alone(dev):
    for n in (70, 1000, 4096):
        m = 9
        c = Case(dev, m, n, BF16, post=RMS, gr=m)
        r0, y0, kw0 = c.check_forward()
        c.b[2, n // 2] = float("nan")
        c.x[5, n - 1] = float("inf")
        r1, y1 = torch.empty_like(r0), torch.empty_like(y0)
        ck = tuple(t.clone() for t in kw0["out_checkpoint"])
        c.plan.execute(c.x, y1, block=c.b, sum=r1, gate=c.g, pre_weight=c.w2, post_weight=c.w1, out_checkpoint=ck)
        keep = [i for i in range(m) if i not in (2, 5)]
        assert torch.equal(r0[keep], r1[keep]) and torch.equal(y0[keep], y1[keep])
        assert torch.equal(ck[0][keep], kw0["out_checkpoint"][0][keep]) and torch.equal(ck[1][keep], kw0["out_checkpoint"][1][keep])
        assert bool(y1[2].isnan().all()) and bool((ck[1][2] == 255).all())
        # an infinite row: 0 where finite, infinity times 0 where not
        assert bool((y1[5, :n - 1] == 0).all()) and bool(y1[5, n - 1].isnan())
        # backward: the row's own gradients, and sums over rows
        st, dx = kw0["stats"].clone(), torch.empty_like(r0)
        st2 = st.clone()
        st2[2, 3] = float("nan")
        clean = torch.empty_like(dx)
        c.plan.backward(st, sum=r0, block=c.b.nan_to_num(), dout=c.dy, dsum=c.ds, gate=c.g, pre_weight=c.w2, post_weight=c.w1, dX=clean)
        c.plan.backward(st2, sum=r0, block=c.b.nan_to_num(), dout=c.dy, dsum=c.ds, gate=c.g, pre_weight=c.w2, post_weight=c.w1, dX=dx)
        keep = [i for i in range(m) if i != 2]
        assert torch.equal(clean[keep], dx[keep]) and bool(dx[2].isnan().all())


def test_norm_without_rows_or_columns(dev):
    e = lambda *s, t=BF16: torch.empty(*s, dtype=t, device=dev)  # noqa: E731
    p = mm.NormPlan(0, 40, mm.BFLOAT16, post=RMS, post_weight=True, pre_bias=True, gate_rows=4, training=True)
    w = torch.ones(40, dtype=BF16, device=dev)
    p.execute(e(0, 40), e(0, 40), block=e(0, 40), sum=e(0, 40), gate=e(0, 40), pre_weight=w, pre_bias=w, post_weight=w)
    dw1, dw2, db2 = (torch.full((40,), 3.0, dtype=BF16, device=dev) for _ in range(3))
    p.backward(e(0, 4, t=F32), sum=e(0, 40), block=e(0, 40), dout=e(0, 40), dsum=e(0, 40), gate=e(0, 40), pre_weight=w,
               post_weight=w, dX=e(0, 40), dblock=e(0, 40), dgate=e(0, 40), dpre_weight=dw2, dpre_bias=db2, dpost_weight=dw1)
    assert not bool(dw1.any()) and not bool(dw2.any()) and not bool(db2.any())
    p = mm.NormPlan(4, 0, mm.BFLOAT16, training=True)
    p.execute(e(4, 0), e(4, 0), block=e(4, 0), pre_weight=e(0))
    p.backward(e(4, 4, t=F32), sum=e(4, 0), dout=e(4, 0), pre_weight=e(0), dX=e(4, 0), dpre_weight=e(0))


def test_norm_gradients_against_differences(dev):
    """FP32 gradients against central differences of the formulas in 64 bits,
    in random directions of each operand."""
    m, n, h = 12, 50, 1e-5
    c = Case(dev, m, n, F32, pre=LAYER, post=RMS, pb=True, qb=True, gr=5, alpha=0.6, kept=mm.FLOAT)
    st, r32 = torch.empty(m, 4, device=dev), torch.empty(m, n, device=dev)
    y = torch.empty(m, n, device=dev)
    c.plan.execute(c.x, y, block=c.b, gate=c.g, pre_weight=c.w2, pre_bias=c.b2, post_weight=c.w1, post_bias=c.b1, stats=st,
                   sum_f32=r32)
    res = {k: v[0] for k, v in c.results().items()}
    c.plan.backward(st, sum=r32, block=c.b, dout=c.dy, dsum=c.ds, gate=c.g, pre_weight=c.w2, post_weight=c.w1,
                    post_bias=c.b1, **res)

    def loss(x, b, g, w2, b2, w1, b1):
        n1 = b * ((b * b).mean(1, keepdim=True) + c.eps) ** -0.5 * w1 + b1
        r = x + 0.6 * rows_of(g, 5, m) * n1
        d = r - mean(r)
        out = d * (mean(d * d) + c.eps) ** -0.5 * w2 + b2
        return (c.ds.double() * r + c.dy.double() * out).sum()

    args = [t.double() for t in (c.x, c.b, c.g, c.w2, c.b2, c.w1, c.b1)]
    for i, k in enumerate(("dX", "dblock", "dgate", "dpre_weight", "dpre_bias", "dpost_weight", "dpost_bias")):
        d = rand(args[i].shape, F32, dev, 80 + i).double()
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * d, args[i] - h * d
        diff = (loss(*up) - loss(*down)) / (2 * h)
        # FP32 gradients: some 2^-20 of each term; the difference's own error is h^2
        assert abs(float((res[k].double() * d).sum() - diff)) <= 1e-5 * float((res[k].double() * d).abs().sum()), k


def test_norm_same_bits_in_a_graph_and_on_another_stream(dev):
    m, n = 500, 1032
    c = Case(dev, m, n, BF16, post=RMS, gr=130, kept=mm.INT8)
    r, y, st = torch.empty(m, n, dtype=BF16, device=dev), torch.empty(m, n, dtype=BF16, device=dev), torch.empty(m, 4, device=dev)
    ck = [(torch.empty(m, n, dtype=torch.int8, device=dev), torch.empty(m, 33, dtype=torch.uint8, device=dev)) for _ in range(2)]
    res = {k: v[0] for k, v in c.results().items()}

    def step(stream=None):
        c.plan.execute(c.x, y, block=c.b, sum=r, gate=c.g, pre_weight=c.w2, post_weight=c.w1, stats=st, sum_checkpoint=ck[0],
                       block_checkpoint=ck[1], stream=stream)
        c.plan.backward(st, sum=ck[0], block=ck[1], dout=c.dy, dsum=c.ds, gate=c.g, pre_weight=c.w2, post_weight=c.w1,
                        stream=stream, **res)

    outs = [r, y, st, *ck[0], *ck[1], *res.values()]
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    side = torch.cuda.Stream()
    for i in range(4):
        for t in (c.x, c.b, c.dy, c.ds):
            t.copy_(rand((m, n), BF16, dev, 90 + i))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for how in ("replay", "side"):
            for t in outs:
                t.zero_()
            if how == "replay":
                g.replay()
            else:
                side.wait_stream(torch.cuda.current_stream())
                step(side)
                torch.cuda.current_stream().wait_stream(side)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, outs)), (i, how)


def test_residual_block_from_checkpoints(dev):
    """A residual block as a training step uses the calls: R = X + B, N = norm(R),
    H = gelu(N W1 + b1), Y = H W2 + b2 + R; kept are the checkpoints of R, N and Z1."""
    m, n, hid, dt, c = 150, 96, 264, F32, mm.FLOAT
    x, b, dy = (rand((m, n), dt, dev, i) for i in (1, 2, 3))
    w, w1, w2 = 1 + rand((n,), dt, dev, 4, 0.1), rand((hid, n), dt, dev, 5, n ** -0.5), rand((n, hid), dt, dev, 6, hid ** -0.5)
    b1, b2 = rand((hid,), dt, dev, 7), rand((n,), dt, dev, 8)
    norm = mm.NormPlan(m, n, c, training=True, kept_type=mm.INT8, pre_eps=1e-5)
    up = mm.LinearPlan(m, n, hid, c, activation=mm.ACT_GELU, trans_w=True, bias=True, training=True, z_type=mm.INT8, x_type=mm.INT8)
    down = mm.LinearPlan(m, hid, n, c, trans_w=True, bias=True, residual=True, training=True, x_type=mm.INT8,
                         x_activation=mm.ACT_GELU)
    ck = lambda k: (torch.empty(m, k, dtype=torch.int8, device=dev), torch.empty(m, mm.checkpoint_blocks(k), dtype=torch.uint8, device=dev))  # noqa: E731
    r, nn, h, y, st = torch.empty_like(x), torch.empty_like(x), torch.empty(m, hid, device=dev), torch.empty_like(x), torch.empty(m, 4, device=dev)
    rk, nk, zk = ck(n), ck(n), ck(hid)
    norm.execute(x, nn, block=b, sum=r, pre_weight=w, stats=st, sum_checkpoint=rk, out_checkpoint=nk)
    up.execute(nn, w1, h, b1, Z=zk[0], z_scale=zk[1])
    down.execute(h, w2, y, b2, r)
    dh, dn, dx, db, dw = torch.empty_like(h), torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    dw1, dw2, db1, db2 = (torch.empty_like(t) for t in (w1, w2, b1, b2))
    down.backward(zk[0], w2, dy, x_scale=zk[1], dX=dh, dW=dw2, dbias=db2)
    up.backward(nk[0], w1, dh, Z=zk[0], z_scale=zk[1], x_scale=nk[1], dX=dn, dW=dw1, dbias=db1)
    norm.backward(st, sum=rk, dout=dn, dsum=dy, pre_weight=w, dX=dx, dblock=db, dpre_weight=dw)
    torch.cuda.synchronize()
    leaves = [t.double().cpu().requires_grad_() for t in (x, b, w, w1, w2, b1, b2)]
    X, B, W, W1, W2, B1, B2 = leaves
    R = X + B
    N = R * (R.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * W
    Y = torch.nn.functional.gelu(N @ W1.t() + B1) @ W2.t() + B2 + R
    Y.backward(dy.double().cpu())
    rel = lambda a, t: float((a.double().cpu() - t).norm() / t.norm())  # noqa: E731
    assert rel(y, Y.detach()) < 1e-6
    # 8 bits of a block of 32 are off by 2^-7 of its largest element at most
    for got, leaf in ((dx, X), (db, B), (dw, W), (dw1, W1), (dw2, W2), (db1, B1), (db2, B2)):
        assert rel(got, leaf.grad) < 2.0 ** -6
