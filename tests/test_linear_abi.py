"""CPU tests of the linear layer's and the checkpoints' C ABI: every refusal,
what a plan resolves, and that its plans run through their own calls only.
Plan creation and refused calls touch no GPU."""
import ctypes

import pytest

from onnx_broadcast_matmul_amd import binding as mm

P = 4096  # a pointer that no refused call follows


def status(call, *args, **kw):
    try:
        call(*args, **kw)
    except mm.MMError as e:
        return e.status
    return 0


def linear(rows=4, k=64, n=32, dtype=mm.BFLOAT16, **kw):
    return mm.LinearPlan(rows, k, n, dtype, **kw)


T = dict(training=True)
A = dict(training=True, activation=mm.ACT_SILU)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), mm.ERR_NEG_DIM), (dict(k=-1), mm.ERR_NEG_DIM), (dict(n=-5), mm.ERR_NEG_DIM),
    (dict(dtype=mm.DOUBLE), mm.ERR_DTYPE), (dict(dtype=mm.INT8), mm.ERR_DTYPE), (dict(dtype=99), mm.ERR_DTYPE),
    (dict(activation=-1), mm.ERR_BAD_OPTION), (dict(activation=6), mm.ERR_BAD_OPTION),
    (dict(w_pitch=31), mm.ERR_BAD_OPTION), (dict(w_pitch=63, trans_w=True), mm.ERR_BAD_OPTION),
    (dict(w_pitch=-1), mm.ERR_BAD_OPTION),
    (dict(z_type=mm.FLOAT), mm.ERR_BAD_OPTION), (dict(z_type=mm.FLOAT, **T), mm.ERR_BAD_OPTION),
    (dict(z_type=mm.FLOAT16, **A), mm.ERR_DTYPE), (dict(z_type=mm.INT32, **A), mm.ERR_DTYPE),
    (dict(x_type=mm.INT8), mm.ERR_BAD_OPTION), (dict(x_type=mm.FLOAT, **T), mm.ERR_DTYPE),
    (dict(x_activation=mm.ACT_RELU, **T), mm.ERR_BAD_OPTION), (dict(x_activation=7, x_type=mm.INT8, **T), mm.ERR_BAD_OPTION),
    (dict(rows=1 << 31), mm.ERR_TOO_LARGE), (dict(k=1 << 31), mm.ERR_TOO_LARGE), (dict(n=1 << 31), mm.ERR_TOO_LARGE),
    (dict(rows=1 << 30, n=1 << 11), mm.ERR_TOO_LARGE), (dict(k=1 << 30, n=1 << 11, rows=1), mm.ERR_TOO_LARGE),
    (dict(k=1 << 12, n=4, w_pitch=1 << 30), mm.ERR_TOO_LARGE),
    (dict(rows=1, k=1, n=1 << 30), mm.ERR_TOO_LARGE), (dict(rows=100, k=1, n=(1 << 31) - 100), mm.ERR_TOO_LARGE),
    (dict(rows=1 << 30, k=1 << 9, n=1, **T), mm.ERR_TOO_LARGE), (dict(rows=1, k=1 << 20, n=1 << 20, **T), mm.ERR_TOO_LARGE),
    (dict(force_algo=mm.ALGO_SKINNY_N), mm.ERR_BAD_OPTION), (dict(force_algo=mm.ALGO_DIRECT), mm.ERR_BAD_OPTION),
    (dict(split_k=-1), mm.ERR_BAD_OPTION), (dict(tile=1, split_k=2), mm.ERR_BAD_OPTION),
    (dict(tile=1, force_algo=mm.ALGO_SPLIT_K), mm.ERR_BAD_OPTION), (dict(rows=33, force_algo=mm.ALGO_SKINNY_M), mm.ERR_BAD_OPTION),
    (dict(force_algo=mm.ALGO_SKINNY_M, z_type=mm.INT8, **A), mm.ERR_BAD_OPTION),
    (dict(tile=4, z_type=mm.INT8, force_algo=mm.ALGO_GENERAL, **A), mm.ERR_BAD_OPTION),
    (dict(tile=4, z_type=mm.INT8, split_k=1, **A), mm.ERR_BAD_OPTION),
    (dict(force_algo=mm.ALGO_SKINNY_M, tile=2), mm.ERR_BAD_OPTION), (dict(force_algo=mm.ALGO_GENERAL, split_k=2), mm.ERR_BAD_OPTION),
    (dict(tile=6), mm.ERR_BAD_OPTION), (dict(tile=-1), mm.ERR_BAD_OPTION),
    (dict(dtype=mm.FLOAT, tile=1), mm.ERR_BAD_OPTION), (dict(dtype=mm.FLOAT, tile=5), mm.ERR_BAD_OPTION),
    (dict(dx_tile=2), mm.ERR_BAD_OPTION), (dict(dw_split_k=2), mm.ERR_BAD_OPTION), (dict(dx_tile=6, **T), mm.ERR_BAD_OPTION),
    (dict(dw_tile=4, **T), mm.ERR_BAD_OPTION), (dict(dx_tile=1, dx_split_k=2, **T), mm.ERR_BAD_OPTION),
    (dict(dw_split_k=-1, **T), mm.ERR_BAD_OPTION), (dict(dtype=mm.FLOAT, dx_tile=1, **T), mm.ERR_BAD_OPTION),
])
def test_linear_refusals(kw, want):
    assert status(linear, **kw) == want


def test_linear_descriptor_fields():
    L = mm.lib()
    h = ctypes.c_void_p()
    for field, value in (("trans_w", 2), ("has_bias", 2), ("has_residual", -1), ("training", 2), ("reserved", 1)):
        d = mm.LinearDesc(4, 64, 32, 0)
        setattr(d, field, value)
        assert L.mm_linear_plan_create(ctypes.byref(d), mm.FLOAT, None, ctypes.byref(h)) == mm.ERR_BAD_OPTION
    d = mm.LinearDesc(4, 64, 32, 0)
    assert L.mm_linear_plan_create(None, mm.FLOAT, None, ctypes.byref(h)) == mm.ERR_NULL_ARG
    assert L.mm_linear_plan_create(ctypes.byref(d), mm.FLOAT, None, None) == mm.ERR_NULL_ARG
    opt = mm.PlanOptions(0, 0, 0, 1)
    assert L.mm_linear_plan_create(ctypes.byref(d), mm.FLOAT, ctypes.byref(opt), ctypes.byref(h)) == mm.ERR_BAD_OPTION


def test_linear_plan_resolves():
    p = linear(200, 96, 264, trans_w=True, bias=True, residual=True, training=True, activation=mm.ACT_GELU,
               z_type=mm.INT8, x_type=mm.INT8, x_activation=mm.ACT_RELU, w_pitch=100)
    d, i = p.desc(), p.info()
    assert (d["rows"], d["in_features"], d["out_features"], d["w_pitch"]) == (200, 96, 264, 100)
    assert (d["z_type"], d["x_type"], d["x_activation"], d["activation"]) == (mm.INT8, mm.INT8, mm.ACT_RELU, mm.ACT_GELU)
    assert d["trans_w"] == d["has_bias"] == d["has_residual"] == d["training"] == 1
    assert d["dx_tile"] >= 1 and d["dw_tile"] >= 1 and d["dx_split_k"] >= 1
    assert p.output_shape == (200, 264) and i["flops"] == 2.0 * 200 * 96 * 264
    assert i["min_bytes"] == 2.0 * (200 * 96 + 96 * 264 + 264 + 2 * 200 * 264)
    # dZ, X^'s values and dZ's column sums
    assert i["workspace_bytes"] >= 2 * 200 * 264 + 2 * 200 * 96 + 4 * 4 * 264
    assert linear(training=True).desc()["z_type"] == 0 and linear(**A).desc()["z_type"] == mm.BFLOAT16
    assert linear(0, 8, 8).info()["algo_name"] == "empty"
    assert linear(1, 4096, 4096, trans_w=True).info()["algo_name"] == "skinny_m"
    assert linear(1, 4096, 4096, trans_w=True, z_type=mm.INT8, **A).info()["algo_name"] != "skinny_m"
    with pytest.raises(mm.MMError):
        mm.GluPlan(4, 8, 8, mm.FLOAT, training=True).options() and mm.LinearPlan.desc(mm.GluPlan(4, 8, 8, mm.FLOAT))


@pytest.mark.parametrize("rows", [1, 20, 32, 33, 300])
@pytest.mark.parametrize("dtype", [mm.FLOAT, mm.BFLOAT16])
def test_checkpoint_of_z_avoids_the_32_row_entry_unless_split(rows, dtype):
    for k, n, split in ((64, 64, 0), (4096, 512, 0), (512, 4096, 0), (100, 40, 0), (128, 72, 2), (64, 64, 2), (4096, 64, 4)):
        i = linear(rows, k, n, dtype, z_type=mm.INT8, split_k=split, **A).info()
        assert i["algo_name"] in ("general", "split_k") and not (i["tile"] == 4 and i["algo_name"] == "general")


def test_linear_execute_refusals():
    L = mm.lib()

    def run(p, X=P, W=P, bias=None, res=None, Y=P, Z=None, zs=None):
        return L.mm_linear_execute(p.handle, X, W, bias, res, Y, Z, zs, None)

    p = linear()
    assert run(p, Y=None) == mm.ERR_NULL_ARG and run(p, X=None) == mm.ERR_NULL_ARG and run(p, W=None) == mm.ERR_NULL_ARG
    assert run(p, bias=P) == mm.ERR_BAD_OPTION and run(p, res=P) == mm.ERR_BAD_OPTION
    assert run(p, Z=P) == mm.ERR_BAD_OPTION and run(p, zs=P) == mm.ERR_BAD_OPTION
    q = linear(bias=True, residual=True, z_type=mm.INT8, **A)
    assert run(q, res=P) == mm.ERR_NULL_ARG and run(q, bias=P) == mm.ERR_NULL_ARG
    assert run(q, bias=P, res=P, Z=P) == mm.ERR_NULL_ARG and run(q, bias=P, res=P, zs=P) == mm.ERR_BAD_OPTION
    assert run(linear(**A), Z=P, zs=P) == mm.ERR_BAD_OPTION
    assert L.mm_linear_execute(None, P, P, None, None, P, None, None, None) == mm.ERR_NULL_ARG
    g = mm.GluPlan(4, 64, 32, mm.BFLOAT16)
    assert run(g) == mm.ERR_BAD_OPTION
    for call in (L.mm_execute, L.mm_execute_noalloc):
        assert call(p.handle, P, P, P, None) == mm.ERR_BAD_OPTION
    assert L.mm_glu_execute(p.handle, P, P, P, P, None, None, None) == mm.ERR_BAD_OPTION
    assert L.mm_gemm_execute(p.handle, P, P, None, P, None) == mm.ERR_BAD_OPTION
    assert L.mm_int_execute(p.handle, P, P, None, None, P, None) == mm.ERR_BAD_OPTION
    assert L.mm_plan_set_constant_b(p.handle, P, 64 * 32, None) == mm.ERR_BAD_OPTION
    assert run(linear(0, 8, 8), X=None, W=None, Y=None) == 0  # nothing to do


def test_linear_backward_refusals():
    L = mm.lib()

    def run(p, X=P, xs=None, W=P, Z=None, zs=None, dY=P, dX=P, dW=P, db=None):
        return L.mm_linear_backward(p.handle, X, xs, W, Z, zs, dY, dX, dW, db, None)

    assert run(linear()) == mm.ERR_BAD_OPTION  # not for training
    p = linear(**T)
    assert run(p, db=P) == mm.ERR_BAD_OPTION and run(p, Z=P) == mm.ERR_BAD_OPTION and run(p, xs=P) == mm.ERR_BAD_OPTION
    assert run(p, zs=P) == mm.ERR_BAD_OPTION
    assert run(p, dY=None) == mm.ERR_NULL_ARG and run(p, X=None) == mm.ERR_NULL_ARG and run(p, W=None) == mm.ERR_NULL_ARG
    q = linear(z_type=mm.INT8, x_type=mm.INT8, bias=True, **A)
    assert run(q, xs=P) == mm.ERR_NULL_ARG and run(q, xs=P, Z=P) == mm.ERR_NULL_ARG
    assert run(q, Z=P, zs=P) == mm.ERR_NULL_ARG
    assert run(p, dX=None, dW=None) == 0  # nothing wanted
    assert L.mm_linear_backward(None, P, None, P, None, None, P, P, P, None, None) == mm.ERR_NULL_ARG
    assert run(mm.GluPlan(4, 64, 32, mm.BFLOAT16, training=True)) == mm.ERR_BAD_OPTION
    assert L.mm_glu_backward(p.handle, P, P, P, P, P, P, P, P, P, None) == mm.ERR_BAD_OPTION
    d = mm.LinearDesc()
    assert L.mm_linear_get_desc(None, ctypes.byref(d)) == mm.ERR_NULL_ARG
    assert L.mm_linear_get_desc(p.handle, None) == mm.ERR_NULL_ARG
    assert L.mm_linear_get_desc(mm.GluPlan(4, 8, 8, mm.FLOAT).handle, ctypes.byref(d)) == mm.ERR_BAD_OPTION


def test_checkpoint_refusals():
    L = mm.lib()
    for call in (lambda r, c, t, *p: L.mm_checkpoint_pack(p[0], t, r, c, p[1], p[2], None),
                 lambda r, c, t, *p: L.mm_checkpoint_unpack(p[0], p[1], r, c, t, p[2], None)):
        assert call(-1, 4, mm.FLOAT, P, P, P) == mm.ERR_NEG_DIM and call(4, -1, mm.FLOAT, P, P, P) == mm.ERR_NEG_DIM
        assert call(4, 4, mm.DOUBLE, P, P, P) == mm.ERR_DTYPE and call(4, 4, mm.INT8, P, P, P) == mm.ERR_DTYPE
        assert call(1 << 31, 4, mm.FLOAT, P, P, P) == mm.ERR_TOO_LARGE
        assert call(1 << 21, 1 << 20, mm.FLOAT, P, P, P) == mm.ERR_TOO_LARGE
        for i in range(3):
            assert call(4, 4, mm.FLOAT, *(None if j == i else P for j in range(3))) == mm.ERR_NULL_ARG
        assert call(0, 4, mm.FLOAT, None, None, None) == 0 and call(4, 0, mm.FLOAT, None, None, None) == 0
    assert L.mm_checkpoint_blocks(-1) == -1
    for n in (0, 1, 31, 32, 33, 1000, 1 << 40):
        assert L.mm_checkpoint_blocks(n) == mm.checkpoint_blocks(n) == (n + 31) // 32


def test_binding_refuses_host_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mm.checkpoint_pack(x)
    with pytest.raises(ValueError):
        mm.checkpoint_unpack(torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8), torch.bfloat16)
    p = linear(bias=True)
    y, w, b = torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(64, 32, dtype=torch.bfloat16), torch.zeros(32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bias"):
        p.execute(x, w, y)
    with pytest.raises(ValueError, match="residual"):
        p.execute(x, w, y, bias=b, residual=y)
    with pytest.raises(ValueError, match="device"):
        p.execute(x, w, y, bias=b)
    with pytest.raises(ValueError, match="device"):
        linear(**T).backward(x, w, y)


@pytest.mark.parametrize("nk", [True, False], ids=["nk", "kn"])
@pytest.mark.parametrize("dtype", [mm.FLOAT16, mm.BFLOAT16])
def test_linear_backward_second_launches(dtype, nk):
    """The sizes whose backward pass is compared as whole rounds and a rest run so."""
    for j, (m, k, n) in enumerate(((4104, 5000, 512), (512, 5000, 4104), (512, 4104, 5000))):
        p = mm.LinearPlan(m, k, n, dtype, activation=mm.ACT_SILU, trans_w=nk, bias=True, training=True, z_type=mm.INT8,
                          x_type=mm.INT8 if j == 2 else 0)
        t = p.tails()
        width = k if j == 0 or nk else n
        split, whole = ("dx", "dw") if j == 0 else ("dw", "dx")
        assert 0 < t[split + "_col"] < width and t[split + "_col"] % 128 == 0 and 1 <= t[split + "_tile"] <= 5, t
        assert t[whole + "_col"] == t[whole + "_tile"] == 0
    p = mm.LinearPlan(4104, 5000, 512, dtype, trans_w=nk, training=True, dx_tile=1, dw_tile=1)
    assert not any(p.tails().values())


def test_linear_tails_refusals():
    L = mm.lib()
    t = mm.LinearTails()
    p = mm.LinearPlan(4, 64, 32, mm.FLOAT, training=True)
    assert L.mm_linear_get_tails(None, ctypes.byref(t)) == mm.ERR_NULL_ARG
    assert L.mm_linear_get_tails(p._handle, None) == mm.ERR_NULL_ARG
    assert L.mm_linear_get_tails(p._handle, ctypes.byref(t)) == 0
    for other in (mm.LinearPlan(4, 64, 32, mm.FLOAT), mm.GluPlan(4, 64, 32, mm.FLOAT, training=True)):
        assert L.mm_linear_get_tails(other._handle, ctypes.byref(t)) == mm.ERR_BAD_OPTION
