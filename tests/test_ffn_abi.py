"""CPU tests of the feed-forward operators' C ABI (the gated block, the scaled
INT8 product, row quantization): every refusal, what a plan resolves, and that
each kind of plan runs through its own calls only.  Plan creation and refused
calls touch no GPU."""
import ctypes

import pytest

from onnx_broadcast_matmul_amd import binding as mm


def status(call, *args, **kw):
    try:
        call(*args, **kw)
    except mm.MMError as e:
        return e.status
    return 0


def glu(rows=4, k=64, n=32, dtype=mm.BFLOAT16, **kw):
    return mm.GluPlan(rows, k, n, dtype, **kw)


def scaled(sa=(4, 64), sb=(64, 32), out=mm.BFLOAT16, **kw):
    return mm.ScaledIntPlan(sa, sb, out, **kw)


# ---- gated block


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), mm.ERR_NEG_DIM), (dict(k=-1), mm.ERR_NEG_DIM), (dict(n=-5), mm.ERR_NEG_DIM),
    (dict(dtype=mm.DOUBLE), mm.ERR_DTYPE), (dict(dtype=mm.INT8), mm.ERR_DTYPE), (dict(dtype=99), mm.ERR_DTYPE),
    (dict(activation=0), mm.ERR_BAD_OPTION), (dict(activation=6), mm.ERR_BAD_OPTION),
    (dict(w_pitch=31), mm.ERR_BAD_OPTION), (dict(w_pitch=63, trans_w=True), mm.ERR_BAD_OPTION),
    (dict(w_pitch=-1), mm.ERR_BAD_OPTION),
    (dict(rows=1 << 31), mm.ERR_TOO_LARGE), (dict(k=1 << 31), mm.ERR_TOO_LARGE), (dict(n=1 << 31), mm.ERR_TOO_LARGE),
    (dict(rows=1 << 30, n=1 << 11), mm.ERR_TOO_LARGE), (dict(k=1 << 30, n=1 << 11, rows=1), mm.ERR_TOO_LARGE),
    (dict(k=1 << 12, n=4, w_pitch=1 << 30), mm.ERR_TOO_LARGE),
    # grids of more than 2^32 threads: few rows, tiles, the two gradients
    (dict(rows=1, k=1, n=1 << 30), mm.ERR_TOO_LARGE), (dict(rows=100, k=1, n=1 << 30), mm.ERR_TOO_LARGE),
    (dict(rows=1 << 30, k=1 << 9, n=1, training=True), mm.ERR_TOO_LARGE),
    (dict(rows=1, k=1 << 20, n=1 << 20, training=True), mm.ERR_TOO_LARGE),
    (dict(force_algo=mm.ALGO_SKINNY_N), mm.ERR_BAD_OPTION), (dict(force_algo=mm.ALGO_DIRECT), mm.ERR_BAD_OPTION),
    (dict(split_k=-1), mm.ERR_BAD_OPTION), (dict(tile=1, split_k=2), mm.ERR_BAD_OPTION),
    (dict(tile=1, force_algo=mm.ALGO_SPLIT_K), mm.ERR_BAD_OPTION), (dict(rows=33, force_algo=mm.ALGO_SKINNY_M), mm.ERR_BAD_OPTION),
    (dict(tile=6), mm.ERR_BAD_OPTION), (dict(tile=-1), mm.ERR_BAD_OPTION),
    (dict(dtype=mm.FLOAT, tile=1), mm.ERR_BAD_OPTION), (dict(dtype=mm.FLOAT, tile=5), mm.ERR_BAD_OPTION),
])
def test_glu_refusals(kw, want):
    assert status(glu, **kw) == want


def test_glu_descriptor_fields():
    L = mm.lib()
    h = ctypes.c_void_p()
    for field, value in (("trans_w", 2), ("training", 2), ("reserved", 1)):
        d = mm.GluDesc(4, 64, 32, 0, 0, mm.ACT_SILU, 0, 0)
        setattr(d, field, value)
        assert L.mm_glu_plan_create(ctypes.byref(d), mm.FLOAT, None, ctypes.byref(h)) == mm.ERR_BAD_OPTION
        assert not h.value
    assert L.mm_glu_plan_create(None, mm.FLOAT, None, ctypes.byref(h)) == mm.ERR_NULL_ARG
    d = mm.GluDesc(4, 64, 32, 0, 0, mm.ACT_SILU, 0, 0)
    assert L.mm_glu_plan_create(ctypes.byref(d), mm.FLOAT, None, None) == mm.ERR_NULL_ARG
    opt = mm.PlanOptions(0, 0, 0, 2)
    assert L.mm_glu_plan_create(ctypes.byref(d), mm.FLOAT, ctypes.byref(opt), ctypes.byref(h)) == mm.ERR_BAD_OPTION


def test_glu_info():
    p = glu(1000, 1024, 4096, trans_w=True)
    i = p.info()
    assert p.output_shape == (1000, 4096) and p.output_numel == 1000 * 4096
    assert i["flops"] == 4.0 * 1000 * 1024 * 4096
    assert i["min_bytes"] == 2.0 * (1000 * 1024 + 2 * 1024 * 4096 + 1000 * 4096)
    assert p.workspace_bytes == 0 and i["algo_name"] == "general"
    assert glu(1, 4096, 512, trans_w=True).info()["algo_name"] == "skinny_m"
    assert glu(0, 64, 32).info()["algo_name"] == "empty"
    s = glu(100, 4096, 64, split_k=4)
    assert s.info()["algo_name"] == "split_k" and s.info()["split_k"] == 4
    assert s.workspace_bytes == 4 * 2 * 100 * 64 * 4
    t = glu(100, 64, 33, training=True)
    assert t.workspace_bytes >= 2 * 100 * 40 * 2  # dG and dU with rows of 40 elements


def test_glu_execute_refusals():
    p = glu()
    for args in ((0, 8, 8, 8, 0, 0), (8, 0, 8, 8, 0, 0), (8, 8, 0, 8, 0, 0), (8, 8, 8, 0, 0, 0), (8, 8, 8, 8, 8, 0),
                 (8, 8, 8, 8, 0, 8)):
        assert status(p.execute_ptr, *args) == mm.ERR_NULL_ARG, args
    L = mm.lib()
    assert L.mm_glu_execute(None, 8, 8, 8, 8, None, None, None) == mm.ERR_NULL_ARG
    back = L.mm_glu_backward
    one = [8] * 9
    assert back(None, *one, None) == mm.ERR_NULL_ARG
    assert back(p.handle, *one, None) == mm.ERR_BAD_OPTION  # not a training plan
    t = glu(training=True)
    assert back(t.handle, *one[:7], 8, None, None) == mm.ERR_NULL_ARG  # dWg without dWu
    for miss in (3, 4, 5):  # G, U, dH
        args = [8] * 9
        args[miss] = None
        assert back(t.handle, *args, None) == mm.ERR_NULL_ARG, miss
    assert back(t.handle, 8, None, 8, 8, 8, 8, 8, None, None, None) == mm.ERR_NULL_ARG  # dX needs the weights
    assert back(t.handle, None, 8, 8, 8, 8, 8, None, 8, 8, None) == mm.ERR_NULL_ARG  # dW needs X
    assert back(t.handle, *one[:6], None, None, None, None) == 0  # nothing asked for
    # empty outputs read nothing
    assert status(glu(0, 64, 32).execute_ptr, 0, 0, 0, 0) == 0
    assert status(glu(4, 64, 0).execute_ptr, 0, 0, 0, 0) == 0


def test_glu_backward_workspace_holds_the_largest_split():
    """A short product with a long reduction splits it: the partial sums
    follow dG and dU in the workspace."""
    t = mm.GluPlan(5000, 64, 64, mm.BFLOAT16, trans_w=True, training=True)
    assert t.workspace_bytes > 2 * 5000 * 64 * 2 + 4 * 2 * 64 * 64


# ---- scaled INT8 product


@pytest.mark.parametrize("kw,want", [
    (dict(sa=(), sb=(4, 4)), mm.ERR_RANK), (dict(sa=(4, -1)), mm.ERR_NEG_DIM), (dict(sa=(4, 63)), mm.ERR_K_MISMATCH),
    (dict(sa=(2, 4, 64), sb=(3, 64, 32)), mm.ERR_BROADCAST),
    (dict(out=mm.DOUBLE), mm.ERR_DTYPE), (dict(out=mm.INT32), mm.ERR_DTYPE),
    (dict(a_type=mm.UINT8), mm.ERR_DTYPE), (dict(a_type=mm.DOUBLE), mm.ERR_DTYPE), (dict(a_type=0), mm.ERR_DTYPE),
    (dict(sa=(64,), sb=(64,), trans_b=True), mm.ERR_BAD_OPTION),
    (dict(sa=(1, 131072), sb=(131072, 1)), mm.ERR_TOO_LARGE), (dict(sa=(1 << 16, 1 << 15, 64)), mm.ERR_TOO_LARGE),
    (dict(sa=(1 << 30, 64), sb=(64, 1 << 11)), mm.ERR_TOO_LARGE),
    # grids of more than 2^32 threads: few rows, tiles, products of a batch
    (dict(sa=(1, 1), sb=(1, 1 << 30)), mm.ERR_TOO_LARGE), (dict(sa=(1000, 1), sb=(1, 1 << 30)), mm.ERR_TOO_LARGE),
    (dict(sa=(1 << 25, 4, 64), sb=(1 << 25, 64, 32)), mm.ERR_TOO_LARGE),
    (dict(force_algo=mm.ALGO_DIRECT), mm.ERR_BAD_OPTION), (dict(force_algo=mm.ALGO_SKINNY_N), mm.ERR_BAD_OPTION),
    (dict(sa=(33, 64), force_algo=mm.ALGO_SKINNY_M), mm.ERR_BAD_OPTION),
    (dict(sa=(2, 4, 64), sb=(2, 64, 32), force_algo=mm.ALGO_SKINNY_M), mm.ERR_BAD_OPTION),
    (dict(tile=6), mm.ERR_BAD_OPTION), (dict(split_k=-1), mm.ERR_BAD_OPTION),
    (dict(tile=1, split_k=2), mm.ERR_BAD_OPTION), (dict(tile=1, force_algo=mm.ALGO_SPLIT_K), mm.ERR_BAD_OPTION),
])
def test_scaled_refusals(kw, want):
    assert status(scaled, **kw) == want


def test_scaled_descriptor_fields():
    L = mm.lib()
    h = ctypes.c_void_p()
    sa, sb = (ctypes.c_int64 * 2)(4, 64), (ctypes.c_int64 * 2)(64, 32)
    for field, value in (("trans_b", 2), ("has_bias", -1), ("reserved", 1)):
        d = mm.ScaledIntDesc(mm.INT8, mm.FLOAT, 0, 0, 0)
        setattr(d, field, value)
        assert L.mm_scaled_int_plan_create(sa, 2, sb, 2, ctypes.byref(d), None, ctypes.byref(h)) == mm.ERR_BAD_OPTION
    assert L.mm_scaled_int_plan_create(sa, 2, sb, 2, None, None, ctypes.byref(h)) == mm.ERR_NULL_ARG
    d = mm.ScaledIntDesc(mm.INT8, mm.FLOAT, 0, 0, 0)
    assert L.mm_scaled_int_plan_create(None, 2, sb, 2, ctypes.byref(d), None, ctypes.byref(h)) == mm.ERR_NULL_ARG
    assert L.mm_scaled_int_plan_create(sa, 11, sb, 2, ctypes.byref(d), None, ctypes.byref(h)) == mm.ERR_RANK


def test_scaled_shapes_and_workspaces():
    p = scaled((2, 5, 64), (3, 1, 64, 32), bias=True)
    assert p.output_shape == (3, 2, 5, 32)
    assert p.a_scale_shape == (2, 5) and p.b_scale_shape == (3, 1, 32)
    t = scaled((2, 5, 64), (3, 1, 32, 64), trans_b=True)
    assert t.output_shape == (3, 2, 5, 32) and t.b_scale_shape == (3, 1, 32)
    v = scaled((64,), (64,))
    assert v.output_shape == () and v.a_scale_shape == () and v.b_scale_shape == ()
    assert scaled((0, 64), (64, 32)).info()["algo_name"] == "empty"
    # an A to be quantized: 200 rows of 112 bytes and their scales, or nothing
    # where the few-row kernel does it
    q = scaled((200, 100), (100, 500), a_type=mm.BFLOAT16)
    assert q.workspace_bytes >= 200 * 112 + 4 * 200
    assert scaled((1, 4096), (512, 4096), a_type=mm.BFLOAT16, trans_b=True).workspace_bytes == 0
    assert scaled((1, 4096), (512, 4096), a_type=mm.FLOAT, trans_b=True).workspace_bytes > 0  # other output type
    s = scaled((64, 11008), (11008, 256), split_k=4)
    assert s.info()["algo_name"] == "split_k" and s.info()["split_k"] == 4
    assert s.workspace_bytes == 4 * 64 * 256 * 4


def test_scaled_execute_refusals():
    L = mm.lib()
    ex = L.mm_scaled_int_execute
    p, b, q = scaled(), scaled(bias=True), scaled((64, 64), a_type=mm.FLOAT)
    assert ex(None, 8, 8, 8, 8, None, 8, None) == mm.ERR_NULL_ARG
    for miss in (0, 1, 2, 3, 5):  # A, B, a_scale, b_scale, Y
        args = [8, 8, 8, 8, None, 8]
        args[miss] = None
        assert ex(p.handle, *args, None) == mm.ERR_NULL_ARG, miss
    assert ex(p.handle, 8, 8, 8, 8, 8, 8, None) == mm.ERR_BAD_OPTION  # a bias the plan lacks
    assert ex(b.handle, 8, 8, 8, 8, None, 8, None) == mm.ERR_NULL_ARG
    assert ex(q.handle, 8, 8, 8, 8, None, 8, None) == mm.ERR_BAD_OPTION  # a_scale for an A it quantizes
    assert ex(scaled((0, 64)).handle, None, None, None, None, None, None, None) == 0


def test_quantize_rows_refusals():
    f = mm.lib().mm_quantize_rows
    assert f(8, mm.FLOAT, -1, 4, 8, 8, None) == mm.ERR_NEG_DIM
    assert f(8, mm.FLOAT, 4, -1, 8, 8, None) == mm.ERR_NEG_DIM
    assert f(8, mm.DOUBLE, 4, 4, 8, 8, None) == mm.ERR_DTYPE
    assert f(8, mm.INT8, 4, 4, 8, 8, None) == mm.ERR_DTYPE
    assert f(8, mm.FLOAT, 1 << 31, 4, 8, 8, None) == mm.ERR_TOO_LARGE
    assert f(8, mm.FLOAT, 1 << 30, 1 << 12, 8, 8, None) == mm.ERR_TOO_LARGE
    for args in ((None, 8, 8), (8, None, 8), (8, 8, None)):
        assert f(args[0], mm.FLOAT, 4, 4, args[1], args[2], None) == mm.ERR_NULL_ARG
    assert f(None, mm.FLOAT, 0, 4, None, None, None) == 0


def test_plans_run_through_their_own_calls_only():
    L = mm.lib()
    kinds = {
        "matmul": mm.Plan((4, 64), (64, 32), mm.FLOAT), "gemm": mm.GemmPlan((4, 64), (64, 32), mm.FLOAT),
        "int": mm.IntPlan((4, 64), (64, 32), mm.INT8, mm.INT8), "scaled": scaled(out=mm.FLOAT),
        "glu": glu(dtype=mm.FLOAT, training=True),
    }
    calls = {
        "matmul": lambda h: L.mm_execute(h, 8, 8, 8, None),
        "gemm": lambda h: L.mm_gemm_execute(h, 8, 8, 8, 8, None),
        "int": lambda h: L.mm_int_execute(h, 8, 8, None, None, 8, None),
        "scaled": lambda h: L.mm_scaled_int_execute(h, 8, 8, 8, 8, None, 8, None),
        "glu": lambda h: L.mm_glu_execute(h, 8, 8, 8, 8, None, None, None),
    }
    for own, plan in kinds.items():
        for name, call in calls.items():
            if name != own:
                assert call(plan.handle) == mm.ERR_BAD_OPTION, (own, name)
    for own in ("scaled", "glu"):
        h = kinds[own].handle
        assert L.mm_execute_noalloc(h, 8, 8, 8, None) == mm.ERR_BAD_OPTION
        assert L.mm_plan_set_constant_b(h, 8, 64 * 32, None) == mm.ERR_BAD_OPTION
        assert L.mm_execute_constant_b(h, 8, 8, None) in (mm.ERR_BAD_OPTION, mm.ERR_NO_CONSTANT_B)
    for own in ("matmul", "gemm", "int", "scaled"):
        assert L.mm_glu_backward(kinds[own].handle, *([8] * 9), None) == mm.ERR_BAD_OPTION


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x, w, h = torch.zeros(4, 64), torch.zeros(64, 32), torch.zeros(4, 32)
    p = glu(dtype=mm.FLOAT)
    with pytest.raises(ValueError):
        p.execute(x, w, w, h)
    with pytest.raises(ValueError):
        p.execute(x, w, w, h, G=h)
    s = scaled(out=mm.FLOAT)
    a, b = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(64, 32, dtype=torch.int8)
    with pytest.raises(ValueError):
        s.execute(a, b, h, a_scale=torch.zeros(4), b_scale=torch.zeros(32))
    with pytest.raises(ValueError):
        s.execute(a, b, h, b_scale=torch.zeros(32))
    with pytest.raises(ValueError):
        mm.quantize_rows(x)


# ---- forced algorithms


@pytest.mark.parametrize("rows,k,n", [(300, 64, 64), (4096, 64, 4096), (2, 35, 9)])
def test_forced_split_is_kept(rows, k, n):
    """SPLIT_K runs as SPLIT_K, with one partition where the plan prefers it."""
    for dtype in (mm.FLOAT, mm.BFLOAT16):
        for kw in ({}, dict(split_k=1), dict(split_k=3), dict(tile=3), dict(tile=4, split_k=2)):
            p = glu(rows, k, n, dtype, force_algo=mm.ALGO_SPLIT_K, **kw)
            i = p.info()
            assert i["algo_name"] == "split_k" and i["split_k"] >= 1, kw
            assert p.workspace_bytes == (i["split_k"] * 2 * rows * n * 4 + 255) // 256 * 256
            assert i["k_chunk"] > 0
    p = scaled((rows, k), (k, n), force_algo=mm.ALGO_SPLIT_K)
    assert p.info()["algo_name"] == "split_k"


@pytest.mark.parametrize("kw", [
    dict(force_algo=mm.ALGO_GENERAL, split_k=2), dict(force_algo=mm.ALGO_SKINNY_M, split_k=2),
    dict(force_algo=mm.ALGO_SKINNY_M, tile=2),
])
def test_options_that_the_forced_algorithm_lacks_are_refused(kw):
    assert status(glu, **kw) == mm.ERR_BAD_OPTION
    assert status(scaled, **kw) == mm.ERR_BAD_OPTION
    # as everywhere, nothing is forced on an empty output
    assert glu(0, 64, 32, **kw).info()["algo_name"] == "empty"
    assert scaled((0, 64), **kw).info()["algo_name"] == "empty"


def test_options_of_one_partition_and_forced_tiles_still_run():
    assert glu(force_algo=mm.ALGO_GENERAL, split_k=1, tile=3).info()["algo_name"] == "general"
    assert scaled(force_algo=mm.ALGO_GENERAL, split_k=1, tile=3).info()["algo_name"] == "general"
    assert glu(force_algo=mm.ALGO_SKINNY_M, split_k=1).info()["algo_name"] == "skinny_m"
    assert scaled(force_algo=mm.ALGO_SKINNY_M, split_k=1).info()["algo_name"] == "skinny_m"


def test_split_of_more_products_than_its_reduction_takes_is_refused():
    """Partial sums are added by a grid of at most 65535 products."""
    many = dict(sa=(65536, 1, 64), sb=(65536, 64, 2))
    assert status(scaled, **many) == 0
    assert status(scaled, **many, force_algo=mm.ALGO_SPLIT_K) == mm.ERR_BAD_OPTION
    assert status(scaled, **many, split_k=2) == mm.ERR_BAD_OPTION


# ---- second launches (the joining of partial sums, the element-wise pass)


@pytest.mark.parametrize("call,kw", [
    (scaled, dict(sa=(1 << 17, 4096), sb=(4096, 1 << 17), split_k=2)),
    (scaled, dict(sa=(1 << 17, 4096), sb=(4096, (1 << 17) - 3), split_k=2)),
    (glu, dict(rows=1 << 17, k=4096, n=1 << 17, split_k=2)),
    # 2^32 - 1 pieces of dG's rows, whole workgroups of them 2^32 threads
    (glu, dict(rows=65537, k=1, n=65535 * 8, training=True)),
])
def test_second_launches_of_2_32_threads_are_refused(call, kw):
    assert status(call, **kw) == mm.ERR_TOO_LARGE


# ---- the backward products' tiling


def test_backward_tiling_is_shown_and_kept():
    d = dict(rows=530, k=328, n=400, training=True)
    for dtype, entries in ((mm.FLOAT, (2, 3, 4)), (mm.BFLOAT16, (1, 2, 3, 5))):
        for t in entries:
            for s in (1, 3) if t > 1 else (1,):
                p = glu(dtype=dtype, **d, dx_tile=t, dw_tile=t, dx_split_k=s, dw_split_k=s)
                i = p.options()
                assert i["dx_tile"] == i["dw_tile"] == t
                # three partitions of dW's reduction over 530 rows may be two of whole stages
                assert i["dx_split_k"] == s and i["dw_split_k"] in (min(s, 2), s)
                parts = max(i["dx_split_k"] * 530 * 328 * (s > 1), i["dw_split_k"] * 2 * 328 * 400 * (s > 1))
                assert p.workspace_bytes >= 2 * 530 * 400 * 2 + 4 * parts
    assert glu(**d, dx_tile=4).options()["dx_tile"] == 4
    i = glu(**d).options()  # the plan's choice
    assert 1 <= i["dx_tile"] <= 5 and 1 <= i["dw_tile"] <= 5 and i["dx_split_k"] >= 1 and i["dw_split_k"] >= 1


def test_large_training_steps_run_on_the_large_entries():
    """The entries that the forced-tile tests compare are those that large
    steps run on."""
    i = glu(8192, 4096, 11008, trans_w=True, training=True).options()
    assert (i["dx_tile"], i["dw_tile"]) == (1, 1)
    i = glu(4096, 2048, 5504, trans_w=True, training=True).options()
    assert (i["dx_tile"], i["dw_tile"]) == (5, 5)


@pytest.mark.parametrize("kw", [
    dict(dx_tile=1), dict(dw_split_k=2),  # no training
    dict(training=True, dx_tile=6), dict(training=True, dw_tile=-1), dict(training=True, dx_split_k=-1),
    dict(training=True, dw_split_k=-2), dict(training=True, dw_tile=4), dict(training=True, dx_tile=1, dx_split_k=2),
    dict(training=True, dtype=mm.FLOAT, dx_tile=1), dict(training=True, dtype=mm.FLOAT, dw_tile=5),
])
def test_backward_tiling_refusals(kw):
    assert status(glu, **kw) == mm.ERR_BAD_OPTION


def test_backward_tiling_calls():
    L = mm.lib()
    t = mm.GluOptions()
    assert L.mm_glu_get_options(None, ctypes.byref(t)) == mm.ERR_NULL_ARG
    assert L.mm_glu_get_options(glu(training=True).handle, None) == mm.ERR_NULL_ARG
    assert L.mm_glu_get_options(glu().handle, ctypes.byref(t)) == mm.ERR_BAD_OPTION
    assert L.mm_glu_get_options(scaled().handle, ctypes.byref(t)) == mm.ERR_BAD_OPTION
    d = mm.GluDesc(4, 64, 32, 0, 0, mm.ACT_SILU, 1, 0)
    h = ctypes.c_void_p()
    assert L.mm_glu_plan_create_ex(ctypes.byref(d), mm.FLOAT, None, None, ctypes.byref(h)) == 0
    assert L.mm_glu_get_options(h, ctypes.byref(t)) == 0 and t.dx_split_k >= 1
    L.mm_plan_destroy(h)
    assert L.mm_glu_plan_create_ex(None, mm.FLOAT, None, None, ctypes.byref(h)) == mm.ERR_NULL_ARG and not h.value
    # empty steps take the options too
    for size in ((0, 64, 32), (4, 0, 32), (4, 64, 0)):
        p = glu(*size, training=True, dx_tile=3, dx_split_k=2, dw_tile=2, dw_split_k=5)
        i = p.options()
        assert i["dx_tile"] == 3 and i["dw_tile"] == 2 and i["dx_split_k"] >= 1 and i["dw_split_k"] >= 1


@pytest.mark.parametrize("dtype", [mm.FLOAT, mm.FLOAT16, mm.BFLOAT16])
def test_kept_type(dtype):
    for training in (False, True):
        for kept in (0, dtype, mm.FLOAT):
            p = glu(dtype=dtype, training=training, kept_type=kept)
            assert not training or p.options()["kept_type"] == (kept or dtype)
        for kept in {mm.FLOAT16, mm.BFLOAT16, mm.DOUBLE, mm.INT8, -1, 99} - {dtype}:
            assert status(glu, dtype=dtype, training=training, kept_type=kept) == mm.ERR_DTYPE
