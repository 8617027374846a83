"""CPU tests of the norms' C ABI: every refusal, what a plan resolves, and that
its plans run through their own calls only."""
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


def norm(rows=4, cols=64, dtype=mm.BFLOAT16, **kw):
    return mm.NormPlan(rows, cols, dtype, **kw)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), mm.ERR_NEG_DIM), (dict(cols=-1), mm.ERR_NEG_DIM), (dict(gate_rows=-1), mm.ERR_NEG_DIM),
    (dict(dtype=mm.DOUBLE), mm.ERR_DTYPE), (dict(dtype=mm.INT8), mm.ERR_DTYPE), (dict(dtype=99), mm.ERR_DTYPE),
    (dict(pre=mm.NORM_NONE, pre_weight=False), mm.ERR_BAD_OPTION), (dict(pre=3), mm.ERR_BAD_OPTION), (dict(post=-1), mm.ERR_BAD_OPTION),
    (dict(pre=mm.NORM_NONE, post=mm.NORM_RMS), mm.ERR_BAD_OPTION), (dict(post_weight=True), mm.ERR_BAD_OPTION),
    (dict(post_bias=True), mm.ERR_BAD_OPTION), (dict(block=False, post=mm.NORM_RMS), mm.ERR_BAD_OPTION),
    (dict(block=False, gate_rows=2), mm.ERR_BAD_OPTION),
    (dict(pre_eps=-1.0), mm.ERR_BAD_OPTION), (dict(post_eps=float("nan")), mm.ERR_BAD_OPTION),
    (dict(pre_eps=float("inf")), mm.ERR_BAD_OPTION), (dict(residual_scale=float("nan")), mm.ERR_BAD_OPTION),
    (dict(residual_scale=float("inf")), mm.ERR_BAD_OPTION),
    (dict(kept_type=mm.INT8), mm.ERR_BAD_OPTION), (dict(kept_type=mm.FLOAT), mm.ERR_BAD_OPTION),
    (dict(kept_type=mm.FLOAT16, training=True), mm.ERR_DTYPE), (dict(kept_type=mm.INT32, training=True), mm.ERR_DTYPE),
    (dict(cols=mm.NORM_MAX_COLS + 1), mm.ERR_TOO_LARGE), (dict(rows=1 << 31), mm.ERR_TOO_LARGE),
    (dict(rows=1 << 27, cols=1 << 14), mm.ERR_TOO_LARGE), (dict(rows=1 << 26, cols=1 << 14), 0),
    (dict(rows=1 << 30, cols=1 << 10), 0), (dict(rows=1 << 30, cols=1 << 10, training=True), 0),
])
def test_norm_refusals(kw, want):
    assert status(norm, **kw) == want


def test_norm_descriptor_fields():
    L = mm.lib()
    h = ctypes.c_void_p()

    def desc(**kw):
        d = mm.NormDesc(4, 64, 0, mm.NORM_NONE, mm.NORM_RMS, 0, 0, 1, 1)
        for k, v in kw.items():
            setattr(d, k, v)
        return ctypes.byref(d)

    assert L.mm_norm_plan_create(desc(), mm.FLOAT, ctypes.byref(h)) == 0
    L.mm_plan_destroy(h)
    for kw in (dict(has_block=2), dict(post_weight=-1), dict(pre_bias=3), dict(training=2), dict(reserved=1)):
        assert L.mm_norm_plan_create(desc(**kw), mm.FLOAT, ctypes.byref(h)) == mm.ERR_BAD_OPTION
    assert L.mm_norm_plan_create(None, mm.FLOAT, ctypes.byref(h)) == mm.ERR_NULL_ARG
    assert L.mm_norm_plan_create(desc(), mm.FLOAT, None) == mm.ERR_NULL_ARG


def test_norm_plan_resolves():
    p = norm(200, 1000, post=mm.NORM_LAYER, gate_rows=50, training=True)
    i = p.info()
    assert p.output_shape == (200, 1000) and i["min_bytes"] == 2.0 * 4 * 200 * 1000 and i["flops"] == 0
    assert p.workspace_bytes > 0 and norm(200, 1000).workspace_bytes == 0
    assert norm(200, 1000, block=False).info()["min_bytes"] == 2.0 * 2 * 200 * 1000
    assert norm(0, 64).info()["algo_name"] == "empty" and norm(4, 0).info()["algo_name"] == "empty"


def run(p, call, fields, given):
    a = fields(**{k: P for k in given.split()})
    return call(p.handle if hasattr(p, "handle") else p, ctypes.byref(a), None)


def test_norm_execute_refusals():
    L = mm.lib()
    f = lambda p, given: run(p, L.mm_norm_execute, mm.NormForwardArgs, given)  # noqa: E731
    p = norm(post=mm.NORM_RMS, post_weight=True, post_bias=True, pre_bias=True, gate_rows=2)
    full = "residual block gate post_weight post_bias pre_weight pre_bias out".split()
    for name in full:
        assert f(p, " ".join(k for k in full if k != name)) == mm.ERR_NULL_ARG, name
    for more in ("stats", "sum_f32", "sum_q sum_scale", "block_q", "out_scale"):
        assert f(p, " ".join(full) + " " + more) == mm.ERR_BAD_OPTION, more  # not for training
    q = norm(pre_weight=False)
    for more in ("gate", "post_weight", "post_bias", "pre_weight", "pre_bias"):
        assert f(q, "residual block out " + more) == mm.ERR_BAD_OPTION, more
    assert f(norm(block=False, pre_weight=False), "residual out block") == mm.ERR_BAD_OPTION
    assert f(norm(pre=mm.NORM_NONE, post=mm.NORM_RMS, pre_weight=False), "residual block out") == mm.ERR_BAD_OPTION
    t = norm(training=True, pre_weight=False)
    for more in ("sum_q", "sum_scale", "block_q", "block_scale", "out_q", "out_scale"):
        assert f(t, "residual block out " + more) == mm.ERR_NULL_ARG, more
    assert f(t, "residual block out sum_f32") == mm.ERR_BAD_OPTION
    assert f(norm(training=True, block=False, pre_weight=False), "residual out block_q block_scale") == mm.ERR_BAD_OPTION
    assert L.mm_norm_execute(None, ctypes.byref(mm.NormForwardArgs()), None) == mm.ERR_NULL_ARG
    assert L.mm_norm_execute(p.handle, None, None) == mm.ERR_NULL_ARG
    assert f(mm.GluPlan(4, 64, 32, mm.FLOAT), "residual") == mm.ERR_BAD_OPTION
    assert f(norm(0, 64), "") == 0
    for call in (L.mm_execute, L.mm_execute_noalloc):
        assert call(p.handle, P, P, P, None) == mm.ERR_BAD_OPTION
    assert L.mm_linear_execute(p.handle, P, P, None, None, P, None, None, None) == mm.ERR_BAD_OPTION
    assert L.mm_plan_set_constant_b(p.handle, P, 0, None) == mm.ERR_BAD_OPTION


def test_norm_backward_refusals():
    L = mm.lib()
    f = lambda p, given: run(p, L.mm_norm_backward, mm.NormBackwardArgs, given)  # noqa: E731
    assert f(norm(), "stats sum dout dresidual pre_weight") == mm.ERR_BAD_OPTION  # not for training
    p = norm(post=mm.NORM_RMS, post_weight=True, post_bias=True, pre_bias=True, gate_rows=2, training=True)
    full = "stats sum block gate post_weight post_bias pre_weight dout dresidual dblock dgate".split()
    for name in full[:8]:
        assert f(p, " ".join(k for k in full if k != name)) == mm.ERR_NULL_ARG, name
    assert f(p, " ".join(full) + " sum_scale") == mm.ERR_BAD_OPTION
    q = norm(pre_weight=False, training=True)
    for more in ("dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias", "gate", "post_weight", "pre_weight"):
        assert f(q, "stats sum dout dresidual dblock " + more) == mm.ERR_BAD_OPTION, more
    assert f(norm(block=False, pre_weight=False, training=True), "stats sum dout dblock") == mm.ERR_BAD_OPTION
    post = norm(pre=mm.NORM_NONE, post=mm.NORM_RMS, pre_weight=False, training=True)
    assert f(post, "stats block dblock") == mm.ERR_NULL_ARG and f(post, "stats block dblock dsum dout") == mm.ERR_BAD_OPTION
    e = norm(post=mm.NORM_RMS, pre_weight=False, training=True, kept_type=mm.INT8)
    assert f(e, "stats sum block block_scale dout dblock") == mm.ERR_NULL_ARG
    assert f(e, "stats sum sum_scale block dout dblock") == mm.ERR_NULL_ARG
    assert f(p, "") == 0  # nothing wanted
    assert L.mm_norm_backward(None, ctypes.byref(mm.NormBackwardArgs()), None) == mm.ERR_NULL_ARG
    assert L.mm_norm_backward(p.handle, None, None) == mm.ERR_NULL_ARG
    assert f(mm.LinearPlan(4, 64, 32, mm.FLOAT, training=True), "stats") == mm.ERR_BAD_OPTION


def test_binding_refuses_what_does_not_fit():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        norm().execute(x, x, block=x)
    with pytest.raises(ValueError, match="device"):
        norm(training=True).backward(torch.zeros(4, 4), sum=x, dout=x, dX=x)
