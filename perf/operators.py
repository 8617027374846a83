"""Measured cases of the gated feed-forward block and of the 8-bit product
with scales for each token and channel.

Kinds of case:

* ``glu``: ``H = act(X Wg) * (X Wu)`` (inference).
* ``glu_train``: the same forward pass, keeping ``G = X Wg`` and ``U = X Wu``,
  then the backward pass from ``dH`` to ``dX``, ``dWg`` and ``dWu``.
* ``product``: ``Y = sa[m] * sb[n] * sum_k A[m][k] B[k][n] (+ bias[n])`` with
  8-bit integers A and B that were quantized before.
* ``linear``: the same with A quantized row by row inside the call from the
  16- or 32-bit X: ``s = amax / 127`` and ``q = rint(x * r)``, ``r = 127 /
  amax`` rounded to 32 bits, where ``amax`` is the row's largest magnitude
  (at least 2^-100).

``own`` selects what ``run`` does: false, the plain form in elementary torch
operations; true, this library's calls.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SMALLEST = 2.0 ** -100  # least row magnitude that the row scale is formed from


def listed():
    """The listed cases.  m: tokens, k: input features, n: output features
    (hidden features of the gated block); nk: weights stored [n, k], as linear
    layers keep them, else [k, n]."""
    return [
        # One decoded token through the block of a 4096-wide model: weights
        # streamed once.
        {"name": "glu_token", "kind": "glu", "dtype": "bf16", "act": "silu", "nk": True, "m": 1, "k": 4096, "n": 11008},
        # A decode batch of 13 sequences of a smaller model whose hidden width
        # (8/3 of 2048) is odd.
        {"name": "glu_batch13_odd", "kind": "glu", "dtype": "fp16", "act": "gelu_tanh", "nk": True, "m": 13, "k": 2048, "n": 5461},
        # A short prompt, weights in the [k, n] order of an ONNX MatMul, exact gelu.
        {"name": "glu_prompt_kn", "kind": "glu", "dtype": "fp16", "act": "gelu", "nk": False, "m": 1000, "k": 1024, "n": 4096},
        # 16 prompts of 512 tokens.
        {"name": "glu_prefill", "kind": "glu", "dtype": "bf16", "act": "silu", "nk": True, "m": 8192, "k": 4096, "n": 11008},
        # Training in 32 bits of a small model on a ragged batch (the kind of
        # run that gradients are checked on), weights [k, n].
        {"name": "glu_train_fp32", "kind": "glu_train", "dtype": "fp32", "act": "gelu", "nk": False, "m": 300, "k": 512, "n": 1364},
        # A training microbatch of 2 x 2048 tokens of a 2048-wide model.
        {"name": "glu_train", "kind": "glu_train", "dtype": "bf16", "act": "silu", "nk": True, "m": 4096, "k": 2048, "n": 5504},
        # A training batch of the 4096-wide model.
        {"name": "glu_train_large", "kind": "glu_train", "dtype": "bf16", "act": "silu", "nk": True, "m": 8192, "k": 4096, "n": 11008},
        # One decoded token through the block's last layer, weights in 8 bits.
        {"name": "linear_token", "kind": "linear", "dtype": "bf16", "out": "bf16", "bias": False, "nk": True, "m": 1, "k": 11008, "n": 4096},
        # A decode batch of 24 sequences through an attention projection with a
        # bias, weights in the [k, n] order.
        {"name": "linear_batch24_kn", "kind": "linear", "dtype": "fp16", "out": "fp16", "bias": True, "nk": False, "m": 24, "k": 4096, "n": 4096},
        # 16 prompts of 512 tokens, activations quantized in the call.
        {"name": "linear_prefill", "kind": "linear", "dtype": "bf16", "out": "bf16", "bias": False, "nk": True, "m": 8192, "k": 4096, "n": 11008},
        # Activations quantized once for several layers; ragged sizes, 32-bit result.
        {"name": "product_ragged", "kind": "product", "out": "fp32", "bias": True, "nk": True, "m": 333, "k": 1000, "n": 1501},
        # The block's last layer over 2048 tokens, operands quantized before.
        {"name": "product_down", "kind": "product", "out": "bf16", "bias": False, "nk": True, "m": 2048, "k": 11008, "n": 4096},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    """One more case of the same ranges: every kind, type, weight order and
    activation, one token to 8192, widths from 64 to 11008, odd and ragged
    sizes among them, no costlier than the largest listed case."""
    kind = rng.choice(["glu", "glu", "glu_train", "glu_train", "linear", "linear", "product"])
    m = _log(rng, 1, 8192)
    k, n = _log(rng, 64, 8192), _log(rng, 64, 11008)
    if rng.random() < 0.5:  # widths of real layers are mostly whole multiples; the rest stay as drawn
        k, n = (k + 63) // 64 * 64, (n + 63) // 64 * 64
    if kind == "glu_train":
        m = max(m, 16)
    case = {"kind": kind, "nk": rng.random() < 0.6, "m": m, "k": k, "n": n}
    if kind in ("glu", "glu_train"):
        case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        case["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
        if case["dtype"] == "fp32":
            case["m"] = max(1, m // 4)  # 32-bit blocks are the small ones
    else:
        case["bias"] = rng.random() < 0.5
        case["out"] = rng.choice(["bf16", "fp16", "fp32"])
        if kind == "linear":
            case["dtype"] = case["out"]
    return case


def prepare(case, seed):
    """Inputs on the GPU (and the plan and result buffers where ``own``)."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    m, k, n = case["m"], case["k"], case["n"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * scale

    st = {"case": case}
    w_shape = (n, k) if case["nk"] else (k, n)
    if case["kind"] in ("glu", "glu_train"):
        dt = DTYPES[case["dtype"]]
        st["x"] = normal(m, k).to(dt)  # after a norm: unit variance
        st["wg"] = normal(*w_shape, scale=k ** -0.5).to(dt)
        st["wu"] = normal(*w_shape, scale=k ** -0.5).to(dt)
        if case["kind"] == "glu_train":
            st["dh"] = normal(m, n, scale=0.1).to(dt)
    else:
        # Activations with a few channels of large magnitude; weights quantized
        # by output channel.
        x = normal(m, k)
        loud = torch.rand(k, generator=gen, device=dev) < 0.01
        x = torch.where(loud, x * 12.0, x)
        w = normal(*w_shape, scale=k ** -0.5)
        amax = w.abs().amax(dim=1 if case["nk"] else 0, keepdim=True).clamp_min(SMALLEST)
        st["w"] = torch.round(w * (127.0 / amax)).clamp_(-127, 127).to(torch.int8)
        st["sb"] = (amax / 127.0).reshape(n).contiguous()
        if case["kind"] == "linear":
            st["x"] = x.to(DTYPES[case["dtype"]])
        else:
            amax = x.abs().amax(dim=1, keepdim=True).clamp_min(SMALLEST)
            st["a"] = torch.round(x * (127.0 / amax)).clamp_(-127, 127).to(torch.int8)
            st["sa"] = (amax / 127.0).reshape(m).contiguous()
        st["bias"] = normal(n).to(DTYPES[case["out"]]) if case["bias"] else None
    if own:
        _plan(case, st, dev)
    return st


def _plan(case, st, dev):
    from onnx_broadcast_matmul_amd import binding as mm

    m, k, n = case["m"], case["k"], case["n"]
    if case["kind"] in ("glu", "glu_train"):
        dt = DTYPES[case["dtype"]]
        train = case["kind"] == "glu_train"
        # A training step keeps G and U in 32 bits, as the plain form does:
        # rounded to 16 they would make the gradients a third less exact.
        st["plan"] = mm.GluPlan(m, k, n, mm.torch_dtype_code(dt), activation=mm.ACTIVATIONS[case["act"]],
                                trans_w=case["nk"], training=train, kept_type=mm.FLOAT if train else 0)
        st["h"] = torch.empty(m, n, dtype=dt, device=dev)
        if train:
            st["g"], st["u"] = (torch.empty(m, n, dtype=torch.float32, device=dev) for _ in range(2))
            st["dx"] = torch.empty_like(st["x"])
            st["dwg"], st["dwu"] = torch.empty_like(st["wg"]), torch.empty_like(st["wu"])
    else:
        dt = DTYPES[case["out"]]
        a = st["x"] if case["kind"] == "linear" else st["a"]
        a_type = mm.torch_dtype_code(a.dtype) if case["kind"] == "linear" else mm.INT8
        st["plan"] = mm.ScaledIntPlan((m, k), tuple(st["w"].shape), mm.torch_dtype_code(dt), a_type=a_type,
                                      trans_b=case["nk"], bias=case["bias"])
        st["y"] = torch.empty(m, n, dtype=dt, device=dev)


def run(state):
    """One pass: H (and the gradients), or Y."""
    kind = state["case"]["kind"]
    if own:
        plan = state["plan"]
        if kind == "glu":
            plan.execute(state["x"], state["wg"], state["wu"], state["h"])
            return state["h"]
        if kind == "glu_train":
            plan.execute(state["x"], state["wg"], state["wu"], state["h"], state["g"], state["u"])
            plan.backward(state["x"], state["wg"], state["wu"], state["g"], state["u"], state["dh"],
                          state["dx"], state["dwg"], state["dwu"])
            return {"h": state["h"], "dx": state["dx"], "dwg": state["dwg"], "dwu": state["dwu"]}
        if kind == "linear":
            plan.execute(state["x"], state["w"], state["y"], b_scale=state["sb"], bias=state["bias"])
        else:
            plan.execute(state["a"], state["w"], state["y"], a_scale=state["sa"], b_scale=state["sb"],
                         bias=state["bias"])
        return state["y"]
    if kind in ("glu", "glu_train"):
        return _plain_glu(state)
    return _plain_product(state)


# ---- plain forms


def _act(name, g):
    """act(g) and its derivative, in g's type."""
    if name == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if name == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * (0.5 ** 0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5
    if name == "gelu_tanh":
        c = (2.0 / math.pi) ** 0.5
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)
    s = 1.0 / (1.0 + torch.exp(-g))
    if name == "sigmoid":
        return s, s * (1.0 - s)
    return g * s, s * (1.0 + g * (1.0 - s))  # silu


def _plain_glu(state):
    case, dt = state["case"], state["x"].dtype
    x, wg, wu = state["x"].float(), state["wg"].float(), state["wu"].float()
    if case["nk"]:
        wg, wu = wg.t(), wu.t()
    g, u = x @ wg, x @ wu
    a, d = _act(case["act"], g)
    h = (a * u).to(dt)
    if case["kind"] == "glu":
        return h
    dh = state["dh"].float()
    dg, du = dh * u * d, dh * a
    dx = dg @ wg.t() + du @ wu.t()
    if case["nk"]:
        dwg, dwu = dg.t() @ x, du.t() @ x
    else:
        dwg, dwu = x.t() @ dg, x.t() @ du
    return {"h": h, "dx": dx.to(dt), "dwg": dwg.to(dt), "dwu": dwu.to(dt)}


def _plain_product(state):
    case = state["case"]
    if case["kind"] == "linear":
        x = state["x"].float()
        amax = x.abs().amax(dim=1, keepdim=True).clamp_min(SMALLEST)
        c127 = torch.full_like(amax, 127.0)
        a = torch.round(x * (c127 / amax)).clamp(-127.0, 127.0)
        sa = amax / c127
    else:
        a, sa = state["a"].float(), state["sa"].reshape(-1, 1)
    w = state["w"].float()
    if case["nk"]:
        w = w.t()
    y = (a @ w) * sa * state["sb"]
    if state["bias"] is not None:
        y = y + state["bias"].float()
    return y.to(DTYPES[case["out"]])


# ---- what a pass cannot do without


def work(case):
    m, k, n = case["m"], case["k"], case["n"]
    if case["kind"] in ("glu", "glu_train"):
        es = 4 if case["dtype"] == "fp32" else 2
        if case["kind"] == "glu":
            return {"bytes": es * (m * k + 2 * k * n + m * n), "flops": 4 * m * k * n}
        # forward, dX and the weight gradients: two products each; inputs
        # X, Wg, Wu, dH and outputs H, dX, dWg, dWu once
        return {"bytes": es * (2 * m * k + 4 * k * n + 2 * m * n), "flops": 12 * m * k * n}
    eo = 4 if case["out"] == "fp32" else 2
    ea = 1 if case["kind"] == "product" else 4 if case["dtype"] == "fp32" else 2
    scales = 4 * (m + n) if case["kind"] == "product" else 4 * n
    return {"bytes": ea * m * k + k * n + scales + eo * (m * n + (n if case["bias"] else 0)), "flops": 2 * m * k * n}


# ---- the definitions in 64 bits


def exact(case, seed):
    """run's results in 64 bits.  The row quantization's reciprocal and product
    are rounded to 32 bits, as its definition says."""
    st = prepare(case, seed)
    if case["kind"] in ("linear", "product"):
        if case["kind"] == "linear":
            x = st["x"].double()
            top = torch.clamp(torch.amax(torch.abs(x), 1), min=SMALLEST)
            r = torch.div(torch.full_like(top, 127.0), top).float().double()
            q = torch.round((x * r[:, None]).float()).double()
            sa = top / torch.full_like(top, 127.0)
        else:
            q, sa = st["a"].double(), st["sa"].double()
        w = st["w"].double()
        y = torch.matmul(q, w.T if case["nk"] else w)
        y *= torch.outer(sa, st["sb"].double())
        if st["bias"] is not None:
            y += st["bias"].double()
        return y

    x = st["x"].double()
    order = (lambda t: t.double().T.contiguous()) if case["nk"] else (lambda t: t.double())
    wg, wu = order(st["wg"]), order(st["wu"])
    g, u = torch.matmul(x, wg), torch.matmul(x, wu)
    act = case["act"]
    if act == "relu":
        f, df = torch.where(g > 0, g, torch.zeros_like(g)), (g > 0).double()
    elif act == "sigmoid":
        f = torch.sigmoid(g)
        df = f * torch.sigmoid(-g)
    elif act == "silu":
        s = torch.sigmoid(g)
        f, df = g * s, s + g * s * torch.sigmoid(-g)
    elif act == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        f, df = g * p, p + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    else:
        z = math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3)
        p = torch.sigmoid(z)  # (1 + tanh(z / 2)) / 2
        f, df = g * p, p + g * p * torch.sigmoid(-z) * math.sqrt(8.0 / math.pi) * (1.0 + 0.134145 * g ** 2)
    if case["kind"] == "glu":
        return f * u
    dh = st["dh"].double()
    dg, du = dh * u * df, dh * f
    dx = torch.matmul(dg, wg.T) + torch.matmul(du, wu.T)
    dwg, dwu = torch.matmul(x.T, dg), torch.matmul(x.T, du)
    if case["nk"]:
        dwg, dwu = dwg.T.contiguous(), dwu.T.contiguous()
    return {"h": f * u, "dx": dx, "dwg": dwg, "dwu": dwu}
