"""Cases of the feed-forward block's operators: the product with an epilogue, the gated product, the way back through
both, pre-activations kept in 8 bits, and layer norm with its gradient.

What each operator computes (rows of A are the concatenation of the shards' rows; W is [parts * n, k], parts = 2 for the
gated product, whose first n rows are the gate's and whose others are the factor's):

  linear     p = A @ W^T + bias, y = act(p) + residual
  gated      p = A @ W^T + bias, y = act(p[:, :n]) * p[:, n:]
             Either also returns p for the way back, if asked: rounded to the operands' type, or in e4m3 with a power of
             two for every 32 columns of a row and part, the smallest s with max |p| <= 448 s.  Kept columns are padded
             with zeros to a multiple of 32 per part.
  gradient   of y with respect to A, W and bias, from the p that was kept
  norm       y = (x - mean) * rstd * weight + bias, rstd = 1 / sqrt(var + eps), over a row
  norm_back  its gradient with respect to x, weight and bias, from the mean and rstd that the way forward returned
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODE = {"bf16": "AGMM_BF16", "fp16": "AGMM_FP16", "fp32": "AGMM_FP32"}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # a decoding step's rows (8 shards of 16) before a projection: the call's own cost counts
        dict(name="norm_decode", op="norm", rows=128, cols=4096, dtype="bf16", wtype="bf16"),
        # a training step's rows, fp32 weights
        dict(name="norm_train", op="norm", rows=8192, cols=8192, dtype="bf16", wtype="fp32"),
        # a fine-tuning step's ragged rows, of an odd width
        dict(name="norm_back_ragged", op="norm_back", rows=1011, cols=4035, dtype="fp16", wtype="fp16"),
        # a training step's gradient; the weight's is a sum over all rows
        dict(name="norm_back_train", op="norm_back", rows=8192, cols=8192, dtype="bf16", wtype="fp32"),
        # one token on each of 8 ranks through the projection that ends a block: bias and the residual stream
        dict(name="linear_token", op="linear", shards=8, ms=1, k=4096, n=1792, dtype="bf16", act="none", bias=True, residual=True, keep=0),
        # a long prompt through a block without a gate
        dict(name="linear_prompt", op="linear", shards=8, ms=1024, k=8192, n=3584, dtype="fp16", act="gelu", bias=True, residual=False, keep=0),
        # a training step's way back through such a block, 16-bit pre-activations
        dict(name="linear_gradient", op="gradient", shards=4, ms=512, k=4096, n=1024, dtype="bf16", act="gelu_tanh", gated=False, bias=True, keep=16),
        # one token on each of 8 ranks through a gated block
        dict(name="gated_token", op="gated", shards=8, ms=1, k=4096, n=1792, dtype="bf16", act="silu", bias=False, keep=0),
        # a ragged prompt: shards that end inside tiles, odd n, 8-bit pre-activations kept
        dict(name="gated_ragged", op="gated", shards=3, ms=337, k=4040, n=2051, dtype="fp16", act="gelu_tanh", bias=True, keep=8),
        # a training step's way forward that keeps its pre-activations in 8 bits
        dict(name="gated_train", op="gated", shards=8, ms=1024, k=8192, n=7168, dtype="bf16", act="silu", bias=False, keep=8),
        # a fine-tuning step's few rows, 16-bit pre-activations, biases
        dict(name="gradient_small", op="gradient", shards=3, ms=37, k=1000, n=2051, dtype="fp16", act="silu", gated=True, bias=True, keep=16),
        # a training step's way back from pre-activations in 8 bits
        dict(name="gradient_train", op="gradient", shards=8, ms=1024, k=8192, n=3584, dtype="bf16", act="silu", gated=True, bias=False, keep=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_back", "linear", "gated", "gradient", "gradient"])
    if op.startswith("norm"):
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 16, 8192), dtype=dtype, wtype=rng.choice([dtype, "fp32"]))
    gated = op == "gated" or (op == "gradient" and rng.random() < 0.6)
    case = dict(op=op, shards=rng.choice([1, 2, 3, 4, 8]), ms=_log(rng, 1, 1024), k=_log(rng, 64, 8192),
                n=_log(rng, 16, 3584 if op == "gradient" else 7168), dtype=rng.choice(["bf16", "fp16"]),
                act=rng.choice(["silu", "gelu", "gelu_tanh", "relu", "none"]), bias=rng.random() < 0.5)
    if op == "gradient":
        return dict(case, gated=gated, keep=rng.choice([8, 16]))
    if op == "linear":
        case["residual"] = rng.random() < 0.5
    return dict(case, keep=rng.choice([0, 0, 8, 16]))


def _cdiv(a, b):
    return -(-a // b)


# ---------------------------------------------------------------- inputs


def _noise(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _gated(case):
    return case["op"] == "gated" or case.get("gated", False)


def _parts(case):
    return 2 if _gated(case) else 1


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case=case)
    dtype = TYPES[case["dtype"]]
    if case["op"].startswith("norm"):
        rows, cols = case["rows"], case["cols"]
        # activations with columns of very different sizes and a mean that is not zero
        x = _noise((rows, cols), gen) * (0.2 + 6.0 * torch.rand((1, cols), generator=gen, device="cuda") ** 8) + 0.3
        state["x"] = x.to(dtype)
        state["weight"] = (1.0 + 0.2 * _noise((cols,), gen)).to(TYPES[case["wtype"]])
        state["bias"] = (0.2 * _noise((cols,), gen)).to(TYPES[case["wtype"]])
        if case["op"] == "norm_back":
            x = state["x"].float()
            state["mean"] = x.mean(1)
            state["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt()
            state["dy"] = (_noise((rows, cols), gen) / 64).to(dtype)
        if own:
            import all_gather_gemm_agmm_amd as agmm
            state["plan"] = agmm.NormPlan(rows, cols, getattr(agmm, CODE[case["dtype"]]), getattr(agmm, CODE[case["wtype"]]))
        return state
    m, k, n, parts = case["shards"] * case["ms"], case["k"], case["n"], _parts(case)
    a = (_noise((m, k), gen) * (0.5 + 2.0 * torch.rand((1, k), generator=gen, device="cuda") ** 8)).to(dtype)
    state["shards"] = [s.clone() for s in a.split(case["ms"])]
    state["weight"] = (_noise((parts * n, k), gen) / math.sqrt(k)).to(dtype)
    state["bias"] = (0.1 * _noise((parts * n,), gen)).to(dtype) if case["bias"] else None
    state["residual"] = _noise((m, n), gen).to(dtype) if case.get("residual") else None
    if case["op"] == "gradient":
        state["dy"] = (_noise((m, n), gen) / 64).to(dtype)
        state["kept"] = _keep(case, _plain_pre(state))
    if own:
        import all_gather_gemm_agmm_amd as agmm
        state["plan"] = agmm.FeedForwardPlan(case["shards"], case["ms"], k, n, getattr(agmm, CODE[case["dtype"]]),
                                             activation=case["act"], gated=_gated(case), with_gradient=case["op"] == "gradient")
    return state


# ---------------------------------------------------------------- one pass


def _plain_pre(state):
    p = torch.cat(state["shards"]).float() @ state["weight"].float().t()
    return p if state["bias"] is None else p + state["bias"].float()


def _keep(case, p):
    """The kept pre-activations [m, parts, n up to 32] of p [m, parts * n]: (values, None), or e4m3 values and scales."""
    m, n, parts = p.shape[0], case["n"], _parts(case)
    full = torch.nn.functional.pad(p.view(m, parts, n), (0, -n % 32))
    if case["keep"] == 16:
        return full.to(TYPES[case["dtype"]]), None
    group = full.view(m, parts, -1, 32)
    mantissa, e = torch.frexp(group.abs().amax(3))           # mantissa in [0.5, 1): 448 = 0.875 * 2^9
    e = torch.clamp(e - 9 + (mantissa > 0.875), min=-126)
    e = torch.where(mantissa == 0, torch.full_like(e, -126), e).to(torch.int32)
    inverse = ((127 - e) << 23).view(torch.float32)          # 2^-e, exactly
    values = (group * inverse[..., None]).view(full.shape).to(torch.float8_e4m3fn)
    return values, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _kept_value(case, kept):
    """p [m, parts * n] as the kept pre-activations hold it, fp32."""
    values, scales = kept
    v = values.float()
    if scales is not None:
        v = (v.view(scales.shape + (32,)) * scales.float()[..., None]).view(values.shape)
    return v[:, :, :case["n"]].reshape(v.shape[0], -1)


def _act(act, x):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * torch.special.erfc(-x * math.sqrt(0.5))
    if act == "gelu_tanh":
        return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return x


def _act_slope(act, x):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if act == "gelu":
        return 0.5 * torch.special.erfc(-x * math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (x + 0.044715 * x * x * x)))
        return s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x * x)
    return torch.ones_like(x)


def _plain_forward(state):
    case, n = state["case"], state["case"]["n"]
    dtype, p = TYPES[case["dtype"]], _plain_pre(state)
    y = _act(case["act"], p[:, :n])
    if _gated(case):
        y = y * p[:, n:]
    if state["residual"] is not None:
        y = y + state["residual"].float()
    y = y.to(dtype)
    if not case["keep"]:
        return [y]
    values, scales = _keep(case, p)
    return [y, values] if scales is None else [y, values, scales]


def _plain_gradient(state):
    case, n = state["case"], state["case"]["n"]
    dtype, p, dy = TYPES[case["dtype"]], _kept_value(case, state["kept"]), state["dy"].float()
    g = p[:, :n]
    if _gated(case):
        d = torch.cat([dy * p[:, n:] * _act_slope(case["act"], g), dy * _act(case["act"], g)], 1)
    else:
        d = dy * _act_slope(case["act"], g)
    da, dw = d @ state["weight"].float(), d.t() @ torch.cat(state["shards"]).float()
    got = [da.to(dtype), dw.to(dtype)]
    return got + [d.sum(0).to(dtype)] if case["bias"] else got


def _plain_norm(state):
    x = state["x"].float()
    mean = x.mean(1)
    off = x - mean[:, None]
    rstd = 1 / torch.sqrt((off * off).mean(1) + EPS)
    y = off * rstd[:, None] * state["weight"].float() + state["bias"].float()
    return [y.to(state["x"].dtype), mean, rstd]


def _plain_norm_back(state):
    x, dy, w, rstd = state["x"].float(), state["dy"].float(), state["weight"], state["rstd"][:, None]
    hat = (x - state["mean"][:, None]) * rstd
    g = dy * w.float()
    dx = rstd * (g - g.mean(1, keepdim=True) - hat * (g * hat).mean(1, keepdim=True))
    return [dx.to(state["x"].dtype), (dy * hat).sum(0).to(w.dtype), dy.sum(0).to(w.dtype)]


def run(state):
    case = state["case"]
    if not own:
        return {"norm": _plain_norm, "norm_back": _plain_norm_back, "gradient": _plain_gradient}.get(case["op"], _plain_forward)(state)
    plan = state["plan"]
    if case["op"] == "norm":
        return list(plan.forward(state["x"], state["weight"], state["bias"], eps=EPS))
    if case["op"] == "norm_back":
        return list(plan.backward(state["x"], state["dy"], state["weight"], state["mean"], state["rstd"]))
    if case["op"] == "gradient":
        import all_gather_gemm_agmm_amd as agmm
        got = plan.backward(state["shards"], state["weight"], agmm.Checkpoint(*state["kept"], case["n"]), state["dy"], need_dbias=case["bias"])
        return list(got) if case["bias"] else list(got[:2])
    if not case["keep"]:
        return [plan.forward(state["shards"], state["weight"], state["bias"], state["residual"])]
    y, kept = plan.forward(state["shards"], state["weight"], state["bias"], state["residual"], keep=case["keep"])
    return [y, kept.values] if kept.scales is None else [y, kept.values, kept.scales]


def work(case):
    if case["op"].startswith("norm"):
        values, s, w = case["rows"] * case["cols"], SIZE[case["dtype"]], SIZE[case["wtype"]]
        if case["op"] == "norm":
            return {"bytes": 2 * s * values + 2 * w * case["cols"] + 8 * case["rows"], "flops": 8 * values}
        return {"bytes": 3 * s * values + 3 * w * case["cols"] + 8 * case["rows"], "flops": 14 * values}
    m, k, n, parts = case["shards"] * case["ms"], case["k"], case["n"], _parts(case)
    kept = m * parts * n * {0: 0, 8: 33 / 32, 16: 2}[case["keep"]]
    if case["op"] == "gradient":
        return {"bytes": 4 * (m + parts * n) * k + 2 * m * n + kept + (2 * parts * n if case["bias"] else 0), "flops": 4 * m * parts * n * k}
    rows = 2 * m * n * (2 if case.get("residual") else 1)
    return {"bytes": 2 * (m + parts * n) * k + rows + kept + (2 * parts * n if case["bias"] else 0), "flops": 2 * m * parts * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits


def _nearest_e4m3(v):
    """Nearest e4m3 value (even mantissa on a tie) of finite 64-bit v within its range."""
    _, e = torch.frexp(v)
    step = ((torch.clamp(e - 1, min=-6).long() - 3 + 1023) << 52).view(torch.float64)
    return torch.round(v / step) * step


def _exact_unit(act, x):
    """An activation and its derivative at 64-bit x."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        return x.clamp(min=0), torch.heaviside(x, torch.zeros_like(x))
    if act == "gelu":
        share = torch.special.ndtr(x)
        return x * share, share + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        share, inner = torch.sigmoid(x), torch.ones_like(x)
    else:
        share = torch.sigmoid(math.sqrt(8 / math.pi) * (x + 0.044715 * x ** 3))
        inner = math.sqrt(8 / math.pi) * (1 + 0.134145 * x ** 2)
    return x * share, share + x * share * (1 - share) * inner


def _exact_forward(state):
    case, n, parts = state["case"], state["case"]["n"], _parts(state["case"])
    a = torch.cat(state["shards"]).double()
    half = []
    for q in range(parts):
        p = a @ state["weight"][q * n:(q + 1) * n].double().t()
        half.append(p if state["bias"] is None else p + state["bias"][q * n:(q + 1) * n].double())
    y = _exact_unit(case["act"], half[0])[0]
    if parts == 2:
        y = y * half[1]
    if state["residual"] is not None:
        y = y + state["residual"].double()
    if case["keep"] == 0:
        return [y]
    m, wide = len(a), _cdiv(n, 32) * 32
    kept = torch.zeros((m, parts, wide), dtype=torch.float64, device=a.device)
    for q in range(parts):
        kept[:, q, :n] = half[q]
    if case["keep"] == 16:
        return [y, kept]
    top = kept.view(m, parts, wide // 32, 32).abs().amax(3)
    power = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, 2.0 ** -130)) / 448)).clamp(min=-126)
    scale = ((power.long() + 1023) << 52).view(torch.float64)
    return [y, _nearest_e4m3(kept / scale.repeat_interleave(32, dim=2)), scale]


def _exact_gradient(state):
    case, n, parts = state["case"], state["case"]["n"], _parts(state["case"])
    values, scales = state["kept"]
    p = values.double() if scales is None else values.double() * scales.double().repeat_interleave(32, dim=2)
    y, slope = _exact_unit(case["act"], p[:, 0, :n])
    dy = state["dy"].double()
    ds = [dy * slope] if parts == 1 else [dy * p[:, 1, :n] * slope, dy * y]
    a, da, dw, db = torch.cat(state["shards"]).double(), 0.0, [], []
    for q in range(parts):
        da = da + ds[q] @ state["weight"][q * n:(q + 1) * n].double()
        dw.append(ds[q].t() @ a)
        db.append(ds[q].sum(0))
    return [da, torch.cat(dw)] + ([torch.cat(db)] if case["bias"] else [])


def _exact_norm(state):
    x = state["x"].double()
    mean, var = x.mean(1), x.var(1, unbiased=False)
    rstd = (var + EPS) ** -0.5
    return [(x - mean[:, None]) * rstd[:, None] * state["weight"].double() + state["bias"].double(), mean, rstd]


def _exact_norm_back(state):
    x, dy = state["x"].double(), state["dy"].double()
    rstd = state["rstd"].double()[:, None]
    hat = (x - state["mean"].double()[:, None]) * rstd
    g = dy * state["weight"].double()
    cols = x.shape[1]
    dx = rstd / cols * (cols * g - g.sum(1, keepdim=True) - hat * (g * hat).sum(1, keepdim=True))
    return [dx, torch.einsum("ij,ij->j", dy, hat), dy.sum(0)]


def exact(case, seed):
    state = prepare(case, seed)
    return {"norm": _exact_norm, "norm_back": _exact_norm_back, "gradient": _exact_gradient}.get(case["op"], _exact_forward)(state)
