"""Cases of the block-scaled 8-bit product, its quantiser, and the vocabulary loss with its gradient.

What each operator computes (rows of A are the concatenation of the shards' rows):

  quantize   x[rows, cols] -> 8-bit values q and one fp32 scale s per block of 128 elements of a row (block_rows 1) or
             per 128 x 128 block, s = max |x| of the block over the format's largest value, q = x / s; of x, of x
             transposed, or of both.  Scales are stored [block of k][row block].
  product    C[i, j] = sum over blocks b of 128 of k: sa[b, i] * sb[b, j / block_rows] * sum_{k in b} qa[i, k] * qb[j, k]
  loss       logits = A @ W^T over a slice of the vocabulary; per row lse = log sum exp, target = the label's logit,
             loss = lse - target (0 for rows whose label is -100)
  gradient   of the loss (and of the lse, as a z-loss needs it) with respect to A and W
"""
import math

import torch

own = False

IGNORE = -100
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CODE = {"bf16": "AGMM_BF16", "fp16": "AGMM_FP16", "fp32": "AGMM_FP32"}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
TINY = 2.0 ** -126


def listed():
    return [
        # activations of a decoding step (8 shards of 16 rows, gathered) before a projection: the call's own cost counts
        dict(name="quantize_decode", op="quantize", rows=128, cols=4096, dtype="bf16", fmt="e4m3", block=1, out="rows"),
        # a training step's activations: row blocks for the forward product, transposed for the weight gradient
        dict(name="quantize_both", op="quantize", rows=8192, cols=8192, dtype="bf16", fmt="e4m3", block=1, out="both"),
        # fp32 master weights of a projection after an optimiser step, both ways round
        dict(name="quantize_weight", op="quantize", rows=7168, cols=8192, dtype="fp32", fmt="e4m3", block=128, out="both"),
        # one token on each of 8 ranks
        dict(name="product_token", op="product", shards=8, ms=1, k=4096, n=1792, fmt="e4m3", block=128, out="bf16"),
        # a decoding batch
        dict(name="product_decode", op="product", shards=8, ms=16, k=8192, n=3584, fmt="e4m3", block=128, out="bf16"),
        # a ragged prompt: shards that end inside tiles, k that ends inside a scale block, odd n
        dict(name="product_ragged", op="product", shards=3, ms=337, k=4040, n=2051, fmt="e4m3", block=128, out="fp16"),
        # a long prompt or a training step's forward product
        dict(name="product_prompt", op="product", shards=8, ms=4096, k=8192, n=7168, fmt="e4m3", block=128, out="bf16"),
        # a weight gradient: both operands transposed activations with a scale per row, e5m2 output gradients, fp32 result
        dict(name="product_wgrad", op="product", shards=1, ms=3584, k=8192, n=4096, fmt="e5m2", block=1, out="fp32"),
        # log-probabilities of one token on each of 8 ranks over a large vocabulary: one pass over the weights
        dict(name="loss_token", op="loss", shards=8, ms=1, k=4096, n=131072, start=0, total=131072, dtype="fp16"),
        # a training step's rows over a large vocabulary
        dict(name="loss_train", op="loss", shards=8, ms=1024, k=4096, n=131072, start=0, total=131072, dtype="bf16"),
        # a fine-tuning step's few rows over a quarter of an odd vocabulary, with the gradient of a z-loss
        dict(name="gradient_small", op="gradient", shards=3, ms=37, k=1000, n=10007, start=10007, total=40028, dtype="fp16", z=True),
        # a training step's rows over one rank's half of the vocabulary
        dict(name="gradient_train", op="gradient", shards=8, ms=1024, k=4096, n=65536, start=65536, total=131072, dtype="bf16", z=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "loss", "gradient"])
    if op == "quantize":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 16, 8192), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    fmt=rng.choice(["e4m3", "e5m2"]), block=rng.choice([1, 128]), out=rng.choice(["rows", "cols", "both"]))
    shards = rng.choice([1, 2, 3, 4, 8])
    if op == "product":
        return dict(op=op, shards=shards, ms=_log(rng, 1, 4096), k=_log(rng, 64, 8192), n=_log(rng, 16, 7168),
                    fmt=rng.choice(["e4m3", "e5m2"]), block=rng.choice([1, 128]), out=rng.choice(["bf16", "fp16", "fp32"]))
    parts = rng.choice([1, 2, 4])
    n = _log(rng, 500, 131072 if op == "loss" else 65536)
    case = dict(op=op, shards=shards, ms=_log(rng, 1, 1024), k=_log(rng, 64, 4096), n=n, start=n * rng.randrange(parts),
                total=n * parts, dtype=rng.choice(["bf16", "fp16"]))
    if op == "gradient":
        case["z"] = rng.random() < 0.5
    return case


def _cdiv(a, b):
    return -(-a // b)


def _round(a, b):
    return _cdiv(a, b) * b


# ---------------------------------------------------------------- inputs


def _noise(shape, gen):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32)


def _quantize_rows(x, fmt, block):
    """Values [rows, cols up to 16] and scales [blocks of cols][rows / block] of x, in elementary operations."""
    rows, cols = x.shape
    kb, rb = _cdiv(cols, 128), _cdiv(rows, block)
    full = torch.nn.functional.pad(x.float(), (0, kb * 128 - cols, 0, rb * block - rows)).view(rb, block, kb, 128)
    size = full.abs()
    size = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(dim=(1, 3))
    scale = torch.clamp(size / TOP[fmt], min=TINY)
    values = (full * (1.0 / scale)[:, None, :, None]).view(rb * block, kb * 128)[:rows, :_round(cols, 16)]
    return values.to(FLOAT8[fmt]).contiguous(), scale.t().contiguous()


def _hidden(case, gen):
    """Shards, W and labels of a loss: logits of spread 1, labels likelier than the rest, one row in ten ignored."""
    m, k, n = case["shards"] * case["ms"], case["k"], case["n"]
    weight = _noise((n, k), gen).mul_(1.0 / math.sqrt(k)).to(TYPES[case["dtype"]])
    labels = torch.randint(0, case["total"], (m,), generator=gen, device=gen.device)
    inside = (labels >= case["start"]) & (labels < case["start"] + n)
    at = torch.where(inside, labels - case["start"], torch.zeros_like(labels))
    pull = torch.rand((m, 1), generator=gen, device=gen.device) * 14 * inside[:, None]
    hidden = (_noise((m, k), gen) + pull * weight[at].float()).to(TYPES[case["dtype"]])
    near = (hidden.float() * weight[at].float()).sum(1)
    lse = torch.log(case["total"] * math.exp(0.5) + torch.where(inside, near.exp(), torch.full_like(near, 50.0)))
    labels = torch.where(torch.rand((m,), generator=gen, device=gen.device) < 0.1, torch.full_like(labels, IGNORE), labels)
    return [s.clone() for s in hidden.split(case["ms"])], weight, labels, lse


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case=case)
    if case["op"] == "quantize":
        x = _noise((case["rows"], case["cols"]), gen) * (0.1 + 8.0 * torch.rand((1, case["cols"]), generator=gen, device="cuda") ** 8)
        state["x"] = x.to(TYPES[case["dtype"]])
        return state
    if case["op"] == "product":
        m, k, n = case["shards"] * case["ms"], case["k"], case["n"]
        a = _noise((m, k), gen) * (0.1 + 4.0 * torch.rand((1, k), generator=gen, device="cuda") ** 8)
        state["shards"] = [_quantize_rows(s, case["fmt"], 1) for s in a.split(case["ms"])]
        state["weight"] = _quantize_rows(_noise((n, k), gen) / math.sqrt(k), "e4m3", case["block"])
        if own:
            import all_gather_gemm_agmm_amd as agmm
            state["plan"] = agmm.ScaledPlan(case["shards"], case["ms"], k, n, case["fmt"], case["block"],
                                            getattr(agmm, CODE[case["out"]]))
        return state
    state["shards"], state["weight"], state["labels"], state["lse"] = _hidden(case, gen)
    if case["op"] == "gradient":
        m = len(state["labels"])
        state["grad_loss"] = torch.full((m,), 1.0 / m, device="cuda")
        state["grad_lse"] = 2e-4 / m * state["lse"] if case["z"] else None
    if own:
        import all_gather_gemm_agmm_amd as agmm
        state["plan"] = agmm.LossPlan(case["shards"], case["ms"], case["k"], case["n"], getattr(agmm, CODE[case["dtype"]]),
                                      vocab_start=case["start"], vocab_size=case["total"])
    return state


# ---------------------------------------------------------------- one pass


def _plain_quantize(case, x):
    if case["out"] == "rows":
        return _quantize_rows(x, case["fmt"], case["block"])
    if case["out"] == "cols":
        return _quantize_rows(x.t(), case["fmt"], case["block"])
    return _quantize_rows(x, case["fmt"], case["block"]) + _quantize_rows(x.t(), case["fmt"], case["block"])


def _spread(values, scales, k, block):
    """The fp32 matrix that 8-bit values [rows, cols up to 16] and scales [k blocks][rows / block] stand for."""
    s = scales.t().repeat_interleave(128, dim=1)[:, :k]
    return values[:, :k].float() * (s.repeat_interleave(block, dim=0)[: values.shape[0]] if block > 1 else s)


def _plain_product(state):
    case = state["case"]
    a = torch.cat([_spread(q, s, case["k"], 1) for q, s in state["shards"]])
    return (a @ _spread(*state["weight"], case["k"], case["block"]).t()).to(TYPES[case["out"]])


def _inside(case, labels):
    here = (labels >= case["start"]) & (labels < case["start"] + case["n"])
    return here, torch.where(here, labels - case["start"], torch.zeros_like(labels))


def _plain_loss(state):
    case, labels = state["case"], state["labels"]
    logits = torch.cat(state["shards"]).float() @ state["weight"].float().t()
    top = logits.amax(1)
    lse = top + (logits - top[:, None]).exp_().sum(1).log()
    here, at = _inside(case, labels)
    target = torch.where(here, logits.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    return torch.where(labels == IGNORE, torch.zeros_like(lse), lse - target), lse, target


def _plain_gradient(state):
    case, labels = state["case"], state["labels"]
    a, w = torch.cat(state["shards"]).float(), state["weight"].float()
    grad = torch.where(labels == IGNORE, torch.zeros_like(state["grad_loss"]), state["grad_loss"])
    both = grad if state["grad_lse"] is None else grad + state["grad_lse"]
    d = (a @ w.t()).sub_(state["lse"][:, None]).exp_().mul_(both[:, None])
    here, at = _inside(case, labels)
    d.scatter_add_(1, at[:, None], torch.where(here, -grad, torch.zeros_like(grad))[:, None])
    return (d @ w).to(state["weight"].dtype), (d.t() @ a).to(state["weight"].dtype)


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "quantize":
            return _plain_quantize(case, state["x"])
        return {"product": _plain_product, "loss": _plain_loss, "gradient": _plain_gradient}[case["op"]](state)
    import all_gather_gemm_agmm_amd as agmm
    if case["op"] == "quantize":
        got = agmm.quantize(state["x"], case["fmt"], block_rows=case["block"], out=case["out"])
        return (got.values, got.scales) if case["out"] != "both" else (got[0].values, got[0].scales, got[1].values, got[1].scales)
    if case["op"] == "product":
        shards = [agmm.Scaled(q, s, case["k"], 1) for q, s in state["shards"]]
        return state["plan"].run(shards, agmm.Scaled(*state["weight"], case["k"], case["block"]))
    if case["op"] == "loss":
        return state["plan"].forward(state["shards"], state["weight"], state["labels"])
    return state["plan"].backward(state["shards"], state["weight"], state["labels"], state["lse"], state["grad_loss"], state["grad_lse"])


def work(case):
    if case["op"] == "quantize":
        ways = 2 if case["out"] == "both" else 1
        values = case["rows"] * case["cols"]
        return {"bytes": values * (SIZE[case["dtype"]] + ways) + 4 * ways * values / (128 * case["block"]), "flops": 3 * ways * values}
    m, k, n = case["shards"] * case["ms"], case["k"], case["n"]
    if case["op"] == "product":
        scales = _cdiv(k, 128) * (m + _cdiv(n, case["block"]))
        return {"bytes": m * k + n * k + 4 * scales + SIZE[case["out"]] * m * n, "flops": 2 * m * n * k}
    if case["op"] == "loss":
        return {"bytes": 2 * (m + n) * k + 20 * m, "flops": 2 * m * n * k}
    return {"bytes": 4 * (m + n) * k + 24 * m, "flops": 6 * m * n * k}


# ---------------------------------------------------------------- the definitions in 64 bits


def _nearest8(v, fmt):
    """Nearest value of the format (even mantissa on a tie) of finite 64-bit v within its range."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (torch.clamp(e - 1, min=low) - bits))
    return torch.round(v / step) * step


def _exact_quantize(x, fmt, block):
    rows, cols = x.shape
    values = torch.zeros((rows, _round(cols, 16)), dtype=torch.float64, device=x.device)
    scales = torch.zeros((_cdiv(cols, 128), _cdiv(rows, block)), dtype=torch.float64, device=x.device)
    for b in range(scales.shape[0]):
        part = x[:, 128 * b: 128 * (b + 1)].double()
        top = part.abs().amax(1)
        group = torch.arange(rows, device=x.device) // block
        size = torch.zeros(scales.shape[1], dtype=torch.float64, device=x.device).scatter_reduce(0, group, top, "amax")
        # the scale is held in 32 bits, and the values are those of x over the scale as it is held
        scales[b] = torch.clamp(size / TOP[fmt], min=TINY).float().double()
        values[:, 128 * b: 128 * b + part.shape[1]] = _nearest8(part / scales[b][group][:, None], fmt)
    return [values, scales]


def _exact_product(state):
    case, out = state["case"], 0.0
    a = torch.cat([q for q, _ in state["shards"]]).double()
    sa = torch.cat([s for _, s in state["shards"]], dim=1).double()
    qb, sb = state["weight"][0].double(), state["weight"][1].double()
    column = torch.arange(case["n"], device=qb.device) // case["block"]
    for b in range(sa.shape[0]):
        lo, hi = 128 * b, min(128 * (b + 1), case["k"])
        out = out + (a[:, lo:hi] * sa[b][:, None]) @ (qb[:, lo:hi] * sb[b][column][:, None]).t()
    return out


def _exact_loss(state):
    case, labels = state["case"], state["labels"]
    a = torch.cat(state["shards"]).double()
    lse = torch.full((len(a),), -math.inf, dtype=torch.float64, device=a.device)
    target = torch.zeros_like(lse)
    for lo in range(0, case["n"], 16384):
        part = a @ state["weight"][lo: lo + 16384].double().t()
        lse = torch.logaddexp(lse, torch.logsumexp(part, dim=1))
        at = labels - case["start"] - lo
        hit = ((at >= 0) & (at < part.shape[1])).nonzero()[:, 0]
        target[hit] = part[hit, at[hit]]
    return [(lse - target) * (labels != IGNORE), lse, target]


def _exact_gradient(state):
    case, labels = state["case"], state["labels"]
    a = torch.cat(state["shards"]).double()
    da, dw = torch.zeros_like(a), torch.zeros(state["weight"].shape, dtype=torch.float64, device=a.device)
    grad = state["grad_loss"].double() * (labels != IGNORE)
    both = grad + (0.0 if state["grad_lse"] is None else state["grad_lse"].double())
    for lo in range(0, case["n"], 16384):
        w = state["weight"][lo: lo + 16384].double()
        d = both[:, None] * torch.exp(a @ w.t() - state["lse"].double()[:, None])
        at = labels - case["start"] - lo
        hit = ((at >= 0) & (at < len(w))).nonzero()[:, 0]
        d[hit, at[hit]] -= grad[hit]
        da += d @ w
        dw[lo: lo + 16384] = d.t() @ a
    return [da, dw]


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "quantize":
        got = _exact_quantize(state["x"], case["fmt"], case["block"]) if case["out"] != "cols" else []
        return got + (_exact_quantize(state["x"].t(), case["fmt"], case["block"]) if case["out"] != "rows" else [])
    return {"product": _exact_product, "loss": _exact_loss, "gradient": _exact_gradient}[case["op"]](state)
