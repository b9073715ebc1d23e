"""The feed-forward block's operators and layer norm in 64 bits, with bounds on
what 32-bit sums and the results' rounding may be off (shared by the GPU tests)."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}      # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # half a subnormal step


def act(name, x):
    """An activation and its derivative at 64-bit x."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "relu":
        return torch.where(x < 0, torch.zeros_like(x), x), (x > 0).double()
    if name == "gelu":
        share = 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
        return x * share, share + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if name == "silu":
        share, inner = torch.sigmoid(x), torch.ones_like(x)
    else:
        c = math.sqrt(8 / math.pi)
        share, inner = torch.sigmoid(c * (x + 0.044715 * x ** 3)), c * (1 + 3 * 0.044715 * x * x)
    return x * share, share + x * share * (1 - share) * inner


def act_error(name, x):
    """Relative error of an activation's 32-bit value: the exponent's argument t
    is rounded (|t| 2^-22 in the exponential), a few operations of 2^-23 each;
    |t| < 8 + 2 x^2 until the activation is 0 or x in 32 bits."""
    return torch.zeros_like(x) if name in ("none", "relu") else (16 + 2 * x * x).clamp(max=256) * 2.0 ** -22


def slope_error(name, x):
    """Absolute error of its 32-bit derivative: terms of at most 1 + |x| each off as above."""
    return torch.zeros_like(x) if name in ("none", "relu") else (16 + 2 * x * x).clamp(max=256) * 2.0 ** -22 * (1 + x.abs()).clamp(max=16)


def pre(a, w, bias):
    """p and the error its 32-bit sum may have: k + 1 additions, each off by a
    step of 2^-24 of a partial sum of at most the sum of sizes (the matrix
    cores' additions are not all rounded to nearest: twice that)."""
    a, w = a.double(), w.double()
    p, size = a @ w.t(), a.abs() @ w.abs().t()
    if bias is not None:
        p, size = p + bias.double(), size + bias.double().abs()
    return p, size * ((a.shape[1] + 2) * 2.0 ** -23)


def forward(name, gated, a, w, bias, residual, dtype):
    """y, its bound, p and p's error."""
    p, e = pre(a, w, bias)
    n = p.shape[1] // (2 if gated else 1)
    g, eg = p[:, :n], e[:, :n]
    v, slope = act(name, g)
    # the slope between g - eg and g + eg: at most 1.13 + what the kink of relu adds
    y, off = v, 1.2 * eg + act_error(name, g) * v.abs()
    if gated:
        u, eu = p[:, n:], e[:, n:]
        y, off = v * u, off * u.abs() + v.abs() * eu + off * eu
    if residual is not None:
        y = y + residual.double()
    off = off + 2.0 ** -22 * y.abs()
    return y, off * (1 + EPS[dtype]) + EPS[dtype] * y.abs() + TINY[dtype], p, e


def scales_of(p, n, parts):
    """Powers of two of the 8-bit form for p [m, parts * n], exactly, and the blocks' largest sizes."""
    m = p.shape[0]
    x = p.view(m, parts, n).abs()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    x = torch.nn.functional.pad(x, (0, -n % 32)).view(m, parts, -1, 32).amax(3)
    f, e = torch.frexp(x)                                  # 448 = 0.875 * 2^9
    code = torch.where(x > 0, e - 9 + (f > 0.875), torch.full_like(e, -126)).clamp(min=-126)
    return ((code.long() + 1023) << 52).view(torch.float64), x


def gradient(name, gated, p, dy, a, w, dtype):
    """d, dA, dW, dbias and bounds of the last three; p is what was kept."""
    p, dy, a, w = p.double(), dy.double(), a.double(), w.double()
    n = dy.shape[1]
    g = p[:, :n]
    v, slope = act(name, g)
    if gated:
        u = p[:, n:]
        d = torch.cat([dy * u * slope, dy * v], 1)
        raw = torch.cat([(dy * u).abs() * slope_error(name, g), (dy * v).abs() * act_error(name, g)], 1) + 2.0 ** -22 * d.abs()
    else:
        d = dy * slope
        raw = dy.abs() * slope_error(name, g) + 2.0 ** -22 * d.abs()
    off = raw + EPS[dtype] * d.abs() + TINY[dtype]         # d as an operand of the products
    da, dw, db = d @ w, d.t() @ a, d.sum(0)
    step = EPS[dtype]

    def bound(error, size, terms, result):
        total = error + size * ((terms + 2) * 2.0 ** -23)
        return total * (1 + step) + step * result.abs() + TINY[dtype]

    big = d.abs() + off
    return (d, (da, bound(off @ w.abs(), big @ w.abs(), d.shape[1], da)),
            (dw, bound(off.t() @ a.abs(), big.t() @ a.abs(), d.shape[0], dw)),
            (db, bound(raw.sum(0), d.abs().sum(0), d.shape[0], db)))


def norm(x, weight, bias, eps, dtype):
    """(y, bound), (mean, bound), (rstd, bound).  A lane adds at most 32 values and
    the lanes' sums are added in a tree of at most 26 levels: 64 steps of 2^-24."""
    x = x.double()
    cols = x.shape[1]
    w = torch.ones(cols, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    b = torch.zeros(cols, dtype=torch.float64, device=x.device) if bias is None else bias.double()
    terms = 64 + cols / 1024 / 4
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    near = 2.0 ** -22 * x.abs().amax(1, keepdim=True)      # differences of 32-bit numbers of this size
    h = (x - mean) * rstd
    y = h * w + b
    rel = terms * 2.0 ** -23 + 2 * near * rstd             # of rstd
    off = (near * rstd + h.abs() * rel) * w.abs() + 2.0 ** -22 * ((h * w).abs() + b.abs())
    return ((y, off + EPS[dtype] * y.abs() + TINY[dtype]), (mean[:, 0], near[:, 0]), (rstd[:, 0], (rstd * rel)[:, 0]))


def norm_gradient(x, dy, weight, mean, rstd, dtype, wtype):
    """(dx, bound), (dweight, bound), (dbias, bound) from 32-bit mean and rstd."""
    x, dy, mean, rstd = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    rows, cols = x.shape
    w = torch.ones(cols, dtype=torch.float64, device=x.device) if weight is None else weight.double()
    h, g = (x - mean) * rstd, dy * w
    terms = (64 + cols / 1024 / 4) * 2.0 ** -23
    a, b = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    dx = rstd * (g - a - h * b)
    ea, eb = terms * g.abs().mean(1, keepdim=True), terms * (g * h).abs().mean(1, keepdim=True)
    off = rstd * (ea + h.abs() * eb + 2.0 ** -21 * (g.abs() + a.abs() + (h * b).abs()))
    dw, db = (dy * h).sum(0), dy.sum(0)
    more = (rows + 4) * 2.0 ** -23                         # additions over rows, in whatever groups
    return ((dx, off + EPS[dtype] * dx.abs() + TINY[dtype]),
            (dw, more * (dy * h).abs().sum(0) * (1 + EPS[wtype]) + EPS[wtype] * dw.abs() + TINY[wtype]),
            (db, more * dy.abs().sum(0) * (1 + EPS[wtype]) + EPS[wtype] * db.abs() + TINY[wtype]))


def check(got, want, bound, what):
    got = got.double().to(want.device)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    over = torch.where(nan, torch.zeros_like(want), (got - want).abs() - bound)
    worst = over.argmax()
    assert (over <= 0).all(), (f"{what}: {int((over > 0).sum())} of {over.numel()} beyond their bounds, worst at "
                               f"{int(worst)}: {got.flatten()[worst].item()} for {want.flatten()[worst].item()} "
                               f"+- {bound.flatten()[worst].item()}")
