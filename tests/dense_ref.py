"""Plain 64-bit forms of the dense product with an epilogue and of the layer for
a few tokens, each with a bound of the kernels' error (see ops_ref.py: results
rounded once, fp32 sums of n terms off by n 2^-23 sum|t| at most).

The activations' bounds: CUDA documents the fast exponential as off by
2 + 1.173 |v| units in the last place and erfc by 4 (their argument's rounding
changes erfc by v^2 2^-24 relative); 8 more units cover the divisions, products
and additions around them."""
import math

import torch

from ops_ref import EPS32, HALF_STEP, TINY

GATED = ("swiglu", "swiglu_clamp", "geglu")
ACTS = ("none", "gelu", "silu", "srelu") + GATED


def halves(act):
    return 2 if act in GATED else 1


def _sigmoid(v):
    return 1 / (1 + torch.exp(-v)), (12 + 1.2 * v.abs()) * EPS32


def _cdf(v):
    return 0.5 * torch.erfc(-v / math.sqrt(2)), (12 + v * v) * EPS32


def _one(v, kind):
    """f(v) = v s(v), f'(v), relative error of f, absolute error of f'."""
    if kind == "cdf":
        s, rel = _cdf(v)
        ds = torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    else:
        s, rel = _sigmoid(v)
        ds = s * (1 - s)
    return v * s, s + v * ds, rel, 2 * rel * (s + (v * ds).abs())


def act(zs, name, alpha=1.0, limit=0.0):
    """zs: list of 64-bit halves -> value, its error, derivatives by half, their errors, and bounds of the derivatives'
    magnitude (the value moves by at most that times a small shift of the half)."""
    g = zs[0]
    if name == "none":
        one = torch.ones_like(g)
        return g, g * 0, [one], [one * 0], [one]
    if name == "srelu":
        r = torch.where(g <= 0, torch.zeros_like(g), g)
        return r * r, 2 * EPS32 * r * r, [2 * r], [2 * EPS32 * r], [2 * g.abs() + 1e-3]
    if name in ("gelu", "silu"):
        f, d, rel, ed = _one(g, "cdf" if name == "gelu" else "sigmoid")
        return f, rel * f.abs(), [d], [ed], [torch.full_like(g, 1.2)]
    u = zs[1]
    if name == "swiglu_clamp":
        gc, uc = g.clamp(-limit, limit), u.clamp(-limit, limit)
        f, d, rel, ed = _one(alpha * gc, "sigmoid")
        f = f / alpha
        inside_g, inside_u = (~(g.abs() > limit)).double(), (~(u.abs() > limit)).double()
    else:
        gc, uc, inside_g, inside_u = g, u, 1.0, 1.0
        f, d, rel, ed = _one(g, "cdf" if name == "geglu" else "sigmoid")
    val = f * uc
    grads = [inside_g * d * uc, inside_u * f]
    errs = [(ed + 4 * EPS32 * d.abs()) * uc.abs(), rel * f.abs()]
    return val, (rel + 4 * EPS32) * val.abs(), grads, errs, [1.2 * uc.abs() + 1e-3, f.abs() + 1e-3]


def product(x, w, bias):
    """z = x w^T + bias, and the bound of its fp32 sum."""
    a, b = x.double(), w.double()
    z, mag = a @ b.t(), a.abs() @ b.abs().t()
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    return z, (x.shape[1] + 8) * EPS32 * mag


def linear(x, w, bias, residual, name, alpha, limit):
    """out, its bound, z, its bound."""
    z, bz = product(x, w, bias)
    zs, bs = z.chunk(halves(name), 1), bz.chunk(halves(name), 1)
    val, err, _, _, lip = act(zs, name, alpha, limit)
    for b, m in zip(bs, lip):
        err = err + b * m
    if len(bs) == 2:
        err = err + 1.2 * bs[0] * bs[1]
    else:
        err = err + 2 * bs[0] * bs[0]
    if residual is not None:
        val = val + residual.double()
        err = err + 2 * EPS32 * val.abs()
    return val, err, z, bz


def linear_dz(dout, z, name, alpha, limit):
    """dz before its rounding, and the bound of its error."""
    d = dout.double()
    if name == "none":
        return d, d * 0
    zs = z.double().chunk(halves(name), 1)
    _, _, grads, errs, _ = act(zs, name, alpha, limit)
    dz = torch.cat([d * v for v in grads], 1)
    return dz, torch.cat([d.abs() * (e + 4 * EPS32 * v.abs()) for v, e in zip(grads, errs)], 1)


def rounded(bound, v, dtype):
    """The bound of v's error once v is rounded to dtype."""
    return bound + HALF_STEP[dtype] * (v.abs() + bound) + TINY[dtype]


def routing(logits, k, scale):
    """Ids (ties to the lower, NaN as -inf) and weights of 64-bit logits [T, E]."""
    v = torch.where(torch.isnan(logits), torch.full_like(logits, -math.inf), logits)
    s, ids = torch.sort(v, dim=1, descending=True, stable=True)
    top = s[:, :k]
    p = torch.exp(top - top[:, :1])
    w = p / p.sum(1, keepdim=True) * scale
    return ids[:, :k], torch.where(top[:, :1] == -math.inf, torch.zeros_like(w), w)


def layer(x, w1, w2, b1, ids, wts, n_shared, name, alpha, limit):
    """out [T, H] and its bound from given ids and weights (a slot whose id is out of range or whose weight is 0 is left
    out). y is a sum of two numbers of x's type, for more than 32 tokens rounded to one."""
    T, H = x.shape
    E, I = w1.shape[0] - n_shared, w2.shape[2]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err, mag = torch.zeros_like(out), torch.zeros_like(out)
    for e in range(E + n_shared):
        if e >= E:
            w = torch.ones(T, dtype=torch.float64, device=x.device)
        else:
            w = (wts.double() * (ids == e)).sum(1)
        t = (w != 0).nonzero()[:, 0]
        if not len(t):
            continue
        y, b, _, _ = linear(x[t], w1[e], None if b1 is None else b1[e], None, name, alpha, limit)
        y, b = y * w[t, None], (b + 4 * EPS32 * y.abs()) * w[t, None].abs()
        if T > 32:
            b = rounded(b, y, x.dtype)
        else:       # half a step of what half a step left, or of the smallest numbers
            f = torch.finfo(x.dtype)
            b = b + (f.eps / 2) ** 2 * (y.abs() + b) + f.smallest_normal * f.eps / 2
        m = w2[e].double()
        out[t] += y @ m.t()
        err[t] += b @ m.abs().t()
        mag[t] += y.abs() @ m.abs().t()
    return out, err + (I * (ids.shape[1] + n_shared) + 16) * EPS32 * (mag + err)
