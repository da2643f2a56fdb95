"""Plain 64-bit forms of the training-side operators, and the error bounds
their tests use.

Every bound is worst case and follows from the arithmetic the header states:
results are rounded once to their type (``HALF_STEP`` = 2^-p for p significant bits),
sums are held in fp32, where n additions of terms t err by at most
n * 2^-23 * sum|t| (2^-23 and not 2^-24: a tensor core may cut instead of
rounding)."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24,
             torch.float8_e4m3fn: 2.0 ** -4}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
EPS32 = 2.0 ** -23
BLOCK = 128


def assert_within(got, ref, bound, what):
    """|got - ref| <= half a step of got's type at ref + bound, everywhere; NaN exactly where ref is NaN."""
    g, r = got.double(), ref.double()
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{what}: NaN in other places"
    lim = HALF_STEP[got.dtype] * (r.abs() + bound) + TINY[got.dtype] + bound
    bad = ((g - r).abs() > lim) & ~torch.isnan(r)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {i}: {float(g[i])} for "
                             f"{float(r[i])}, bound {float(lim[i])}")


def strided(t, pad=0, fill=float("nan"), whole=1):
    """A copy of t whose rows lie in a wider buffer (row length rounded up to `whole`, plus pad), the rest filled."""
    n = t.shape[-1]
    ld = -(-n // whole) * whole + pad
    if t.dtype == torch.float8_e4m3fn:
        buf = torch.full((*t.shape[:-1], ld), 0x7F, dtype=torch.uint8, device=t.device).view(t.dtype)
    else:
        buf = torch.full((*t.shape[:-1], ld), fill, dtype=t.dtype, device=t.device)
    buf[..., :n].copy_(t)
    return buf[..., :n], buf


# ---- layer norm ---------------------------------------------------------------
def norm_fwd(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    rstd = 1 / torch.sqrt((x - mean[:, None]).pow(2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean, rstd


def norm_bwd(dy, x, gamma, mean, rstd):
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x - mean) * rstd
    t = dy if gamma is None else dy * gamma.double()
    dx = rstd * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# ---- 128-block quantisers ---------------------------------------------------------
def e4m3_grid(device="cpu"):
    """Every finite E4M3 value by its byte, and NaN at 0x7f and 0xff."""
    v = []
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        a = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v.append(math.nan if (e, m) == (15, 7) else -a if s else a)
    return torch.tensor(v, dtype=torch.float64, device=device)


def decode(q):
    return e4m3_grid(q.device)[q.view(torch.uint8).long()]


def scale_of(amax):
    """The fp32 scale of blocks whose largest finite magnitude is amax (fp32)."""
    return torch.clamp_min(amax.float() * torch.tensor(1 / 448, dtype=torch.float32), 2.0 ** -126)


def finite_mag(v):
    return torch.where(torch.isfinite(v), v.abs(), torch.zeros_like(v))


def row_scales(v):
    R, C = v.shape
    nb = -(-C // BLOCK)
    p = torch.zeros(R, nb * BLOCK, device=v.device)
    p[:, :C] = finite_mag(v.float())
    return scale_of(p.view(R, nb, BLOCK).amax(2))


def assert_codes(q, v, s, what):
    """q is the E4M3 value nearest to v / s (v fp32; s its elements' scales), up to the fp32 rounding of the quotient."""
    t = v.double() / s.double()
    got = decode(q)
    bad = ~torch.isfinite(v)
    assert torch.equal(torch.isnan(got), bad), f"{what}: NaN codes in other places"
    t, got = t[~bad], got[~bad]
    step = torch.exp2(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -6))).clamp_min(-6) - 3)
    err = (got - t).abs()
    # fl(1/s), the product: 2 roundings of 2^-24, and the next binade's step at its edge
    lim = 0.5 * step * (1 + 2.0 ** -20) + t.abs() * 2.0 ** -22
    assert bool((err <= lim).all()), f"{what}: {int((err > lim).sum())} codes are not the nearest"


# ---- products -----------------------------------------------------------------------
def grouped(x, w, off):
    """(out, sum of |terms|) in 64 bits; w [G, N, K]; rows outside the groups are zero."""
    R, N = x.shape[0], w.shape[1]
    out = torch.zeros(R, N, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e in range(w.shape[0]):
        r = slice(off[e], off[e + 1])
        if off[e + 1] > off[e]:
            a, b = x[r].double(), w[e].double().t()
            out[r] = a @ b
            mag[r] = a.abs() @ b.abs()
    return out, mag


def grouped_wgrad(dy, x, off):
    G = len(off) - 1
    out = torch.zeros(G, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    for e in range(G):
        r = slice(off[e], off[e + 1])
        out[e] = dy[r].double().t() @ x[r].double()
        mag[e] = dy[r].double().abs().t() @ x[r].double().abs()
    return out, mag


# ---- activation -----------------------------------------------------------------------
def activation(h, act, alpha, limit):
    """h: list of halves (64 bits) -> (act, derivatives by each half)."""
    g = h[0]
    if act == "srelu":
        r = torch.where(g <= 0, torch.zeros_like(g), g)
        return r * r, [2 * r]
    u = h[1]
    if act == "geglu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2))
        pdf = torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        return g * c * u, [(c + g * pdf) * u, g * c]
    if act == "swiglu":
        s = torch.sigmoid(g)
        return g * s * u, [(s + g * s * (1 - s)) * u, g * s]
    gc, uc = g.clamp(-limit, limit), u.clamp(-limit, limit)
    s = torch.sigmoid(alpha * gc)
    dg = (s + alpha * gc * s * (1 - s)) * uc
    return gc * s * uc, [torch.where(g.abs() > limit, torch.zeros_like(g), dg),
                         torch.where(u.abs() > limit, torch.zeros_like(u), gc * s)]
