"""Cases for the training-side operators of the routed-MoE block, and their plain forms.

Operators: layer norm (forward, backward), products grouped by expert with
ragged sizes (forward, gradient of the rows, gradient of the weights), the FP8
product with a scale for each block of 128 (forward with ready weights; a
training step that quantises weights, rows and gradients), and the gated
activation with an 8-bit checkpoint (forward, backward from the checkpoint).

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, with the library's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
BLOCK = 128
EPS = 1e-5


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # one token of a decode step, the norm in front of the router: latency
        {"name": "norm_fwd_decode", "op": "norm", "dir": "forward", "T": 1, "H": 7168, "dtype": "bf16", "wdtype": "bf16", "pad": 0},
        # fp32 activations of an odd width in rows of a wider buffer (an evaluation script)
        {"name": "norm_fwd_odd_f32", "op": "norm", "dir": "forward", "T": 3331, "H": 2881, "dtype": "f32", "wdtype": "f32", "pad": 7},
        # the training batch's backward with the reduction of the weight's gradient
        {"name": "norm_bwd_train", "op": "norm", "dir": "backward", "T": 16384, "H": 2880, "dtype": "bf16", "wdtype": "f32", "pad": 0},
        # W1 of one decoded token: eight rows, each with an expert of its own; streaming weights
        {"name": "grouped_fwd_decode", "op": "grouped", "dir": "forward", "R": 8, "G": 32, "N": 4096, "K": 7168, "empty": 0, "skew": 0.0, "dtype": "bf16"},
        # W1 of the training batch, forward: the largest call
        {"name": "grouped_fwd_train", "op": "grouped", "dir": "forward", "R": 65536, "G": 128, "N": 5760, "K": 2880, "empty": 0, "skew": 0.3, "dtype": "bf16"},
        # gradient of the rows through W2, ragged groups, some without rows, f16, odd sizes
        {"name": "grouped_dgrad_ragged", "op": "grouped", "dir": "dgrad", "R": 8191, "G": 40, "N": 1999, "K": 2880, "empty": 9, "skew": 0.6, "dtype": "f16"},
        # gradient of W2 of a training batch, ragged groups, some without rows
        {"name": "grouped_wgrad_train", "op": "grouped", "dir": "wgrad", "R": 30011, "G": 64, "N": 2880, "K": 2880, "empty": 5, "skew": 0.4, "dtype": "bf16"},
        # an FP8 projection of a few decoded tokens with weights quantised once: latency and weight streaming
        {"name": "fp8_fwd_decode", "op": "fp8", "dir": "forward", "R": 3, "G": 0, "N": 7168, "K": 2048, "empty": 0, "skew": 0.0, "dtype": "bf16"},
        # the experts' FP8 products of a prefill, ragged groups
        {"name": "fp8_fwd_grouped", "op": "fp8", "dir": "forward", "R": 12289, "G": 32, "N": 4096, "K": 7168, "empty": 3, "skew": 0.4, "dtype": "bf16"},
        # a training step of an FP8 projection: weights, rows and gradient quantised, y and dx
        {"name": "fp8_step_train", "op": "fp8", "dir": "step", "R": 8192, "G": 0, "N": 7168, "K": 4096, "empty": 0, "skew": 0.0, "dtype": "bf16"},
        # the experts' activation of the training batch, saving 8 bits
        {"name": "ckpt_fwd_train", "op": "ckpt", "dir": "forward", "R": 65536, "I": 2880, "act": "swiglu_clamp", "dtype": "bf16"},
        # its backward on a smaller batch of an odd width, from the 8-bit checkpoint
        {"name": "ckpt_bwd_odd", "op": "ckpt", "dir": "backward", "R": 16385, "I": 2047, "act": "swiglu", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "grouped", "fp8", "ckpt"])
    if op == "norm":
        H = _log(rng, 17, 16384)
        T = min(_log(rng, 1, 65536), 200_000_000 // H)
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        return {"op": op, "dir": rng.choice(["forward", "backward"]), "T": T, "H": H, "dtype": dtype,
                "wdtype": rng.choice(["f32", dtype]), "pad": rng.choice([0, 0, 8, 5])}
    if op == "ckpt":
        I = _log(rng, 33, 8192)
        R = min(_log(rng, 1, 65536), 180_000_000 // I)
        return {"op": op, "dir": rng.choice(["forward", "backward"]), "R": R, "I": I,
                "act": rng.choice(["swiglu", "swiglu_clamp", "geglu", "srelu"]), "dtype": rng.choice(["bf16", "bf16", "f16"])}
    K = _log(rng, 64, 7168)
    N = _log(rng, 64, 7168)
    if rng.random() < 0.5:  # model widths are multiples of 64 as a rule
        K, N = max(64, K // 64 * 64), max(64, N // 64 * 64)
    G = _log(rng, 1, 160)
    if op == "fp8" and rng.random() < 0.4:
        G = 0
    while G * N * K > 1_200_000_000:
        G = G * 3 // 4
    R = min(_log(rng, 1, 65536), int(8e11 / (N * K)))
    empty = rng.randint(0, G // 3) if G > 1 else 0
    case = {"op": op, "dir": None, "R": max(1, R), "G": G, "N": N, "K": K, "empty": empty,
            "skew": round(rng.uniform(0.0, 0.6), 2), "dtype": "bf16"}
    if op == "grouped":
        case["dir"] = rng.choice(["forward", "dgrad", "wgrad"])
        case["dtype"] = rng.choice(["bf16", "bf16", "f16"])
    else:
        case["dir"] = rng.choice(["forward", "step"])
    return case


# ---- inputs -----------------------------------------------------------------
def _sizes(case, seed):
    """Rows of each group: `empty` groups have none, the others at least one where the rows suffice."""
    R, G = case["R"], case["G"]
    r = random.Random(seed * 7919 + 13)
    live = sorted(r.sample(range(G), max(1, G - case["empty"])))
    if R <= len(live):
        live = sorted(r.sample(live, R))
    share = [math.exp(case["skew"] * r.gauss(0, 1)) for _ in live]
    total, acc, given = sum(share), 0.0, 0
    counts = [0] * G
    for g, s in zip(live, share):
        acc += s
        upto = round((R - len(live)) * acc / total)
        counts[g] = 1 + upto - given
        given = upto
    return counts


def _randn(gen, *shape, dtype=torch.bfloat16, std=1.0, step=8):
    """Normal values in rows whose stride is a multiple of `step` elements."""
    ld = -(-shape[-1] // step) * step
    t = torch.empty(*shape[:-1], ld, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)
    return t[..., : shape[-1]]


def _out(*shape, dtype, step=8):
    ld = -(-shape[-1] // step) * step
    return torch.zeros(*shape[:-1], ld, dtype=dtype, device="cuda")[..., : shape[-1]]


def _library():
    import quantized_grouped_gemm_topk_gb300 as m

    return m


def _quant(v):
    """E4M3 codes and fp32 scales of v [..., C] (fp32) in blocks of 128 along C."""
    C = v.shape[-1]
    nb = -(-C // BLOCK)
    p = torch.nn.functional.pad(v, (0, nb * BLOCK - C)).unflatten(-1, (nb, BLOCK))
    s = (p.abs().amax(-1) * (1.0 / 448.0)).clamp_min(2.0 ** -126)
    q = (p * (1.0 / s).unsqueeze(-1)).to(E4M3)
    return q.flatten(-2)[..., :C], s


def _quant_weights(w):
    """E4M3 codes and fp32 scales of w [G, N, K] (fp32) in blocks of 128 x 128."""
    G, N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    p = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(G, nb, BLOCK, kb, BLOCK)
    s = (p.abs().amax((2, 4)) * (1.0 / 448.0)).clamp_min(2.0 ** -126)
    q = (p * (1.0 / s)[:, :, None, :, None]).to(E4M3)
    return q.view(G, nb * BLOCK, kb * BLOCK)[:, :N, :K], s


def _rows16(q):
    """8-bit codes in rows whose stride is a multiple of 16 bytes."""
    out = _out(*q.shape, dtype=E4M3, step=16)
    out.copy_(q)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, d = case["op"], case["dir"]
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if op == "norm":
        T, H = case["T"], case["H"]
        wdt = DTYPES[case["wdtype"]]

        def rows(std):
            return _randn(gen, T, H + case["pad"], dtype=dt, std=std, step=1)[:, :H]

        st["x"] = rows(1.5)
        st["x"][:, :: max(1, H // 5)] *= 8  # the few loud channels that a residual stream has
        st["x"] += 0.25
        st["gamma"] = (1 + 0.2 * torch.randn(H, generator=gen, device="cuda")).to(wdt)
        st["beta"] = (0.1 * torch.randn(H, generator=gen, device="cuda")).to(wdt)
        if d == "forward":
            st["y"] = torch.empty(T, H, dtype=dt, device="cuda")
            st["mean"] = torch.empty(T, device="cuda")
            st["rstd"] = torch.empty(T, device="cuda")
        else:
            st["dy"] = rows(1.0)
            v = st["x"].float()
            st["mean"] = v.mean(1)
            st["rstd"] = (v.var(1, unbiased=False) + EPS).rsqrt()
            st["dx"] = torch.empty(T, H, dtype=dt, device="cuda")
            st["dgamma"], st["dbeta"] = torch.empty_like(st["gamma"]), torch.empty_like(st["beta"])
            # a plain count of bytes: two fp32 rows for each partial sum of the weight's gradient
            st["ws"] = torch.zeros(256 + 2 * 4 * H * 1024, dtype=torch.uint8, device="cuda")
        return st
    if op == "ckpt":
        R, I = case["R"], case["I"]
        halves = 1 if case["act"] == "srelu" else 2
        st["w"] = torch.rand(R, generator=gen, device="cuda") * 0.5 + 0.05
        nb = halves * -(-I // BLOCK)
        h = torch.randn(R, halves * I, generator=gen, device="cuda", dtype=dt) * 2
        st["y"] = torch.empty(R, I, dtype=dt, device="cuda")
        if d == "forward":
            st["h"] = h
            st["q"] = torch.empty(R, halves * I, dtype=E4M3, device="cuda")
            st["s"] = torch.empty(R, nb, device="cuda")
        else:
            q, s = _quant(h.view(R, halves, I).float())
            st["q"], st["s"] = q.reshape(R, halves * I).contiguous(), s.reshape(R, nb)
            st["dy"] = torch.randn(R, I, generator=gen, device="cuda", dtype=dt)
            st["dh"] = torch.empty(R, halves * I, dtype=dt, device="cuda")
            st["dw"] = torch.empty(R, device="cuda")
        return st
    R, G, N, K = case["R"], case["G"], case["N"], case["K"]
    groups = max(G, 1)
    if G:
        counts = _sizes(case, seed)
        off = [0]
        for c in counts:
            off.append(off[-1] + c)
        st["offsets"] = torch.tensor(off, dtype=torch.int32).cuda()
        st["cap"] = max(counts)
    # room for the status word and for fp32 partial sums of a product split along its sum
    st["ws"] = torch.zeros(256 + 64 * 1024 * 1024, dtype=torch.uint8, device="cuda")
    if op == "grouped":
        std = 0.02
        if d == "forward":
            st["x"], st["w"] = _randn(gen, R, K, dtype=dt), _randn(gen, G, N, K, dtype=dt, std=std)
            st["out"] = _out(R, N, dtype=dt)
        elif d == "dgrad":
            st["dy"], st["w"] = _randn(gen, R, N, dtype=dt), _randn(gen, G, N, K, dtype=dt, std=std)
            st["out"] = _out(R, K, dtype=dt)
        else:
            st["dy"], st["x"] = _randn(gen, R, N, dtype=dt, std=0.1), _randn(gen, R, K, dtype=dt)
            st["out"] = _out(G, N, K, dtype=dt)
        return st
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    st["x"] = _randn(gen, R, K, dtype=dt)
    st["xq"], st["xs"] = _out(R, K, dtype=E4M3, step=16), torch.zeros(R, kb, device="cuda")
    st["out"] = _out(R, N, dtype=dt)
    w = _randn(gen, groups, N, K, dtype=dt, std=0.02)
    if d == "forward":
        st["wq"] = _out(groups, N, K, dtype=E4M3, step=16)
        st["wscale"] = torch.zeros(groups, nb, kb, device="cuda")
        for g in range(groups):
            q, s = _quant_weights(w[g : g + 1].float())
            st["wq"][g], st["wscale"][g] = q[0], s[0]
        return st
    st["w"] = w
    st["dy"] = _randn(gen, R, N, dtype=dt)
    st["wq"], st["wscale"] = _out(groups, N, K, dtype=E4M3, step=16), torch.zeros(groups, nb, kb, device="cuda")
    st["wtq"], st["wtscale"] = _out(groups, K, N, dtype=E4M3, step=16), torch.zeros(groups, kb, nb, device="cuda")
    st["dyq"], st["dys"] = _out(R, N, dtype=E4M3, step=16), torch.zeros(R, nb, device="cuda")
    st["dx"] = _out(R, K, dtype=dt)
    return st


# ---- the library's calls ------------------------------------------------------
def _run_own(st):
    m = _library()
    case = st["case"]
    op, d = case["op"], case["dir"]
    if op == "norm":
        if d == "forward":
            m.moe_layer_norm_forward(st["x"], st["gamma"], st["beta"], EPS, st["y"], st["mean"], st["rstd"])
            return {"y": st["y"], "mean": st["mean"], "rstd": st["rstd"]}
        m.moe_layer_norm_backward(st["dy"], st["x"], st["gamma"], st["mean"], st["rstd"], st["dx"], st["dgamma"], st["dbeta"], st["ws"])
        return {"dx": st["dx"], "dgamma": st["dgamma"], "dbeta": st["dbeta"]}
    if op == "ckpt":
        act = {"act": case["act"], "alpha": 1.702, "limit": 7.0}
        if d == "forward":
            m.moe_act_ckpt_forward(st["h"], st["w"], st["y"], st["q"], st["s"], **act)
            return {"y": st["y"], "q": st["q"], "s": st["s"]}
        m.moe_act_ckpt_backward(st["dy"], st["q"], st["s"], st["w"], st["dh"], st["dw"], st["y"], **act)
        return {"dh": st["dh"], "dw": st["dw"], "y": st["y"]}
    if op == "grouped":
        if d == "forward":
            m.moe_grouped_mm(st["x"], st["w"], st["offsets"], st["out"], st["ws"])
        elif d == "dgrad":
            m.moe_grouped_mm(st["dy"], st["w"], st["offsets"], st["out"], st["ws"], trans_w=True)
        else:
            m.moe_grouped_mm_wgrad(st["dy"], st["x"], st["offsets"], st["out"], st["ws"])
        return {"out": st["out"]}
    off = st.get("offsets")
    if d == "step":
        m.moe_fp8_quant_weights(st["w"], st["wq"], st["wscale"], st["wtq"], st["wtscale"])
    m.moe_fp8_quant_rows(st["x"], st["xq"], st["xs"])
    m.moe_fp8_mm(st["xq"], st["xs"], st["wq"], st["wscale"], st["out"], st["ws"], offsets=off)
    if d == "forward":
        return {"out": st["out"]}
    m.moe_fp8_quant_rows(st["dy"], st["dyq"], st["dys"])
    m.moe_fp8_mm(st["dyq"], st["dys"], st["wtq"], st["wtscale"], st["dx"], st["ws"], offsets=off)
    return {"out": st["out"], "dx": st["dx"]}


# ---- the plain forms ------------------------------------------------------------
def _cdf(g):
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))


def _activation(h, act):
    """act(h) of h [R, halves, I]; also its derivatives by each half."""
    g = h[:, 0]
    if act == "srelu":
        r = g.clamp_min(0)
        return r * r, (2 * r,)
    u = h[:, 1]
    if act == "swiglu":
        s = torch.sigmoid(g)
        return g * s * u, ((s + g * s * (1 - s)) * u, g * s)
    if act == "geglu":
        c = _cdf(g)
        return g * c * u, ((c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)) * u, g * c)
    alpha, lim = 1.702, 7.0
    gc, uc = g.clamp(-lim, lim), u.clamp(-lim, lim)
    s = torch.sigmoid(alpha * gc)
    dg = torch.where(g.abs() <= lim, (s + alpha * gc * s * (1 - s)) * uc, torch.zeros_like(g))
    du = torch.where(u.abs() <= lim, gc * s, torch.zeros_like(u))
    return gc * s * uc, (dg, du)


def _places(st):
    """Each row's group, and its place in the group."""
    off = st["offsets"].long()
    r = torch.arange(st["case"]["R"], device="cuda")
    g = torch.searchsorted(off[1:], r, right=True)
    return g, r - off[g]


def _padded(v, g, p, G, cap):
    out = torch.zeros(G, cap, v.shape[1], device="cuda")
    out[g, p] = v
    return out


def _grouped_product(st, x, w):
    """x [R, K] times w [G, N, K] of each row's group, in fp32."""
    R, G = x.shape[0], w.shape[0]
    if "offsets" not in st:
        return x @ w[0].t()
    g, p = _places(st)
    if R <= G // 2:
        return torch.bmm(w[g], x.unsqueeze(2)).squeeze(2)
    return torch.bmm(_padded(x, g, p, G, st["cap"]), w.transpose(1, 2))[g, p]


def _expand(s, N, K):
    return s.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]


def _unquant_rows(q, s):
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def _run_plain(st):
    case = st["case"]
    op, d = case["op"], case["dir"]
    dt = DTYPES[case["dtype"]]
    if op == "norm":
        x, gamma = st["x"].float(), st["gamma"].float()
        if d == "forward":
            mean = x.mean(1)
            c = x - mean[:, None]
            rstd = 1 / torch.sqrt((c * c).mean(1) + EPS)
            y = c * rstd[:, None] * gamma + st["beta"].float()
            return {"y": y.to(dt), "mean": mean, "rstd": rstd}
        dy, r = st["dy"].float(), st["rstd"][:, None]
        xh = (x - st["mean"][:, None]) * r
        t = dy * gamma
        dx = r * (t - t.mean(1, keepdim=True) - xh * (t * xh).mean(1, keepdim=True))
        wdt = st["gamma"].dtype
        return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(0).to(wdt), "dbeta": dy.sum(0).to(wdt)}
    if op == "ckpt":
        R, I, w = case["R"], case["I"], st["w"][:, None]
        halves = 1 if case["act"] == "srelu" else 2
        if d == "forward":
            h = st["h"].view(R, halves, I).float()
            q, s = _quant(h)
            return {"y": (w * _activation(h, case["act"])[0]).to(dt), "q": q.reshape(R, halves * I), "s": s.reshape(R, -1)}
        s = st["s"].view(R, halves, -1).repeat_interleave(BLOCK, 2)[:, :, :I]
        a, grads = _activation(st["q"].view(R, halves, I).float() * s, case["act"])
        dy = st["dy"].float()
        dh = torch.stack([w * dy * g for g in grads], 1).view(R, halves * I)
        return {"dh": dh.to(dt), "dw": (dy * a).sum(1), "y": (w * a).to(dt)}
    if op == "grouped":
        if d == "forward":
            w = st["w"] if case["R"] <= case["G"] // 2 else st["w"].float()
            if w.dtype != torch.float32:  # few rows: only their experts are widened
                g, _ = _places(st)
                return {"out": torch.bmm(w[g].float(), st["x"].float().unsqueeze(2)).squeeze(2).to(dt)}
            return {"out": _grouped_product(st, st["x"].float(), w).to(dt)}
        if d == "dgrad":
            return {"out": _grouped_product(st, st["dy"].float(), st["w"].float().transpose(1, 2)).to(dt)}
        g, p = _places(st)
        a = _padded(st["dy"].float(), g, p, case["G"], st["cap"])
        b = _padded(st["x"].float(), g, p, case["G"], st["cap"])
        return {"out": torch.bmm(a.transpose(1, 2), b).to(dt)}
    N, K = case["N"], case["K"]
    q, s = (st["wq"], st["wscale"]) if d == "forward" else _quant_weights(st["w"].float())
    w = q.float() * _expand(s, N, K)
    out = _grouped_product(st, _unquant_rows(*_quant(st["x"].float())), w).to(dt)
    if d == "forward":
        return {"out": out}
    dx = _grouped_product(st, _unquant_rows(*_quant(st["dy"].float())), w.transpose(1, 2)).to(dt)
    return {"out": out, "dx": dx}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------
def work(case):
    op, d = case["op"], case["dir"]
    if op == "norm":
        n, e, we = case["T"] * case["H"], 4 if case["dtype"] == "f32" else 2, 4 if case["wdtype"] == "f32" else 2
        if d == "forward":
            return {"bytes": 2 * n * e + 2 * case["H"] * we + 8 * case["T"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 3 * case["H"] * we + 8 * case["T"], "flops": 14 * n}
    if op == "ckpt":
        n, R = case["R"] * case["I"], case["R"]
        halves = 1 if case["act"] == "srelu" else 2
        scales = 4 * R * halves * -(-case["I"] // BLOCK)
        if d == "forward":
            return {"bytes": n * (3 * halves + 2) + scales + 4 * R, "flops": 12 * n}
        return {"bytes": n * (halves + 2 + 2 * halves + 2) + scales + 8 * R, "flops": 24 * n}
    R, N, K, G = case["R"], case["N"], case["K"], max(1, case["G"])
    live = min(R, max(1, G - case["empty"]))
    flops = 2 * R * N * K
    if op == "grouped":
        if d == "wgrad":
            return {"bytes": 2 * R * (N + K) + 2 * G * N * K, "flops": flops}
        return {"bytes": 2 * R * (N + K) + 2 * live * N * K + 4 * (case["G"] + 1), "flops": flops}
    scales = 4 * live * -(-N // BLOCK) * -(-K // BLOCK)
    if d == "forward":
        return {"bytes": 2 * R * (K + N) + live * N * K + scales, "flops": flops}
    # the weights and both gradients' operands are read in 16 bits, and each group's weights, with rows or without, become 8 bits
    return {"bytes": 4 * R * (K + N) + 2 * G * N * K, "flops": 2 * flops}


# ---- the definition in 64 bits ---------------------------------------------------
def _code(v, r):
    """E4M3 nearest (ties to even) to v * r: three bits of mantissa, subnormals below 2^-6, at most 448."""
    t = v.double() * r.double()
    _, e = torch.frexp(t)
    ulp = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return torch.round(t / ulp).mul(ulp).clamp(-448.0, 448.0)


def _blocks(v):
    """v [R, C]: (each element's scale, each block's scale), the scales being the fp32 numbers of the format."""
    R, C = v.shape
    nb = -(-C // BLOCK)
    p = torch.zeros(R, nb * BLOCK, dtype=torch.float32, device=v.device)
    p[:, :C] = v
    s = torch.maximum(p.view(R, nb, BLOCK).abs().max(2).values * torch.tensor(1.0 / 448.0, device=v.device), torch.tensor(2.0 ** -126, device=v.device))
    return s[:, :, None].expand(R, nb, BLOCK).reshape(R, nb * BLOCK)[:, :C], s


def _dequant_rows64(v):
    e, _ = _blocks(v.float())
    return _code(v.float(), 1.0 / e) * e.double()


def _dequant_weights64(w):
    N, K = w.shape
    row, _ = _blocks(w.float())  # 1 x 128 scales, joined over 128 rows
    nb = -(-N // BLOCK)
    p = torch.zeros(nb * BLOCK, K, device=w.device)
    p[:N] = row
    e = p.view(nb, BLOCK, K).max(1).values.repeat_interleave(BLOCK, 0)[:N]
    return _code(w.float(), 1.0 / e) * e.double()


def exact(case, seed):
    st = prepare(case, seed)
    op, d = case["op"], case["dir"]
    if op == "norm":
        x, gamma, beta = st["x"].double(), st["gamma"].double(), st["beta"].double()
        if d == "forward":
            H = case["H"]
            mean = x.sum(1) / H
            var = (x - mean[:, None]).pow(2).sum(1) / H
            rstd = (var + EPS) ** -0.5
            return {"y": (x - mean[:, None]) * rstd[:, None] * gamma + beta, "mean": mean, "rstd": rstd}
        mean, rstd = st["mean"].double()[:, None], st["rstd"].double()[:, None]
        dy, H = st["dy"].double(), case["H"]
        xh = (x - mean) * rstd
        dxh = dy * gamma
        dx = (dxh - dxh.sum(1, keepdim=True) / H - xh * (dxh * xh).sum(1, keepdim=True) / H) * rstd
        return {"dx": dx, "dgamma": (dy * xh).sum(0), "dbeta": dy.sum(0)}
    if op == "ckpt":
        R, I, act = case["R"], case["I"], case["act"]
        halves = 1 if act == "srelu" else 2
        w = st["w"].double()[:, None]
        if d == "forward":
            cols = [st["h"][:, k * I : (k + 1) * I] for k in range(halves)]
            a, _ = _activation64([c.double() for c in cols], act)
            es, ss = zip(*[_blocks(c.float()) for c in cols])
            q = torch.cat([_code(c.float(), 1.0 / e) for c, e in zip(cols, es)], 1)
            return {"y": w * a, "q": q, "s": torch.cat(ss, 1).double()}
        nb = -(-I // BLOCK)
        at = torch.arange(I, device="cuda") // BLOCK
        hs = [st["q"][:, k * I : (k + 1) * I].double() * st["s"][:, k * nb + at].double() for k in range(halves)]
        a, grads = _activation64(hs, act)
        dy = st["dy"].double()
        return {"dh": torch.cat([g * dy * w for g in grads], 1), "dw": (dy * a).sum(1), "y": w * a}
    R, G, N, K = case["R"], max(1, case["G"]), case["N"], case["K"]
    off = st["offsets"].tolist() if case["G"] else [0, R]
    spans = [(g, slice(off[g], off[g + 1])) for g in range(G) if off[g + 1] > off[g]]
    if op == "grouped":
        if d == "wgrad":
            out = torch.zeros(G, N, K, dtype=torch.float64, device="cuda")
            for g, s in spans:
                out[g] = st["dy"][s].double().t() @ st["x"][s].double()
            return {"out": out}
        rows = st["x"] if d == "forward" else st["dy"]
        out = torch.zeros(R, N if d == "forward" else K, dtype=torch.float64, device="cuda")
        for g, s in spans:
            w = st["w"][g].double()
            out[s] = rows[s].double() @ (w.t() if d == "forward" else w)
        return {"out": out}
    x = _dequant_rows64(st["x"])
    out = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    dx = torch.zeros(R, K, dtype=torch.float64, device="cuda")
    dy = _dequant_rows64(st["dy"]) if d == "step" else None
    n_at, k_at = torch.arange(N, device="cuda") // BLOCK, torch.arange(K, device="cuda") // BLOCK
    for g, s in spans:
        if d == "forward":
            w = st["wq"][g].double() * st["wscale"][g].double()[n_at][:, k_at]
        else:
            w = _dequant_weights64(st["w"][g])
        out[s] = x[s] @ w.t()
        if d == "step":
            dx[s] = dy[s] @ w
    return {"out": out} if d == "forward" else {"out": out, "dx": dx}


def _activation64(h, act):
    """The activation and its derivatives by the formulas, on 64-bit halves."""
    if act == "srelu":
        pos = (h[0] > 0).double()
        return pos * h[0] ** 2, [2 * pos * h[0]]
    g, u = h
    if act == "geglu":
        phi = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        return g * phi * u, [u * (phi + g * torch.exp(-(g ** 2) / 2) / math.sqrt(2 * math.pi)), g * phi]
    if act == "swiglu":
        s = 1 / (1 + torch.exp(-g))
        return g * u * s, [u * s * (1 + g * (1 - s)), g * s]
    a, lim = 1.702, 7.0
    gin, uin = (g >= -lim) & (g <= lim), (u >= -lim) & (u <= lim)
    gc, uc = torch.minimum(torch.maximum(g, -torch.full_like(g, lim)), torch.full_like(g, lim)), u.clip(-lim, lim)
    s = 1 / (1 + torch.exp(-a * gc))
    return gc * uc * s, [gin.double() * uc * s * (1 + a * gc * (1 - s)), uin.double() * gc * s]
