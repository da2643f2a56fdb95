"""Cases for the serving and dense operators next to the routed layer, and their plain forms.

Operators: the whole Mixture-of-Experts layer with 16-bit experts for a few
tokens (router, top-k, both products, combine), and the dense product with
bias, activation and residual in its epilogue (forward, and the backward from
its saved pre-activation).

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, with the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ALPHA, LIMIT = 1.702, 7.0
GATED = ("swiglu", "swiglu_clamp", "geglu")


# ---- cases ------------------------------------------------------------------
def _layer(name, T, H, I, E, k, shared, act, dtype, bias, scale, pad):
    return {"name": name, "op": "layer", "T": T, "H": H, "I": I, "E": E, "k": k, "shared": shared, "act": act,
            "dtype": dtype, "bias": bias, "scale": scale, "pad": pad}


def _linear(name, d, R, N, K, act, dtype, wdtype, bias, residual, save, pad):
    """N: output columns; a gated activation's weights have 2 N rows. wdtype: of the bias and its gradient."""
    return {"name": name, "op": "linear", "dir": d, "R": R, "N": N, "K": K, "act": act, "dtype": dtype, "wdtype": wdtype,
            "bias": bias, "residual": residual, "save": save, "pad": pad}


def listed():
    return [
        # one token through a small layer: the launches and the waits between the steps
        _layer("layer_small_1", 1, 256, 128, 8, 2, 0, "swiglu", "bf16", False, 1.0, 0),
        # one decoded token of a large layer: eight experts' weights stream through once
        _layer("layer_decode_1", 1, 7168, 2048, 256, 8, 0, "swiglu", "bf16", False, 1.0, 0),
        # a decode batch with an always-on shared expert and scaled routing weights
        _layer("layer_shared_16", 16, 6144, 1536, 160, 8, 1, "swiglu", "bf16", False, 2.5, 0),
        # the largest batch of the call, nearly every expert touched, biased clamped activation, as a trained block is served
        _layer("layer_batch_64", 64, 2880, 2880, 128, 4, 0, "swiglu_clamp", "f16", True, 1.0, 0),
        # odd widths in rows of a wider buffer, few experts, a batch of five
        _layer("layer_odd_5", 5, 1999, 1001, 24, 3, 1, "geglu", "f16", True, 1.0, 8),
        # a projection of one decoded token that adds to the residual stream: latency
        _linear("linear_decode_1", "forward", 1, 7168, 2048, "none", "bf16", "bf16", False, True, False, 0),
        # a shared expert's first product for a decode batch, gate and up in one call
        _linear("linear_gated_16", "forward", 16, 2048, 7168, "swiglu", "bf16", "f32", True, False, False, 0),
        # an odd width and a ragged batch, f16, with everything in the epilogue
        _linear("linear_odd_333", "forward", 333, 2881, 1999, "gelu", "f16", "f16", True, True, True, 3),
        # the training batch's gated first product, saving what the backward needs
        _linear("linear_gated_train", "forward", 16384, 2880, 2880, "swiglu_clamp", "bf16", "f32", True, False, True, 0),
        # a prefill's projection into the residual stream: the largest forward
        _linear("linear_residual_prefill", "forward", 16384, 7168, 4096, "none", "bf16", "bf16", True, True, False, 0),
        # the backward of the training batch's gated product: the largest call
        _linear("linear_bwd_train", "backward", 16384, 2880, 2880, "swiglu_clamp", "bf16", "f32", True, False, True, 0),
        # a small ragged batch's backward at odd widths
        _linear("linear_bwd_odd", "backward", 1003, 1441, 1999, "gelu", "f16", "f16", True, False, True, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Model widths are multiples of 64 as a rule."""
    v = _log(rng, lo, hi)
    return max(lo, v // 64 * 64) if rng.random() < 0.6 else v


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if rng.random() < 0.45:
        T, k = _log(rng, 1, 64), rng.randint(1, 8)
        H, I = _width(rng, 64, 7168), _width(rng, 64, 2880)
        E = max(k, _log(rng, 4, 256))
        shared = rng.choice([0, 0, 1])
        # the touched weights stay below the largest listed batch's
        while 3 * H * I * min(E, T * k) > 2_700_000_000 or 3 * H * I * E > 11_000_000_000:
            H, I = max(64, H * 7 // 8), max(64, I * 7 // 8)
        act = rng.choice(["swiglu", "swiglu_clamp", "geglu", "srelu"])
        case = _layer("", T, H, I, E, k, shared, act, dtype, act != "srelu" and rng.random() < 0.4, rng.choice([1.0, 2.5]),
                      rng.choice([0, 0, 8]))
        del case["name"]
        return case
    d = rng.choice(["forward", "forward", "backward"])
    act = rng.choice(["none", "gelu", "silu", "srelu", "swiglu", "swiglu_clamp", "geglu"])
    K, N = _width(rng, 64, 7168), _width(rng, 64, 7168)
    halves = 2 if act in GATED else 1
    R = max(1, min(_log(rng, 1, 16384), 270_000_000_000 // (N * K * halves)))
    case = _linear("", d, R, N, K, act, dtype, rng.choice(["f32", dtype]), rng.random() < 0.5, rng.random() < 0.5,
                   rng.random() < 0.5, rng.choice([0, 0, 3, 8]))
    del case["name"]
    return case


# ---- inputs -----------------------------------------------------------------
def _randn(gen, *shape, dtype, std=1.0, pad=0, step=8):
    """Normal values in rows whose stride is a multiple of `step` elements, pad more."""
    ld = -(-(shape[-1] + pad) // step) * step
    t = torch.empty(*shape[:-1], ld, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)
    return t[..., : shape[-1]]


def _out(*shape, dtype, pad=0, step=8):
    ld = -(-(shape[-1] + pad) // step) * step
    return torch.zeros(*shape[:-1], ld, dtype=dtype, device="cuda")[..., : shape[-1]]


def _library():
    import quantized_grouped_gemm_topk_gb300 as m

    return m


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "layer":
        T, H, I, E, k, pad = case["T"], case["H"], case["I"], case["E"], case["k"], case["pad"]
        G = E + case["shared"]
        halves = 2 if case["act"] in GATED else 1
        st["x"] = _randn(gen, T, H, dtype=dt, pad=pad)
        st["W_r"] = torch.randn(H, E, generator=gen, device="cuda") * H ** -0.5
        st["w1"] = _randn(gen, G, halves * I, H, dtype=dt, std=H ** -0.5, pad=pad)
        st["w2"] = _randn(gen, G, H, I, dtype=dt, std=I ** -0.5, pad=pad)
        st["b1"] = torch.randn(G, 2 * I, generator=gen, device="cuda") * 0.1 if case["bias"] else None
        st["out"] = _out(T, H, dtype=dt, pad=pad)
        st["ids"] = torch.zeros(T, k, dtype=torch.int32, device="cuda")
        st["wts"] = torch.zeros(T, k, device="cuda")
        # a plain count of bytes: the hidden rows and their products, the router's and the split products' partial sums
        st["ws"] = torch.zeros((96 << 20) + 8 * T * (k + 1) * (H + I), dtype=torch.uint8, device="cuda")
        return st
    R, N, K, pad = case["R"], case["N"], case["K"], case["pad"]
    act, wdt = case["act"], DTYPES[case["wdtype"]]
    rows = 2 * N if act in GATED else N
    st["x"], st["w"] = _randn(gen, R, K, dtype=dt), _randn(gen, rows, K, dtype=dt, std=K ** -0.5)
    st["bias"] = (torch.randn(rows, generator=gen, device="cuda") * 0.1).to(wdt) if case["bias"] else None
    st["ws"] = torch.zeros((96 << 20) + 64 * rows, dtype=torch.uint8, device="cuda")
    if case["dir"] == "forward":
        st["residual"] = _randn(gen, R, N, dtype=dt, pad=pad, step=1) if case["residual"] else None
        st["out"] = _out(R, N, dtype=dt, pad=pad, step=1)
        st["z"] = _out(R, rows, dtype=dt) if case["save"] and act != "none" else None
        return st
    st["dout"] = _randn(gen, R, N, dtype=dt)
    st["z"] = _randn(gen, R, rows, dtype=dt, std=1.5) if act != "none" else None
    st["dz"] = _out(R, rows, dtype=dt) if act != "none" else None
    st["dx"], st["dw"] = _out(R, K, dtype=dt), _out(rows, K, dtype=dt)
    st["db"] = torch.zeros(rows, dtype=wdt, device="cuda")
    return st


# ---- the library's calls ------------------------------------------------------
def _run_own(st):
    m = _library()
    case = st["case"]
    act = {"act": case["act"], "alpha": ALPHA, "limit": LIMIT}
    if case["op"] == "layer":
        m.moe_layer16_forward(st["x"], st["W_r"], None, st["w1"], st["w2"], st["out"], st["ids"], st["wts"], st["ws"],
                              b1=st["b1"], n_shared=case["shared"], routed_scale=case["scale"], **act)
        return {"out": st["out"], "ids": st["ids"], "wts": st["wts"]}
    if case["dir"] == "forward":
        m.moe_linear_forward(st["x"], st["w"], st["out"], st["ws"], bias=st["bias"], residual=st["residual"], z=st["z"], **act)
        return {"out": st["out"]} if st["z"] is None else {"out": st["out"], "z": st["z"]}
    m.moe_linear_backward(st["dout"], st["x"], st["w"], st["z"], st["dz"], st["dx"], st["dw"], st["db"], st["ws"], **act)
    return {"dx": st["dx"], "dw": st["dw"], "db": st["db"]}


# ---- the plain forms ------------------------------------------------------------
def _cdf(v):
    return 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))


def _activation(z, act, grads=False):
    """act of z [R, halves * N] by rows; with grads its derivatives by each half."""
    if act in GATED:
        g, u = z.chunk(2, -1)
        if act == "geglu":
            c = _cdf(g)
            a = g * c * u
            d = (c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)) * u, g * c
        elif act == "swiglu":
            s = torch.sigmoid(g)
            a = g * s * u
            d = (s + g * s * (1 - s)) * u, g * s
        else:
            gc, uc = g.clamp(-LIMIT, LIMIT), u.clamp(-LIMIT, LIMIT)
            s = torch.sigmoid(ALPHA * gc)
            a = gc * s * uc
            d = ((g.abs() <= LIMIT) * (s + ALPHA * gc * s * (1 - s)) * uc, (u.abs() <= LIMIT) * gc * s)
    elif act == "srelu":
        r = z.clamp_min(0)
        a, d = r * r, (2 * r,)
    elif act == "gelu":
        c = _cdf(z)
        a, d = z * c, (c + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi),)
    elif act == "silu":
        s = torch.sigmoid(z)
        a, d = z * s, (s + z * s * (1 - s),)
    else:
        a, d = z, (torch.ones_like(z),)
    return (a, d) if grads else a


def _route(x, W_r, k, scale):
    """Ids (ties to the lowest) and softmax weights; the logits in 64 bits, as two may lie next to each other."""
    v, ids = torch.sort(x.double() @ W_r.double(), dim=1, descending=True, stable=True)
    e = torch.exp(v[:, :k] - v[:, :1])
    return ids[:, :k], (e / e.sum(1, keepdim=True) * scale).float()


def _plain_layer(st):
    case = st["case"]
    T, E, k, act = case["T"], case["E"], case["k"], case["act"]
    w1, w2, b1 = st["w1"], st["w2"], st["b1"]
    x = st["x"].float()
    ids, wts = _route(st["x"], st["W_r"], k, case["scale"])
    out = torch.zeros(T, case["H"], device="cuda")

    def expert(rows, a, b, bias):
        h = rows @ a.float().t()
        return _activation(h if bias is None else h + bias, act) @ b.float().t()

    if T * k <= E:  # a few assignments: only their experts are read
        for t in range(T):
            for j in range(k):
                e = ids[t, j : j + 1]
                bias = None if b1 is None else b1[e][0]
                out[t] += wts[t, j] * expert(x[t : t + 1], w1[e][0], w2[e][0], bias)[0]
    else:
        share = torch.zeros(T, E, device="cuda").scatter_(1, ids, wts)
        for e in range(E):
            out += share[:, e, None] * expert(x, w1[e], w2[e], None if b1 is None else b1[e])
    for e in range(E, E + case["shared"]):
        out += expert(x, w1[e], w2[e], None if b1 is None else b1[e])
    return {"out": out.to(st["out"].dtype), "ids": ids.int(), "wts": wts}


def _run_plain(st):
    case = st["case"]
    if case["op"] == "layer":
        return _plain_layer(st)
    dt, act = DTYPES[case["dtype"]], case["act"]
    x, w = st["x"].float(), st["w"].float()
    if case["dir"] == "forward":
        z = x @ w.t()
        if st["bias"] is not None:
            z += st["bias"].float()
        out = _activation(z, act)
        if st["residual"] is not None:
            out = out + st["residual"].float()
        return {"out": out.to(dt)} if st["z"] is None else {"out": out.to(dt), "z": z.to(dt)}
    dz = st["dout"].float()
    if act != "none":
        dz = torch.cat([dz * g for g in _activation(st["z"].float(), act, True)[1]], 1)
    return {"dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt), "db": dz.sum(0).to(st["db"].dtype)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- what a pass cannot do without ---------------------------------------------
def work(case):
    if case["op"] == "layer":
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
        per = (3 if case["act"] in GATED else 2) * H * I
        # experts that some token chooses, when each chooses k of E at random
        touched = E * (1 - (1 - k / E) ** T) + case["shared"]
        bias = touched * 8 * I if case["bias"] else 0
        return {"bytes": int(2 * touched * per + bias + 4 * H * E + 4 * T * H + 8 * T * k),
                "flops": 2 * T * (k + case["shared"]) * per + 2 * T * H * E}
    R, N, K, rows = case["R"], case["N"], case["K"], case["N"] * (2 if case["act"] in GATED else 1)
    we = 4 if case["wdtype"] == "f32" else 2
    saved = 2 * R * rows if case["act"] != "none" else 0
    if case["dir"] == "forward":
        return {"bytes": 2 * R * K + 2 * rows * K + (we * rows if case["bias"] else 0) + 2 * R * N * (2 if case["residual"] else 1)
                + (saved if case["save"] else 0), "flops": 2 * R * rows * K}
    return {"bytes": 2 * R * N + saved + 4 * R * K + 4 * rows * K + we * rows, "flops": 4 * R * rows * K}


# ---- the definition in 64 bits ---------------------------------------------------
def _act64(parts, act):
    """Value and derivatives by the formulas, on 64-bit columns (gate, up) or (h,)."""
    if act == "none":
        return parts[0], [torch.ones_like(parts[0])]
    g = parts[0]
    if act == "srelu":
        pos = (g > 0).double()
        return pos * g ** 2, [2 * pos * g]
    u = parts[1] if len(parts) == 2 else torch.ones_like(g)
    if act in ("gelu", "geglu"):
        phi = 0.5 * torch.erfc(-g / math.sqrt(2.0))
        f, df = g * phi, phi + g * torch.exp(-(g ** 2) / 2) / math.sqrt(2 * math.pi)
    elif act in ("silu", "swiglu"):
        s = 1 / (1 + torch.exp(-g))
        f, df = g * s, s * (1 + g * (1 - s))
    else:
        lim = torch.full_like(g, LIMIT)
        gc = torch.minimum(torch.maximum(g, -lim), lim)
        s = 1 / (1 + torch.exp(-ALPHA * gc))
        f, df = gc * s, (g == gc).double() * s * (1 + ALPHA * gc * (1 - s))
        uc = torch.minimum(torch.maximum(u, -lim), lim)
        return f * uc, [df * uc, (u == uc).double() * f]
    return f * u, [df * u, f][: len(parts)]


def exact(case, seed):
    st = prepare(case, seed)
    act, halves = case["act"], 2 if case["act"] in GATED else 1
    if case["op"] == "layer":
        T, H, I, E, k = case["T"], case["H"], case["I"], case["E"], case["k"]
        x = st["x"].double()
        logits = (x @ st["W_r"].double()).tolist()
        ids, wts, rows = [], [], [[] for _ in range(E)]
        for t, row in enumerate(logits):
            best = sorted(range(E), key=lambda e: (-row[e], e))[:k]
            p = [math.exp(row[e] - row[best[0]]) for e in best]
            ids.append(best)
            wts.append([v * case["scale"] / math.fsum(p) for v in p])
            for e, w in zip(best, wts[-1]):
                rows[e].append((t, w))
        rows += [[(t, 1.0) for t in range(T)] for _ in range(case["shared"])]
        out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for e, chosen in enumerate(rows):
            if not chosen:
                continue
            at = torch.tensor([t for t, _ in chosen], device="cuda")
            by = torch.tensor([w for _, w in chosen], dtype=torch.float64, device="cuda")
            parts = []
            for c in range(halves):
                h = x[at] @ st["w1"][e, c * I : (c + 1) * I].double().t()
                parts.append(h if st["b1"] is None else h + st["b1"][e, c * I : (c + 1) * I].double())
            y = _act64(parts, act)[0] * by[:, None]
            out.index_add_(0, at, y @ st["w2"][e].double().t())
        return {"out": out, "ids": torch.tensor(ids, device="cuda"), "wts": torch.tensor(wts, dtype=torch.float64, device="cuda")}
    R, N, K = case["R"], case["N"], case["K"]
    x, w = st["x"].double(), st["w"].double()
    if case["dir"] == "forward":
        z = torch.empty(R, halves * N, dtype=torch.float64, device="cuda")
        torch.mm(x, w.t(), out=z)
        if st["bias"] is not None:
            z += st["bias"].double()
        out = _act64(list(z.split(N, 1)), act)[0]
        if st["residual"] is not None:
            out = out + st["residual"].double()
        return {"out": out} if st["z"] is None else {"out": out, "z": z}
    d = st["dout"].double()
    dz = d if act == "none" else torch.cat([d * g for g in _act64(list(st["z"].double().split(N, 1)), act)[1]], 1)
    return {"dx": dz @ w, "dw": dz.t() @ x, "db": dz.sum(0)}
