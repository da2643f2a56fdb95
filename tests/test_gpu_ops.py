"""Training-side operators on the GPU against their 64-bit plain forms
(ops_ref.py), at the sizes, strides, types and masks where they can go wrong."""
import pytest
import torch

import quantized_grouped_gemm_topk_gb300 as m
import ops_ref as P

from util import cuda_device

pytestmark = pytest.mark.gpu

BF16, F16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
NAN = float("nan")


def _gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _canary(buf, cols, what):
    """The buffer's columns past `cols` still hold what strided() put there."""
    rest = buf[..., cols:]
    assert bool(torch.isnan(rest.float()).all()), f"{what}: wrote past its rows"


# ---- layer norm -----------------------------------------------------------------
NORM_SIZES = [(1, 1), (1, 7168), (3, 8), (5, 31), (2, 256), (7, 264), (33, 257), (2, 2880), (3, 4099), (700, 64),
              (2, 16384), (2, 16392), (1, 33000), (2, 40000), (1300, 1031)]


@pytest.mark.parametrize("T,H", NORM_SIZES)
@pytest.mark.parametrize("dtype,wdtype,pad", [(BF16, BF16, 0), (BF16, F32, 8), (F16, F16, 3), (F32, F32, 0)])
def test_layer_norm(T, H, dtype, wdtype, pad):
    cuda_device()
    g = _gen(T * 131 + H)
    x, _ = P.strided(_randn(g, T, H, dtype=dtype, std=2.0) + 0.5, pad)
    gamma, beta = (_randn(g, H) * 0.3 + 1).to(wdtype), _randn(g, H).to(wdtype)
    y, ybuf = P.strided(torch.zeros(T, H, dtype=dtype, device="cuda"), pad)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    eps = 1e-5
    m.moe_layer_norm_forward(x, gamma, beta, eps, y, mean, rstd)
    ry, rm, rr = P.norm_fwd(x, gamma, beta, eps)
    # the mean: H additions of x; the variance: H of (x - mu)^2, its relative error halved by the root
    mag = x.double().abs().mean(1)
    P.assert_within(mean, rm, (H + 4) * P.EPS32 * mag, "mean")
    dmean = (H + 4) * P.EPS32 * mag
    # a shift d of the mean adds d^2 to the variance; 8 EPS32: the root and the product with 1 / H
    rel = (H + 8) * P.EPS32 + (dmean * rr) ** 2
    P.assert_within(rstd, rr, rr * rel, "rstd")
    c = (x.double() - rm[:, None]).abs() * rr[:, None]
    gm = gamma.double().abs()
    bound = (c * (rel[:, None] + 4 * P.EPS32) + (dmean * rr)[:, None]) * gm + 2 * P.EPS32 * beta.double().abs()
    P.assert_within(y, ry, bound, "y")
    if pad:
        _canary(ybuf, H, "y")

    dy, _ = P.strided(_randn(g, T, H, dtype=dtype), pad)
    dx, dxbuf = P.strided(torch.zeros(T, H, dtype=dtype, device="cuda"), pad)
    dgamma, dbeta = torch.full_like(gamma, NAN), torch.full_like(beta, NAN)
    ws = torch.empty(m.moe_layer_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    m.moe_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws)
    rdx, rdg, rdb = P.norm_bwd(dy, x, gamma, mean, rstd)
    xh = (x.double() - mean.double()[:, None]).abs() * rstd.double()[:, None]
    t = dy.double().abs() * gm
    # three roundings a term, and the sums of H terms
    b = rstd.double()[:, None] * (4 * P.EPS32 * t + (H + 4) * P.EPS32 * t.mean(1, keepdim=True) +
                                  (H + 8) * P.EPS32 * xh * (t * xh).mean(1, keepdim=True))
    P.assert_within(dx, rdx, b, "dx")
    P.assert_within(dgamma, rdg, (T + 4) * P.EPS32 * (dy.double().abs() * xh).sum(0), "dgamma")
    P.assert_within(dbeta, rdb, (T + 4) * P.EPS32 * dy.double().abs().sum(0), "dbeta")
    if pad:
        _canary(dxbuf, H, "dx")
    # dx alone gives the same bits
    dx2 = torch.empty(T, H, dtype=dtype, device="cuda")
    m.moe_layer_norm_backward(dy, x, gamma, mean, rstd, dx2)
    if pad == 0:
        assert torch.equal(dx2, dx)


@pytest.mark.parametrize("T,H", [(700, 264), (1300, 2880), (900, 4096), (640, 7168), (620, 8200), (615, 16384), (1500, 520)])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (F16, F16), (F32, F32)])
def test_layer_norm_many_rows(T, H, dtype, wdtype):
    test_layer_norm(T, H, dtype, wdtype, 0)


@pytest.mark.parametrize("T,H,pad", [(700, 259, 0), (1300, 1031, 0), (610, 2881, 7), (900, 4099, 3), (650, 8195, 1), (640, 264, 3)])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (F16, F16), (F32, F32)])
def test_layer_norm_many_rows_at_any_alignment(T, H, pad, dtype, wdtype):
    test_layer_norm(T, H, dtype, wdtype, pad)


def test_layer_norm_rows_that_start_and_end_off_a_boundary():
    """A tensor that begins and ends inside 16-byte units: its neighbours in memory are NaN and stay unread."""
    cuda_device()
    g = _gen(21)
    for H, lead in ((301, 1), (1031, 3), (520, 5)):
        T = 700
        buf = torch.full((T * H + 16,), NAN, dtype=BF16, device="cuda")
        x = buf[lead:lead + T * H].view(T, H)
        x.copy_(_randn(g, T, H))
        y, mean, rstd = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        m.moe_layer_norm_forward(x, None, None, 1e-5, y, mean, rstd)
        z, mean2, rstd2 = torch.empty_like(y), torch.empty_like(mean), torch.empty_like(rstd)
        m.moe_layer_norm_forward(x.clone(), None, None, 1e-5, z, mean2, rstd2)
        assert torch.equal(y, z) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)


def test_layer_norm_without_weights_and_repeatable():
    cuda_device()
    g = _gen(5)
    x = _randn(g, 2500, 1100, dtype=BF16)
    y = torch.empty_like(x)
    m.moe_layer_norm_forward(x, None, None, 1e-6, y)
    P.assert_within(y, P.norm_fwd(x, None, None, 1e-6)[0], torch.full_like(y, 1e-5, dtype=torch.float64), "y")
    st = [torch.empty(2500, device="cuda") for _ in range(2)]
    m.moe_layer_norm_forward(x, None, None, 1e-6, y, *st)
    dy, dx = _randn(g, 2500, 1100, dtype=BF16), torch.empty_like(x)
    ws = torch.empty(m.moe_layer_norm_workspace_size(2500, 1100), dtype=torch.uint8, device="cuda")
    outs = []
    for _ in range(2):
        dg, db = torch.empty(1100, device="cuda"), torch.empty(1100, device="cuda")
        m.moe_layer_norm_backward(dy, x, None, *st, dx, dg, db, ws)
        outs.append((dg, db))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_layer_norm_gradient_by_differences():
    """dx, dgamma, dbeta of L = sum(c * y) against central differences of the 64-bit forward."""
    cuda_device()
    g = _gen(9)
    T, H = 3, 24
    x, c = _randn(g, T, H), _randn(g, T, H)
    gamma, beta = _randn(g, H), _randn(g, H)
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    m.moe_layer_norm_forward(x, gamma, beta, 1e-3, y, mean, rstd)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    ws = torch.empty(m.moe_layer_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    m.moe_layer_norm_backward(c, x, gamma, mean, rstd, dx, dg, db, ws)

    def loss(x, gamma, beta):
        return float((c.double() * P.norm_fwd(x, gamma, beta, 1e-3)[0]).sum())

    d = 1e-6      # 64 bits: differences are good to about 1e-9 of the loss's terms
    args = [x.double(), gamma.double(), beta.double()]
    for k, got in enumerate((dx, dg, db)):
        for i in range(0, got.numel(), 5):
            up, dn = [a.clone() for a in args], [a.clone() for a in args]
            up[k].view(-1)[i] += d
            dn[k].view(-1)[i] -= d
            num = (loss(*up) - loss(*dn)) / (2 * d)
            assert abs(num - float(got.view(-1)[i])) < 1e-4 * (1 + abs(num)), (k, i)


def test_layer_norm_nan_stays_in_its_row_and_no_rows():
    cuda_device()
    g = _gen(11)
    x = _randn(g, 9, 512, dtype=BF16)
    x[4, 7] = NAN
    x[6, 1] = float("inf")
    y = torch.empty_like(x)
    m.moe_layer_norm_forward(x, None, None, 1e-5, y)
    bad = torch.isnan(y.float()).any(1).tolist()
    assert bad == [i in (4, 6) for i in range(9)]
    dg, db = torch.full((512,), NAN, device="cuda"), torch.full((512,), NAN, device="cuda")
    e = torch.empty(0, 512, dtype=BF16, device="cuda")
    z = torch.empty(0, device="cuda")
    m.moe_layer_norm_forward(e, None, None, 1e-5, e)
    m.moe_layer_norm_backward(e, e, None, z, z, e, dg, db, torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert float(dg.abs().sum()) == 0 and float(db.abs().sum()) == 0
    # a constant row: variance zero, eps alone
    one = torch.full((1, 77), 3.0, device="cuda")
    yo, mean, rstd = torch.empty_like(one), torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    m.moe_layer_norm_forward(one, None, None, 1e-5, yo, mean, rstd)
    assert float(yo.abs().max()) <= 1e-3 and abs(float(mean) - 3) < 1e-5


# ---- activation checkpoints --------------------------------------------------------
CKPT_SIZES = [(1, 1), (3, 128), (2, 129), (17, 96), (5, 2047), (33, 2048), (1, 8192), (700, 40), (9, 1000)]


@pytest.mark.parametrize("act", ["swiglu", "swiglu_clamp", "geglu", "srelu"])
@pytest.mark.parametrize("R,I", CKPT_SIZES)
@pytest.mark.parametrize("dtype,pad", [(BF16, 0), (F16, 8), (BF16, 3)])
def test_activation_checkpoint(R, I, act, dtype, pad):
    cuda_device()
    g = _gen(R * 31 + I)
    halves = 1 if act == "srelu" else 2
    nb = -(-I // 128)
    kw = dict(act=act, alpha=1.702, limit=2.5)
    h, _ = P.strided(_randn(g, R, halves * I, dtype=dtype, std=2.0), pad)
    w = torch.rand(R, generator=g, device="cuda")
    y, ybuf = P.strided(torch.zeros(R, I, dtype=dtype, device="cuda"), pad)
    q, qbuf = P.strided(torch.zeros(R, halves * I, dtype=E4M3, device="cuda"), pad)
    s = torch.full((R, halves * nb), NAN, device="cuda")
    m.moe_act_ckpt_forward(h, w, y, q, s, **kw)
    hs = [h[:, k * I:(k + 1) * I] for k in range(halves)]
    a, _ = P.activation([v.double() for v in hs], act, 1.702, 2.5)
    # the fast exponential and divide: a few 2^-22 relative, growing with the exponent (|alpha g| / 2^23)
    rel = 2.0 ** -19
    wd = w.double()[:, None]
    P.assert_within(y, wd * a, rel * (wd * a).abs() + 1e-30, "y")
    for k, v in enumerate(hs):
        sk = s[:, k * nb:(k + 1) * nb]
        assert torch.equal(sk, P.row_scales(v)), "scales"
        P.assert_codes(q[:, k * I:(k + 1) * I], v.float(), sk.repeat_interleave(128, 1)[:, :I], "codes")
    if pad:
        _canary(ybuf, I, "y")
        assert bool((qbuf[:, halves * I:].view(torch.uint8) == 0x7F).all())

    dy, _ = P.strided(_randn(g, R, I, dtype=dtype), pad)
    dh, dhbuf = P.strided(torch.zeros(R, halves * I, dtype=dtype, device="cuda"), pad)
    dw = torch.full((R,), NAN, device="cuda")
    y2 = torch.empty(R, I, dtype=dtype, device="cuda")
    m.moe_act_ckpt_backward(dy, q, s, w, dh, dw, y2, **kw)
    ht = [P.decode(q[:, k * I:(k + 1) * I]) * s[:, k * nb:(k + 1) * nb].repeat_interleave(128, 1)[:, :I].double()
          for k in range(halves)]
    # h~ itself is rounded to fp32 once; a value that this moves across the clamp would change its gradient
    ht = [v.float().double() for v in ht]
    a, grads = P.activation(ht, act, 1.702, 2.5)
    d = dy.double()
    # cancellation in s + g s (1 - s): absolute error against |s| + |g s|
    big = 1 + sum(v.abs() for v in ht) ** 2
    for k, gr in enumerate(grads):
        P.assert_within(dh[:, k * I:(k + 1) * I], wd * d * gr, 2.0 ** -18 * (wd * d).abs() * big + 1e-30, f"dh{k}")
    P.assert_within(y2, wd * a, rel * (wd * a).abs() + 1e-30, "y again")
    P.assert_within(dw, (d * a).sum(1), ((I + 8) * P.EPS32 + rel) * (d * a).abs().sum(1) + 1e-30, "dw")
    if pad:
        _canary(dhbuf, halves * I, "dh")
    dh2 = torch.empty(R, halves * I, dtype=dtype, device="cuda")
    m.moe_act_ckpt_backward(dy, q, s, w, dh2, **kw)      # without dw and y
    if pad == 0:
        assert torch.equal(dh2, dh)


# more rows than there are warps, at odd widths and strides too: rows of less than a block, of one quarter's and of four quarters' blocks
@pytest.mark.parametrize("act", ["swiglu", "srelu"])
@pytest.mark.parametrize("R,I", [(5001, 100), (4999, 129), (6000, 383), (5003, 512), (20001, 41)])
@pytest.mark.parametrize("dtype,pad", [(BF16, 0), (F16, 8), (BF16, 3)])
def test_activation_checkpoint_many_rows(R, I, act, dtype, pad):
    test_activation_checkpoint(R, I, act, dtype, pad)


@pytest.mark.parametrize("R,I", [(1, 5), (3, 7), (40, 301), (5000, 131)])
@pytest.mark.parametrize("lead", [1, 6])
def test_activation_checkpoint_of_tensors_off_a_boundary(R, I, lead):
    """Tensors that begin and end inside 16-byte units: their neighbours in memory stay unread and unwritten."""
    cuda_device()
    g = _gen(R + I)

    def inside(cols, dtype):
        raw = torch.full(((R * cols + 32) * dtype.itemsize,), 0x7F, dtype=torch.uint8, device="cuda")
        if dtype == BF16:
            raw.view(BF16).fill_(NAN)
        before = raw.clone()
        a, n = lead * dtype.itemsize, R * cols * dtype.itemsize

        def untouched():
            return torch.equal(raw[:a], before[:a]) and torch.equal(raw[a + n:], before[a + n:])
        return raw[a:a + n].view(dtype).view(R, cols), untouched

    nb = -(-I // 128)
    h, _ = inside(2 * I, BF16)
    h.copy_(_randn(g, R, 2 * I, std=2.0))
    dy, _ = inside(I, BF16)
    dy.copy_(_randn(g, R, I))
    w = torch.rand(R, generator=g, device="cuda")
    (y, fy), (q, fq), (dh, fh) = inside(I, BF16), inside(2 * I, E4M3), inside(2 * I, BF16)
    s, dw = torch.empty(R, 2 * nb, device="cuda"), torch.empty(R, device="cuda")
    m.moe_act_ckpt_forward(h, w, y, q, s)
    m.moe_act_ckpt_backward(dy, q, s, w, dh, dw)
    assert fy() and fq() and fh()
    y2, q2, s2 = torch.empty(R, I, dtype=BF16, device="cuda"), torch.empty(R, 2 * I, dtype=E4M3, device="cuda"), torch.empty_like(s)
    dh2, dw2 = torch.empty(R, 2 * I, dtype=BF16, device="cuda"), torch.empty_like(dw)
    m.moe_act_ckpt_forward(h.clone(), w, y2, q2, s2)
    m.moe_act_ckpt_backward(dy.clone(), q2, s2, w, dh2, dw2)
    assert torch.equal(y, y2) and torch.equal(q.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s, s2)
    assert torch.equal(dh, dh2) and torch.equal(dw, dw2) and bool(torch.isfinite(dw).all())


def test_activation_checkpoint_special_values():
    """Zeros, the smallest and largest values, infinities and NaN; no weight; no rows."""
    cuda_device()
    I = 256
    h = torch.zeros(6, 2 * I, dtype=BF16, device="cuda")
    h[1] = 2.0 ** -133                                   # the smallest subnormals
    h[2] = 3.38e38
    h[3, 5], h[3, I + 9] = NAN, float("inf")
    h[3, 6] = 2.0
    h[4] = -50.0
    h[4, I:] = 1.0
    h[5] = 120.0
    y, q = torch.empty(6, I, dtype=BF16, device="cuda"), torch.empty(6, 2 * I, dtype=E4M3, device="cuda")
    s = torch.empty(6, 4, device="cuda")
    m.moe_act_ckpt_forward(h, None, y, q, s, act="swiglu")
    assert torch.equal(s, torch.cat([P.row_scales(h[:, :I]), P.row_scales(h[:, I:])], 1))
    v = P.decode(q)
    assert bool((v[0] == 0).all()) and bool((v[1] == 2.0 ** -7).all())   # 2^-133 over the smallest scale
    assert bool((v[2] == 448).all())
    nan = torch.isnan(v).nonzero().tolist()
    assert nan == [[3, 5], [3, I + 9]]
    assert torch.isnan(y.float()).nonzero().tolist()[0] == [3, 5]
    assert float(v[3, 6]) * float(s[3, 0]) == pytest.approx(2.0, rel=2 ** -4)
    dy = torch.ones(6, I, dtype=BF16, device="cuda")
    dh, dw = torch.empty(6, 2 * I, dtype=BF16, device="cuda"), torch.empty(6, device="cuda")
    m.moe_act_ckpt_backward(dy, q, s, None, dh, dw, act="swiglu")
    assert torch.isnan(dw).tolist() == [False, False, False, True, False, False]
    assert bool(torch.isnan(dh[3].float()).sum() == 3)           # gate 5, up 5; gate 9 (up's derivative is g sigmoid(g))
    assert bool((dh[4].float().abs() < 1e-18).all())             # sigmoid(-50)
    e = h[:0]
    m.moe_act_ckpt_forward(e, None, y[:0], q[:0], s[:0], act="swiglu")
    m.moe_act_ckpt_backward(dy[:0], q[:0], s[:0], None, e, act="swiglu")


def test_activation_gradient_by_differences():
    """dh against central differences of the 64-bit activation at the checkpointed point, and dw."""
    cuda_device()
    g = _gen(2)
    R, I = 4, 160
    for act in ("swiglu", "swiglu_clamp", "geglu", "srelu"):
        halves = 1 if act == "srelu" else 2
        kw = dict(act=act, alpha=1.702, limit=2.5)
        h = _randn(g, R, halves * I, dtype=F16)
        w = torch.rand(R, generator=g, device="cuda")
        y, q = torch.empty(R, I, dtype=F16, device="cuda"), torch.empty(R, halves * I, dtype=E4M3, device="cuda")
        s = torch.empty(R, 2 * halves, device="cuda")
        m.moe_act_ckpt_forward(h, w, y, q, s, **kw)
        dy = _randn(g, R, I, dtype=F16)
        dh, dw = torch.empty_like(h), torch.empty(R, device="cuda")
        m.moe_act_ckpt_backward(dy, q, s, w, dh, dw, **kw)
        ht = [P.decode(q[:, k * I:(k + 1) * I]) * s[:, 2 * k:2 * k + 2].repeat_interleave(128, 1)[:, :I].double()
              for k in range(halves)]
        d = 1e-6
        for k in range(halves):
            up = [v + (d if j == k else 0) for j, v in enumerate(ht)]
            dn = [v - (d if j == k else 0) for j, v in enumerate(ht)]
            num = (P.activation(up, act, 1.702, 2.5)[0] - P.activation(dn, act, 1.702, 2.5)[0]) / (2 * d)
            ref = w.double()[:, None] * dy.double() * num
            got = dh[:, k * I:(k + 1) * I].double()
            edge = (ht[k].abs() - 2.5).abs() < 1e-4 if act == "swiglu_clamp" else ht[k].abs() < 1e-4
            assert bool(((got - ref).abs() <= 2e-3 * ref.abs() + 1e-5)[~edge].all()), (act, k)


# ---- FP8 quantisers --------------------------------------------------------------------
@pytest.mark.parametrize("R,C", [(1, 1), (3, 128), (2, 129), (65, 1000), (4, 7168), (300, 40), (2, 2047)])
@pytest.mark.parametrize("dtype,pad", [(BF16, 0), (F16, 5), (F32, 0), (F32, 4)])
def test_fp8_quant_rows(R, C, dtype, pad):
    cuda_device()
    g = _gen(R + C)
    x, _ = P.strided(_randn(g, R, C, dtype=dtype, std=30.0), pad)
    x[0, 0] = 0.0
    if C > 130:
        x[:, 128:] = 0           # a block of zeros, and one with an infinity and a NaN in the first
        x[0, 1], x[0, 2] = NAN, -float("inf")
    q, qbuf = P.strided(torch.zeros(R, C, dtype=E4M3, device="cuda"), pad, whole=16)
    s = torch.full((R, -(-C // 128) + 3), NAN, device="cuda")
    m.moe_fp8_quant_rows(x, q, s[:, :-3])
    assert torch.equal(s[:, :-3], P.row_scales(x))
    assert bool(torch.isnan(s[:, -3:]).all())
    P.assert_codes(q, x.float(), s[:, :-3].repeat_interleave(128, 1)[:, :C], "codes")
    assert bool((qbuf[:, C:].view(torch.uint8) == 0x7F).all())


@pytest.mark.parametrize("R,C,lead", [(1, 3, 1), (3, 300, 7), (700, 131, 5)])
def test_fp8_quant_rows_of_tensors_off_a_boundary(R, C, lead):
    """Rows that begin and end inside 16-byte units, codes at odd addresses: the neighbours stay unread and unwritten."""
    cuda_device()
    buf = torch.full((R * C + 32,), NAN, dtype=BF16, device="cuda")
    x = buf[lead:lead + R * C].view(R, C)
    x.copy_(_randn(_gen(C), R, C))
    raw = torch.full((R * C + 32,), 0x7F, dtype=torch.uint8, device="cuda")
    q = raw[lead:lead + R * C].view(E4M3).view(R, C)
    s, s2 = torch.empty(R, -(-C // 128), device="cuda"), torch.empty(R, -(-C // 128), device="cuda")
    m.moe_fp8_quant_rows(x, q, s)
    assert bool((raw[:lead] == 0x7F).all()) and bool((raw[lead + R * C:] == 0x7F).all())
    q2 = torch.empty(R, C, dtype=E4M3, device="cuda")
    m.moe_fp8_quant_rows(x.clone(), q2, s2)
    assert torch.equal(s, s2) and torch.equal(q.contiguous().view(torch.uint8), q2.view(torch.uint8))
    assert torch.equal(s, P.row_scales(x))


@pytest.mark.parametrize("G,N,K", [(1, 1, 1), (2, 128, 128), (3, 130, 257), (1, 2048, 200), (2, 96, 1031), (1, 16, 4096)])
@pytest.mark.parametrize("dtype,pad", [(BF16, 0), (F32, 3)])
@pytest.mark.parametrize("transposed", [True, False])
def test_fp8_quant_weights(G, N, K, dtype, pad, transposed):
    cuda_device()
    g = _gen(G + N + K)
    w, _ = P.strided(_randn(g, G, N, K, dtype=dtype), pad)
    w[-1, N // 2, K // 2] = NAN
    nb, kb = -(-N // 128), -(-K // 128)
    q, qbuf = P.strided(torch.zeros(G, N, K, dtype=E4M3, device="cuda"), pad, whole=16)
    qt, qtbuf = P.strided(torch.zeros(G, K, N, dtype=E4M3, device="cuda"), pad, whole=16)
    s, st = torch.full((G, nb, kb), NAN, device="cuda"), torch.full((G, kb, nb), NAN, device="cuda")
    m.moe_fp8_quant_weights(w, q, s, *((qt, st) if transposed else ()))
    p = torch.zeros(G, nb * 128, kb * 128, device="cuda")
    p[:, :N, :K] = P.finite_mag(w.float())
    assert torch.equal(s, P.scale_of(p.view(G, nb, 128, kb, 128).amax((2, 4))))
    e = s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    P.assert_codes(q, w.float(), e, "codes")
    assert bool((qbuf[:, :, K:].view(torch.uint8) == 0x7F).all())
    if transposed:
        assert torch.equal(qt.view(torch.uint8), q.view(torch.uint8).transpose(1, 2))
        assert torch.equal(st, s.transpose(1, 2))
        assert bool((qtbuf[:, :, N:].view(torch.uint8) == 0x7F).all())


# ---- products --------------------------------------------------------------------------
def _offsets(sizes):
    off = [0]
    for c in sizes:
        off.append(off[-1] + c)
    return off, torch.tensor(off, dtype=torch.int32, device="cuda")


def _workspace(kind, R, N, K, G):
    n = m.moe_mm_workspace_size(kind, R, N, K, G)
    assert n <= 256 + (64 << 20)
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


GROUPS = [[1], [0, 0], [5, 0, 1, 130], [128, 256, 64], [0, 300, 0, 17, 1], [1] * 40, [700]]
SHAPES = [(1, 1), (64, 64), (72, 40), (256, 512), (300, 129), (1031, 200), (520, 1999)]


@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: "-".join(map(str, s[:5])))
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("dtype,out,trans", [(BF16, F32, False), (BF16, BF16, True), (F16, F16, False), (F16, F32, True)])
def test_grouped_mm(sizes, N, K, dtype, out, trans):
    cuda_device()
    g = _gen(N + K + len(sizes))
    off, offsets = _offsets(sizes)
    R, G = off[-1] + 3, len(sizes)                   # three rows in no group
    x, _ = P.strided(_randn(g, R, K, dtype=dtype), 8, whole=8)
    x[off[-1]:] = NAN                                # they reach no one
    w, _ = P.strided(_randn(g, G, K, N, dtype=dtype) if trans else _randn(g, G, N, K, dtype=dtype), 8, whole=8)
    for e, c in enumerate(sizes):
        if c == 0:
            w[e] = NAN                               # nor do the weights of groups without rows
    y, ybuf = P.strided(torch.full((R, N), NAN, dtype=out, device="cuda"), 5)
    ws = _workspace(m.MOE_MM_ROWS, R, N, K, G)
    m.moe_grouped_mm(x, w, offsets, y, ws, trans_w=trans)
    ref, mag = P.grouped(x, w.transpose(1, 2) if trans else w, off)
    P.assert_within(y, ref, (K + 4) * P.EPS32 * mag, "out")
    assert bool((y[off[-1]:] == 0).all())
    _canary(ybuf, N, "out")
    assert m.moe_mm_read_status(ws) == 0
    y2 = torch.empty(R, N, dtype=out, device="cuda")
    m.moe_grouped_mm(x, w, offsets, y2, ws, trans_w=trans)
    assert torch.equal(y2.view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: "-".join(map(str, s[:5])))
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("dtype,out", [(BF16, F32), (F16, F16)])
def test_grouped_mm_wgrad(sizes, N, K, dtype, out):
    cuda_device()
    g = _gen(N + K + len(sizes))
    off, offsets = _offsets(sizes)
    R, G = off[-1] + 20, len(sizes)
    dy, _ = P.strided(_randn(g, R, N, dtype=dtype), 8, whole=8)
    x, _ = P.strided(_randn(g, R, K, dtype=dtype), 8, whole=8)
    dy[off[-1]:], x[off[-1]:] = NAN, NAN             # rows past the last group, right behind its last tile
    dw, buf = P.strided(torch.full((G, N, K), NAN, dtype=out, device="cuda"), 3)
    ws = _workspace(m.MOE_MM_WGRAD, R, N, K, G)
    m.moe_grouped_mm_wgrad(dy, x, offsets, dw, ws)
    ref, mag = P.grouped_wgrad(dy, x, off)
    cnt = torch.tensor(sizes, device="cuda", dtype=torch.float64)[:, None, None]
    P.assert_within(dw, ref, (cnt + 4) * P.EPS32 * mag, "dw")
    _canary(buf, K, "dw")
    assert m.moe_mm_read_status(ws) == 0


@pytest.mark.parametrize("N,K", [(1536, 64), (1500, 200), (2001, 1003), (1600, 1024)])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F32)])
@pytest.mark.parametrize("what", ["forward", "dgrad", "wgrad"])
def test_products_of_many_tiles(N, K, dtype, out, what):
    """Enough tiles for every pair of SMs, ragged groups of one row to thousands."""
    sizes = [300, 0, 17, 1, 1000, 256, 31, 2100, 0]
    if what == "wgrad":
        test_grouped_mm_wgrad(sizes, N, K, dtype, out)
    else:
        test_grouped_mm(sizes, N, K, dtype, out, what == "dgrad")


def test_grouped_mm_wgrad_nan_stays_in_its_group():
    cuda_device()
    g = _gen(1)
    off, offsets = _offsets([37, 50, 3, 64, 90])
    dy, x = _randn(g, off[-1], 136, dtype=BF16), _randn(g, off[-1], 264, dtype=BF16)
    dy[off[1]:off[2]], x[off[1]:off[2]] = NAN, float("inf")
    dw = torch.empty(5, 136, 264, device="cuda")
    m.moe_grouped_mm_wgrad(dy, x, offsets, dw, _workspace(m.MOE_MM_WGRAD, off[-1], 136, 264, 5))
    assert [bool(torch.isnan(dw[e]).any()) for e in range(5)] == [False, True, False, False, False]
    y = torch.empty(off[-1], 136, device="cuda")
    w = _randn(g, 5, 136, 264, dtype=BF16)
    m.moe_grouped_mm(x, w, offsets, y, _workspace(m.MOE_MM_ROWS, off[-1], 136, 264, 5))
    bad = ~torch.isfinite(y).all(1)
    assert bool(bad[off[1]:off[2]].all()) and not bool(bad[:off[1]].any()) and not bool(bad[off[2]:].any())


@pytest.mark.parametrize("R,N,K", [(1, 64, 8192), (16, 128, 4096), (40, 7168, 512), (4096, 256, 96), (2000, 1000, 3000),
                                   (20000, 64, 72)])
def test_products_of_one_group(R, N, K):
    """One group, where the reduction may be split over the SMs: all three directions and FP8."""
    cuda_device()
    g = _gen(R + N)
    off, offsets = _offsets([R])
    x, w = _randn(g, R, K, dtype=BF16), _randn(g, 1, N, K, dtype=BF16, std=0.05)
    for out in (BF16, F32):
        y = torch.full((R, N), NAN, dtype=out, device="cuda")
        ws = _workspace(m.MOE_MM_ROWS, R, N, K, 1)
        m.moe_grouped_mm(x, w, offsets, y, ws)
        ref, mag = P.grouped(x, w, off)
        P.assert_within(y, ref, (K + 4) * P.EPS32 * mag, "out")
        assert m.moe_mm_read_status(ws) == 0
    dy = _randn(g, R, N, dtype=BF16)
    dx = torch.full((R, K), NAN, dtype=BF16, device="cuda")
    m.moe_grouped_mm(dy, w, offsets, dx, _workspace(m.MOE_MM_ROWS, R, K, N, 1), trans_w=True)
    ref, mag = P.grouped(dy, w.transpose(1, 2), off)
    P.assert_within(dx, ref, (N + 4) * P.EPS32 * mag, "dx")
    dw = torch.full((1, N, K), NAN, device="cuda")
    m.moe_grouped_mm_wgrad(dy, x, offsets, dw, _workspace(m.MOE_MM_WGRAD, R, N, K, 1))
    ref, mag = P.grouped_wgrad(dy, x, off)
    P.assert_within(dw, ref, (R + 4) * P.EPS32 * mag, "dw")


def _fp8(g, R, N, K, G, extra=0):
    x, w = _randn(g, R, K, std=2.0), _randn(g, G, N, K, std=0.05)
    xq, _ = P.strided(torch.zeros(R, K, dtype=E4M3, device="cuda"), 16 * extra, whole=16)
    wq, _ = P.strided(torch.zeros(G, N, K, dtype=E4M3, device="cuda"), 16 * extra, whole=16)
    kb, nb = -(-K // 128), -(-N // 128)
    xs = torch.empty(R, kb + extra, device="cuda")[:, :kb]
    ws = torch.empty(G, nb, kb, device="cuda")
    m.moe_fp8_quant_rows(x, xq, xs)
    m.moe_fp8_quant_weights(w, wq, ws)
    x64 = P.decode(xq) * xs.double().repeat_interleave(128, 1)[:, :K]
    w64 = P.decode(wq) * ws.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    return xq, xs, wq, ws, x64, w64


@pytest.mark.parametrize("sizes", GROUPS, ids=lambda s: "-".join(map(str, s[:5])))
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("out,extra", [(F32, 1), (BF16, 0)])
def test_fp8_mm_grouped(sizes, N, K, out, extra):
    cuda_device()
    g = _gen(N + K + len(sizes))
    off, offsets = _offsets(sizes)
    R, G = off[-1] + 2, len(sizes)
    xq, xs, wq, wsc, x64, w64 = _fp8(g, R, N, K, G, extra)
    xq[off[-1]:].view(torch.uint8).fill_(0x7F)
    xs[off[-1]:] = NAN
    for e, c in enumerate(sizes):
        if c == 0:
            wsc[e] = NAN
    y, buf = P.strided(torch.full((R, N), NAN, dtype=out, device="cuda"), 3)
    ws = _workspace(m.MOE_MM_FP8, R, N, K, G)
    m.moe_fp8_mm(xq, xs, wq, wsc, y, ws, offsets=offsets)
    ref, mag = P.grouped(x64, w64, off)
    P.assert_within(y, ref, (K + 8) * P.EPS32 * mag, "out")
    assert bool((y[off[-1]:] == 0).all())
    _canary(buf, N, "out")
    assert m.moe_mm_read_status(ws) == 0


@pytest.mark.parametrize("R,N,K", [(1, 1, 1), (1, 7168, 2048), (3, 129, 7168), (130, 256, 640), (257, 520, 1000),
                                   (2048, 384, 384), (64, 8192, 128)])
@pytest.mark.parametrize("out", [F32, BF16, F16])
def test_fp8_mm_dense(R, N, K, out):
    cuda_device()
    xq, xs, wq, wsc, x64, w64 = _fp8(_gen(R + N + K), R, N, K, 1)
    y = torch.full((R, N), NAN, dtype=out, device="cuda")
    ws = _workspace(m.MOE_MM_FP8, R, N, K, 1)
    m.moe_fp8_mm(xq, xs, wq, wsc, y, ws)
    ref, mag = P.grouped(x64, w64, [0, R])
    P.assert_within(y, ref, (K + 8) * P.EPS32 * mag, "out")
    y2 = torch.full((R, N), NAN, dtype=out, device="cuda")
    m.moe_fp8_mm(xq, xs, wq, wsc, y2, ws)
    assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8))
    assert m.moe_mm_read_status(ws) == 0


# enough rows and columns for the wider tiles (128 columns; 256 in two halves): groups and columns that end inside a
# tile, columns that end in either half, an empty group
@pytest.mark.parametrize("sizes", [(2500,), (1290, 0, 2310), (4097,), (1025, 3001)], ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("N,K", [(2100, 700), (2432, 384), (4160, 1000)])
@pytest.mark.parametrize("out", [F32, BF16])
def test_fp8_mm_many_rows(sizes, N, K, out):
    cuda_device()
    off, offsets = _offsets(sizes)
    R, G = off[-1] + 3, len(sizes)
    xq, xs, wq, wsc, x64, w64 = _fp8(_gen(R + N), R, N, K, G)
    xq[off[-1]:].view(torch.uint8).fill_(0x7F)
    xs[off[-1]:] = NAN
    y, buf = P.strided(torch.full((R, N), NAN, dtype=out, device="cuda"), 8)
    ws = _workspace(m.MOE_MM_FP8, R, N, K, G)
    m.moe_fp8_mm(xq, xs, wq, wsc, y, ws, offsets=offsets)
    ref, mag = P.grouped(x64, w64, off)
    P.assert_within(y, ref, (K + 8) * P.EPS32 * mag, "out")
    assert bool((y[off[-1]:] == 0).all())
    _canary(buf, N, "out")
    assert m.moe_mm_read_status(ws) == 0


def test_fp8_mm_blocks_of_zeros_and_wide_scales():
    """Blocks of zeros next to blocks near fp32's ends: the scales multiply outside the sum over a block."""
    cuda_device()
    g = _gen(4)
    R, N, K = 70, 200, 700
    x, w = _randn(g, R, K), _randn(g, 1, N, K)
    x[:, :128] *= 1e18
    w[:, :, :128] *= 1e-18
    x[:, 256:384] = 0
    x[:, 384:512] *= 1e-20
    w[:, 128:, 384:512] *= 1e20
    w[:, :128, 512:] = 0
    xq, wq = torch.zeros(R, 704, dtype=E4M3, device="cuda")[:, :K], torch.zeros(1, N, 704, dtype=E4M3, device="cuda")[:, :, :K]
    xs, wsc = torch.empty(R, 6, device="cuda"), torch.empty(1, 2, 6, device="cuda")
    m.moe_fp8_quant_rows(x, xq, xs)
    m.moe_fp8_quant_weights(w, wq, wsc)
    y = torch.empty(R, N, device="cuda")
    m.moe_fp8_mm(xq, xs, wq, wsc, y, _workspace(m.MOE_MM_FP8, R, N, K, 1))
    x64 = P.decode(xq) * xs.double().repeat_interleave(128, 1)[:, :K]
    w64 = P.decode(wq) * wsc.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    ref, mag = P.grouped(x64, w64, [0, R])
    P.assert_within(y, ref, (K + 8) * P.EPS32 * mag, "out")


def test_products_with_wrong_offsets_stay_in_bounds():
    """Offsets that descend or leave [0, R]: clamped, flagged, every row written."""
    cuda_device()
    g = _gen(3)
    R, N, K = 100, 72, 64
    x, w = _randn(g, R, K, dtype=BF16), _randn(g, 4, N, K, dtype=BF16)
    ws = _workspace(m.MOE_MM_ROWS, R, N, K, 4)
    for raw, eff in (([0, 40, 20, 60, 500], [0, 40, 40, 60, 100]), ([-5, 10, 10, 2 ** 31 - 1, 90], [0, 10, 10, 100, 100])):
        y = torch.full((R, N), NAN, device="cuda")
        m.moe_grouped_mm(x, w, torch.tensor(raw, dtype=torch.int32, device="cuda"), y, ws)
        ref, mag = P.grouped(x, w, eff)
        P.assert_within(y, ref, (K + 4) * P.EPS32 * mag, "out")
        assert m.moe_mm_read_status(ws) == m.MOE_DEV_BAD_OFFSETS
    # rows before the first group are in none
    y = torch.full((R, N), NAN, device="cuda")
    off = [30, 40, 40, 60, 90]
    m.moe_grouped_mm(x, w, torch.tensor(off, dtype=torch.int32, device="cuda"), y, ws)
    ref, mag = P.grouped(x, w, off)
    P.assert_within(y, ref, (K + 4) * P.EPS32 * mag, "out")
    assert m.moe_mm_read_status(ws) == 0


def test_products_many_groups_and_no_rows():
    cuda_device()
    g = _gen(6)
    G, N, K = 2048, 24, 32
    sizes = [(7 * e) % 5 if e % 3 else 0 for e in range(G)]
    off, offsets = _offsets(sizes)
    R = off[-1]
    x, w = _randn(g, R, K, dtype=F16), _randn(g, G, N, K, dtype=F16)
    y = torch.full((R, N), NAN, device="cuda")
    m.moe_grouped_mm(x, w, offsets, y, _workspace(m.MOE_MM_ROWS, R, N, K, G))
    ref, mag = P.grouped(x, w, off)
    P.assert_within(y, ref, (K + 4) * P.EPS32 * mag, "out")
    none = torch.zeros(4, dtype=torch.int32, device="cuda")
    dw = torch.full((3, N, K), NAN, device="cuda")
    m.moe_grouped_mm_wgrad(torch.empty(0, N, dtype=F16, device="cuda"), torch.empty(0, K, dtype=F16, device="cuda"),
                           none, dw, _workspace(m.MOE_MM_WGRAD, 0, N, K, 3))
    assert bool((dw == 0).all())
    m.moe_grouped_mm(torch.empty(0, K, dtype=F16, device="cuda"), w[:3], none, torch.empty(0, N, device="cuda"),
                     _workspace(m.MOE_MM_ROWS, 0, N, K, 3))


def test_operators_on_another_stream_and_in_a_graph():
    """The chain of a block on a side stream and captured: the same bits as on the default stream."""
    cuda_device()
    g = _gen(8)
    R, H, I = 200, 256, 128
    off, offsets = _offsets([50, 0, 120, 30])
    x = _randn(g, R, H, dtype=BF16)
    w1 = _randn(g, 4, 2 * I, H, dtype=BF16, std=0.05)
    wrow = torch.rand(R, generator=g, device="cuda")
    y, h, a = (torch.empty(R, n, dtype=BF16, device="cuda") for n in (H, 2 * I, I))
    q, s = torch.empty(R, 2 * I, dtype=E4M3, device="cuda"), torch.empty(R, 2, device="cuda")
    ws = _workspace(m.MOE_MM_ROWS, R, 2 * I, H, 4)

    def chain():
        m.moe_layer_norm_forward(x, None, None, 1e-5, y)
        m.moe_grouped_mm(y, w1, offsets, h, ws)
        m.moe_act_ckpt_forward(h, wrow, a, q, s)

    chain()
    ref = [t.clone() for t in (y, h, a, q.view(torch.uint8), s)]
    side = torch.cuda.Stream()
    for t in (y, h, a, s):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, r) for p, r in zip((y, h, a, q.view(torch.uint8), s), ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for t in (y, h, a, s):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for p, r in zip((y, h, a, q.view(torch.uint8), s), ref))


def test_elements_past_32_bits():
    """More than 2^31 elements: the last rows come out as they do alone."""
    cuda_device()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    g, L = _gen(31), 70

    def last(t):
        return t[-L:].clone()

    R, I = 380001, 2881
    nb = -(-I // 128)
    h = torch.empty(R, 2 * I, dtype=BF16, device="cuda").normal_(generator=g)
    w = torch.rand(R, generator=g, device="cuda")

    def forward(h, w):
        n = h.shape[0]
        y, q = torch.empty(n, I, dtype=BF16, device="cuda"), torch.empty(n, 2 * I, dtype=E4M3, device="cuda")
        s = torch.empty(n, 2 * nb, device="cuda")
        m.moe_act_ckpt_forward(h, w, y, q, s)
        return y, q, s
    y, q, s = forward(h, w)
    y2, q2, s2 = forward(last(h), last(w))
    assert torch.equal(y[-L:], y2) and torch.equal(q[-L:].view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s[-L:], s2)
    dh2 = torch.empty(L, 2 * I, dtype=BF16, device="cuda")
    m.moe_act_ckpt_backward(last(y), q2, s2, last(w), dh2)
    m.moe_act_ckpt_backward(y, q, s, w, h)
    assert torch.equal(h[-L:], dh2)

    K, N, G = 2 * I + 6, 64, 3           # rows of h's buffer, as a product's: a stride that is a multiple of 8
    x = h.view(-1)[:R * 2 * I // K * K].view(-1, K)
    x.normal_(generator=g)
    T = x.shape[0]
    off = torch.tensor([0, 100000, 100000, T], dtype=torch.int32, device="cuda")
    wt = _randn(g, G, N, K, dtype=BF16, std=0.05)
    o = torch.empty(T, N, device="cuda")
    m.moe_grouped_mm(x, wt, off, o, _workspace(m.MOE_MM_ROWS, T, N, K, G))
    ref, mag = P.grouped(last(x), wt[2:], [0, L])
    P.assert_within(o[-L:], ref, (K + 4) * P.EPS32 * mag, "product")
    xq, xs = torch.empty(T, K, dtype=E4M3, device="cuda"), torch.empty(T, -(-K // 128), device="cuda")
    xq2, xs2 = torch.empty(L, K, dtype=E4M3, device="cuda"), torch.empty(L, -(-K // 128), device="cuda")
    m.moe_fp8_quant_rows(x, xq, xs)
    m.moe_fp8_quant_rows(last(x), xq2, xs2)
    assert torch.equal(xq[-L:].view(torch.uint8), xq2.view(torch.uint8)) and torch.equal(xs[-L:], xs2)


# tiles of 64, 128 and 256 columns, and a reduction in pieces
@pytest.mark.parametrize("R,N,K", [(70, 200, 700), (600, 1100, 640), (2500, 2100, 700), (4100, 2100, 300), (16, 300, 4200)])
@pytest.mark.parametrize("swap", [False, True])
def test_fp8_mm_scales_whose_product_leaves_fp32(R, N, K, swap):
    """Two scales whose product overflows, over a block of zeros, and two whose product is subnormal, over a block whose
    sum times them is not. The other rows keep their bits."""
    cuda_device()
    g = _gen(R)
    kb, nb = -(-K // 128), -(-N // 128)
    big, less, small, tiny = (1e4, 1e35, 1e-16, 1e-27) if swap else (1e35, 1e4, 1e-27, 1e-16)
    xq, _ = P.strided(_randn(g, R, K, std=100.0).abs().clamp(max=448.0).to(E4M3), 0, whole=16)
    wq, _ = P.strided(_randn(g, 1, N, K, std=100.0).abs().clamp(max=448.0).to(E4M3), 0, whole=16)
    xs, wsc = torch.rand(R, kb, generator=g, device="cuda") + 0.5, torch.rand(1, nb, kb, generator=g, device="cuda") + 0.5
    wq[:, :, 128:256] = 0
    wsc[:, :, 1] = less
    wsc[:, -1] = tiny
    wsc[:, -1, 1] = less
    plain = xs.clone()
    xs[::3, 1] = big                  # next to ordinary blocks
    xs[1::3] *= small                 # every block of the row
    out, out2 = torch.empty(R, N, device="cuda"), torch.empty(R, N, device="cuda")
    ws = _workspace(m.MOE_MM_FP8, R, N, K, 1)
    m.moe_fp8_mm(xq, xs, wq, wsc, out, ws)
    m.moe_fp8_mm(xq, plain, wq, wsc, out2, ws)
    x64 = P.decode(xq) * xs.double().repeat_interleave(128, 1)[:, :K]
    w64 = P.decode(wq) * wsc.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]
    ref, mag = P.grouped(x64, w64, [0, R])
    P.assert_within(out, ref, (K + 8) * P.EPS32 * mag, "out")
    assert torch.equal(out[2::3], out2[2::3])
    assert torch.equal(out[::3, :(nb - 1) * 128], out2[::3, :(nb - 1) * 128])

def test_fp8_quant_weights_groups_behind_the_last_row():
    """Groups that begin right behind the last row's elements, as the products take them: w, q and qt."""
    cuda_device()
    g = _gen(12)
    G, N, K, ld = 3, 40, 144, 160
    gs = (N - 1) * ld + K                      # N ld would be 16 more
    w = torch.as_strided(_randn(g, G * gs, dtype=BF16), (G, N, K), (gs, ld, 1))
    q = torch.as_strided(torch.zeros(G * gs, dtype=torch.uint8, device="cuda"), (G, N, K), (gs, ld, 1))
    ldt = 64
    gt = (K - 1) * ldt + N
    qt = torch.as_strided(torch.zeros(G * gt, dtype=torch.uint8, device="cuda"), (G, K, N), (gt, ldt, 1))
    s, st = torch.empty(G, 1, 2, device="cuda"), torch.empty(G, 2, 1, device="cuda")
    m.moe_fp8_quant_weights(w, q, s, qt, st)
    q2, s2 = torch.empty(G, N, K, dtype=torch.uint8, device="cuda"), torch.empty_like(s)
    m.moe_fp8_quant_weights(w.contiguous(), q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2) and torch.equal(qt, q2.transpose(1, 2)) and torch.equal(st, s.transpose(1, 2))
    R = 50
    xq, xs = torch.empty(R, K, dtype=torch.uint8, device="cuda"), torch.empty(R, 2, device="cuda")
    m.moe_fp8_quant_rows(_randn(g, R, K, dtype=BF16), xq, xs)
    off, offsets = _offsets([20, 0, 30])
    y, y2 = torch.empty(R, N, device="cuda"), torch.empty(R, N, device="cuda")
    m.moe_fp8_mm(xq, xs, q, s, y, _workspace(m.MOE_MM_FP8, R, N, K, G), offsets=offsets)
    m.moe_fp8_mm(xq, xs, q2, s2, y2, _workspace(m.MOE_MM_FP8, R, N, K, G), offsets=offsets)
    assert torch.equal(y, y2)

# ---- both sides of the rules that pick a kernel ------------------------------------------
# Sizes in rows an SM, as the rules count them, so that they follow the machine.
def _rows(per_sm, more):
    return per_sm * torch.cuda.get_device_properties(0).multi_processor_count + more


def _check_norm_forward(x, gamma, beta, eps, y, mean, rstd):
    """The bounds of test_layer_norm."""
    H = x.shape[1]
    ry, rm, rr = P.norm_fwd(x, gamma, beta, eps)
    dmean = (H + 4) * P.EPS32 * x.double().abs().mean(1)
    P.assert_within(mean, rm, dmean, "mean")
    rel = (H + 8) * P.EPS32 + (dmean * rr) ** 2
    P.assert_within(rstd, rr, rr * rel, "rstd")
    c = (x.double() - rm[:, None]).abs() * rr[:, None]
    gm = 1.0 if gamma is None else gamma.double().abs()
    b = 0.0 if beta is None else beta.double().abs()
    P.assert_within(y, ry, (c * (rel[:, None] + 4 * P.EPS32) + (dmean * rr)[:, None]) * gm + 2 * P.EPS32 * b, "y")


def _check_norm_dx(dy, x, gamma, mean, rstd, dx):
    """The bounds of test_layer_norm."""
    H = x.shape[1]
    xh = (x.double() - mean.double()[:, None]).abs() * rstd.double()[:, None]
    t = dy.double().abs() * (1.0 if gamma is None else gamma.double().abs())
    b = rstd.double()[:, None] * (4 * P.EPS32 * t + (H + 4) * P.EPS32 * t.mean(1, keepdim=True) +
                                  (H + 8) * P.EPS32 * xh * (t * xh).mean(1, keepdim=True))
    P.assert_within(dx, P.norm_bwd(dy, x, gamma, mean, rstd)[0], b, "dx")


# aligned 16-bit forward: rows run ahead in shared memory from 48 rows an SM and H > 2048 on; one, two and four packs a
# thread, the last CTA's rows even and odd in number
@pytest.mark.parametrize("more", [-1, 0, 1, 333])
@pytest.mark.parametrize("H", [2048, 2056, 2880, 4096, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (F16, F16)])
def test_layer_norm_forward_of_a_training_batch(more, H, dtype, wdtype):
    cuda_device()
    T, g = _rows(48, more), _gen(H + more)
    x = _randn(g, T, H, dtype=dtype, std=2.0) + 0.5
    gamma, beta = (_randn(g, H) * 0.3 + 1).to(wdtype), _randn(g, H).to(wdtype)
    y, ybuf = P.strided(torch.zeros(T, H, dtype=dtype, device="cuda"), 8)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    m.moe_layer_norm_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _check_norm_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _canary(ybuf, H, "y")
    y2 = torch.empty(T, H, dtype=dtype, device="cuda")
    m.moe_layer_norm_forward(x, gamma, beta, 1e-5, y2)
    assert torch.equal(y2, y)


# off a boundary: fp32 forward runs rows ahead from 4 rows an SM on, any backward from half a row an SM on
@pytest.mark.parametrize("per_sm,more", [(0, 40), (1, 1), (4, -1), (4, 1), (9, 5)])
@pytest.mark.parametrize("H,lead", [(301, 1), (1031, 3), (520, 1), (4099, 2), (2881, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layer_norm_of_tensors_off_a_boundary(per_sm, more, H, lead, dtype):
    """Tensors that begin and end inside 16-byte units: their neighbours in memory are NaN, stay unread and unwritten."""
    cuda_device()
    T, g = _rows(per_sm, more), _gen(H + more)

    def inside(std):
        buf = torch.full((T * H + 16,), NAN, dtype=dtype, device="cuda")
        t = buf[lead:lead + T * H].view(T, H)
        t.copy_(_randn(g, T, H, std=std))
        return t, buf

    def untouched(buf, what):
        assert bool(torch.isnan(buf[:lead]).all()) and bool(torch.isnan(buf[lead + T * H:]).all()), what

    (x, _), (dy, _), (y, ybuf), (dx, dxbuf) = inside(2.0), inside(1.0), inside(0.0), inside(0.0)
    gamma, beta = _randn(g, H) * 0.3 + 1, _randn(g, H)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    m.moe_layer_norm_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _check_norm_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    dgamma, dbeta = torch.full_like(gamma, NAN), torch.full_like(beta, NAN)
    ws = torch.empty(m.moe_layer_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    m.moe_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws)
    _check_norm_dx(dy, x, gamma, mean, rstd, dx)
    _, rdg, rdb = P.norm_bwd(dy, x, gamma, mean, rstd)
    xh = (x.double() - mean.double()[:, None]).abs() * rstd.double()[:, None]
    P.assert_within(dgamma, rdg, (T + 4) * P.EPS32 * (dy.double().abs() * xh).sum(0), "dgamma")
    P.assert_within(dbeta, rdb, (T + 4) * P.EPS32 * dy.double().abs().sum(0), "dbeta")
    untouched(ybuf, "y")
    untouched(dxbuf, "dx")


# odd alignments, a warp a row from 96 rows an SM on: rows of two blocks (two quarter-warps a row), of three (one, three
# rounds), of four and of sixteen (four quarter-warps a row)
@pytest.mark.parametrize("more", [-1, 1])
@pytest.mark.parametrize("I,act,dtype,pad", [(129, "swiglu", BF16, 0), (255, "srelu", F16, 8), (200, "geglu", BF16, 3),
                                             (383, "swiglu", F16, 0), (511, "swiglu_clamp", BF16, 0),
                                             (512, "swiglu", F16, 3), (2047, "swiglu", BF16, 0)])
def test_activation_checkpoint_a_warp_a_row(more, I, act, dtype, pad):
    test_activation_checkpoint(_rows(96, more), I, act, dtype, pad)


def _needs_gb(n):
    cuda_device()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < n << 30:
        pytest.skip(f"needs {n} GB")


@pytest.mark.parametrize("H", [2880, 2881])
def test_layer_norm_elements_past_32_bits(H):
    """More than 2^31 elements: the last rows, and the sums over all rows."""
    _needs_gb(40)
    g, T, L = _gen(H), 2 ** 31 // H + 3001, 70
    x = torch.empty(T, H, dtype=BF16, device="cuda").normal_(generator=g)
    gamma, beta = _randn(g, H), _randn(g, H)
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    m.moe_layer_norm_forward(x, gamma, beta, 1e-5, y, mean, rstd)
    _check_norm_forward(x[-L:], gamma, beta, 1e-5, y[-L:], mean[-L:], rstd[-L:])
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    ws = torch.empty(m.moe_layer_norm_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    m.moe_layer_norm_backward(y, x, gamma, mean, rstd, dx, dgamma, dbeta, ws)
    _check_norm_dx(y[-L:], x[-L:], gamma, mean[-L:], rstd[-L:], dx[-L:])
    ref = [torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(4)]
    for a in range(0, T, 50000):
        d = y[a:a + 50000].double()
        xh = (x[a:a + 50000].double() - mean[a:a + 50000, None]) * rstd[a:a + 50000, None]
        for r, v in zip(ref, (d * xh, d, (d * xh).abs(), d.abs())):
            r += v.sum(0)
    P.assert_within(dgamma, ref[0], (T + 4) * P.EPS32 * ref[2], "dgamma")
    P.assert_within(dbeta, ref[1], (T + 4) * P.EPS32 * ref[3], "dbeta")


def test_weight_gradient_elements_past_32_bits():
    """More than 2^31 elements of rows, and of gradients."""
    _needs_gb(30)
    g = _gen(41)
    N, K = 64, 5776
    R = 2 ** 31 // K + 1001
    off, offsets = _offsets([R - 3000, 0, 3000])
    dy, x = _randn(g, R, N, dtype=BF16), torch.empty(R, K, dtype=BF16, device="cuda").normal_(generator=g)
    dw = torch.full((3, N, K), NAN, device="cuda")
    m.moe_grouped_mm_wgrad(dy, x, offsets, dw, _workspace(m.MOE_MM_WGRAD, R, N, K, 3))
    ref, mag = P.grouped_wgrad(dy[-3000:], x[-3000:], [0, 3000])
    P.assert_within(dw[2], ref[0], (3000 + 4) * P.EPS32 * mag[0], "last group")
    assert bool((dw[1] == 0).all())
    ref, mag = torch.zeros(N, K, dtype=torch.float64, device="cuda"), torch.zeros(N, K, dtype=torch.float64, device="cuda")
    for a in range(0, R - 3000, 50000):
        s = slice(a, min(a + 50000, R - 3000))
        r, v = P.grouped_wgrad(dy[s], x[s], [0, s.stop - s.start])
        ref += r[0]
        mag += v[0]
    P.assert_within(dw[0], ref, (R + 4) * P.EPS32 * mag, "first group")
    del x, dw
    N = K = 5632
    G = 2 ** 31 // (N * K) + 2
    off, offsets = _offsets([5] * G)
    dy, x = _randn(g, 5 * G, N, dtype=BF16), _randn(g, 5 * G, K, dtype=BF16)
    dw = torch.empty(G, N, K, dtype=BF16, device="cuda")
    m.moe_grouped_mm_wgrad(dy, x, offsets, dw, _workspace(m.MOE_MM_WGRAD, 5 * G, N, K, G))
    ref, mag = P.grouped_wgrad(dy[-5:], x[-5:], [0, 5])
    P.assert_within(dw[-1], ref[0], 9 * P.EPS32 * mag[0], "last gradient")


def test_fp8_elements_past_32_bits():
    """More than 2^31 elements of weights, with their transposed copy, and of rows: the quantisers and the products."""
    _needs_gb(30)
    g = _gen(42)
    N, K = 5640, 5632
    G = 2 ** 31 // (N * K) + 2
    w = torch.empty(G, N, K, dtype=BF16, device="cuda").normal_(0.0, 0.05, generator=g)
    nb, kb = -(-N // 128), -(-K // 128)
    q, s = torch.empty(G, N, K, dtype=E4M3, device="cuda"), torch.empty(G, nb, kb, device="cuda")
    ld = -(-N // 16) * 16
    qt = torch.zeros(G, K, ld, dtype=E4M3, device="cuda")[:, :, :N]
    st = torch.empty(G, kb, nb, device="cuda")
    m.moe_fp8_quant_weights(w, q, s, qt, st)
    q1, s1 = torch.empty(1, N, K, dtype=E4M3, device="cuda"), torch.empty(1, nb, kb, device="cuda")
    m.moe_fp8_quant_weights(w[-1:].clone(), q1, s1)
    assert torch.equal(q[-1:].view(torch.uint8), q1.view(torch.uint8)) and torch.equal(s[-1:], s1)
    assert torch.equal(qt[-1].view(torch.uint8), q1[0].view(torch.uint8).t()) and torch.equal(st[-1], s1[0].t())
    del w
    R = 300
    off, offsets = _offsets([0] * (G - 1) + [R])
    x = _randn(g, R, K, dtype=BF16)
    xq, xs = torch.empty(R, K, dtype=E4M3, device="cuda"), torch.empty(R, kb, device="cuda")
    m.moe_fp8_quant_rows(x, xq, xs)

    def value(q, s):
        return P.decode(q) * s.double().repeat_interleave(128, 1)[:, :q.shape[1]]

    def weight(q, s):
        return P.decode(q) * s.double().repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]

    out = torch.empty(R, N, device="cuda")
    m.moe_fp8_mm(xq, xs, q, s, out, _workspace(m.MOE_MM_FP8, R, N, K, G), offsets=offsets)
    ref, mag = P.grouped(value(xq, xs), weight(q[-1], s[-1])[None], [0, R])
    P.assert_within(out, ref, (K + 8) * P.EPS32 * mag, "the last group's weights")
    del q, qt
    N, L = 64, 70
    R = 2 ** 31 // K + 301
    xq = torch.randint(0, 0x7F, (R, K), dtype=torch.uint8, device="cuda", generator=g).view(E4M3)
    xs = torch.rand(R, kb, device="cuda", generator=g)
    wq, ws = q1[:, :N].contiguous(), s1[:, :1].contiguous()
    out = torch.empty(R, N, device="cuda")
    m.moe_fp8_mm(xq, xs, wq, ws, out, _workspace(m.MOE_MM_FP8, R, N, K, 1))
    ref, mag = P.grouped(value(xq[-L:], xs[-L:]), weight(wq[0], ws[0])[None], [0, L])
    P.assert_within(out[-L:], ref, (K + 8) * P.EPS32 * mag, "the last rows")
