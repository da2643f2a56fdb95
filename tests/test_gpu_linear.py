"""The dense product with bias, activation and residual on the GPU, forward and
backward, against its 64-bit form."""
import math

import pytest
import torch

import dense_ref as D
import ops_ref as P
import quantized_grouped_gemm_topk_gb300 as m

from util import cuda_device

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAN = float("nan")
ALPHA, LIMIT = 1.702, 2.0


def _gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _rows(g, r, c, dtype, std=1.0, pad=0):
    """Rows that tensor copies take: a stride of a multiple of 8 elements, NaN behind each row."""
    return P.strided(_randn(g, r, c, dtype=dtype, std=std), pad, whole=8)[0]


def _ws(R, rows, K, backward=False):
    return torch.zeros(m.moe_linear_workspace_size(R, rows, K, backward), dtype=torch.uint8, device="cuda")


def _canary(buf, cols, what):
    assert bool(torch.isnan(buf[..., cols:].float()).all()), f"{what}: wrote past its rows"


def _forward(R, N, K, act, dtype, wdtype=F32, bias=True, residual=True, save=True, pad=0, seed=0):
    cuda_device()
    g = _gen(seed + R * 7 + N * 3 + K)
    rows = D.halves(act) * N
    x, w = _rows(g, R, K, dtype, pad=8 if pad else 0), _rows(g, rows, K, dtype, std=1.5 * K ** -0.5)
    b = _randn(g, rows, dtype=wdtype, std=0.3) if bias else None
    res = P.strided(_randn(g, R, N, dtype=dtype), pad)[0] if residual else None
    out, obuf = P.strided(torch.zeros(R, N, dtype=dtype, device="cuda"), pad)
    z, zbuf = P.strided(torch.zeros(R, rows, dtype=dtype, device="cuda"), pad) if save else (None, None)
    ws = _ws(R, rows, K)
    m.moe_linear_forward(x, w, out, ws, bias=b, residual=res, z=z, act=act, alpha=ALPHA, limit=LIMIT)
    ro, bo, rz, bz = D.linear(x, w, b, res, act, ALPHA, LIMIT)
    P.assert_within(out, ro, bo, "out")
    if save:
        P.assert_within(z, rz, bz, "z")
        if pad:
            _canary(zbuf, rows, "z")
    if pad:
        _canary(obuf, N, "out")
    assert m.moe_mm_read_status(ws) == 0
    return x, w, b, res, out, z, ws


SIZES = [(1, 1, 1), (1, 7168, 72), (3, 40, 129), (16, 130, 2048), (17, 64, 64), (64, 264, 200), (65, 257, 1000), (128, 72, 640),
         (130, 520, 96), (200, 1031, 333), (257, 256, 2049), (700, 100, 65), (1100, 640, 128)]


@pytest.mark.parametrize("R,N,K", SIZES)
@pytest.mark.parametrize("act", D.ACTS)
def test_linear_forward(R, N, K, act):
    _forward(R, N, K, act, BF16)


@pytest.mark.parametrize("R,N,K", SIZES)
@pytest.mark.parametrize("act", ["none", "gelu", "swiglu", "geglu"])
@pytest.mark.parametrize("kw", [dict(dtype=F16, wdtype=F16, pad=3), dict(dtype=F16, bias=False, residual=False, save=False, pad=8),
                                dict(dtype=BF16, wdtype=BF16, residual=False, pad=1), dict(dtype=BF16, bias=False, save=False)],
                         ids=["f16-all", "f16-bare", "bf16-bias-z", "bf16-residual"])
def test_linear_forward_options(R, N, K, act, kw):
    _forward(R, N, K, act, **kw)


@pytest.mark.parametrize("R,N,K", [(1, 4096, 7168), (8, 7168, 2048), (33, 2880, 2880), (64, 2048, 4096), (300, 2880, 1000),
                                   (4096, 512, 96), (2500, 2880, 200), (5001, 1100, 520), (1, 40000, 64)])
@pytest.mark.parametrize("act", ["none", "swiglu_clamp", "silu"])
def test_linear_forward_of_many_tiles(R, N, K, act):
    _forward(R, N, K, act, BF16, residual=act == "none", save=act != "none")


@pytest.mark.parametrize("act", ["gelu", "silu", "geglu"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("R", [1, 300])
def test_linear_activation_over_its_range(act, dtype, R):
    """z = w (x and K are one): every value of the type from -14 to 14 in steps, and the smallest, through the activation and
    its derivative; relative to the result, which is tiny on the left."""
    cuda_device()
    v = torch.cat([torch.linspace(-14, 14, 5000), torch.logspace(-4, 1, 300), -torch.logspace(-4, 1, 300)]).to("cuda", dtype)
    n = v.numel()
    rows = D.halves(act) * n
    w = torch.zeros(rows, 8, dtype=dtype, device="cuda")[:, :1]
    w[:n, 0] = v
    if rows > n:
        w[n:, 0] = 1
    x = torch.ones(R, 8, dtype=dtype, device="cuda")[:, :1]
    out, z = torch.empty(R, n, dtype=dtype, device="cuda"), torch.empty(R, rows, dtype=dtype, device="cuda")
    m.moe_linear_forward(x, w, out, _ws(R, rows, 1), z=z, act=act)
    ro, bo, rz, _ = D.linear(x, w, None, None, act, 1.0, 0.0)
    assert torch.equal(z.double(), rz)
    val, err, _, _, _ = D.act(rz.chunk(D.halves(act), 1), act)       # z is exact: the activation's error alone
    P.assert_within(out, val, err, "out")
    dz = torch.empty_like(z)
    m.moe_linear_backward(torch.ones_like(out), x, w, z, dz, None, None, None, _ws(R, rows, 1, True), act=act)
    rdz, bdz = D.linear_dz(torch.ones_like(out), z, act, 1.0, 0.0)
    P.assert_within(dz, rdz, bdz, "dz")


# both sides of the rules that pick a kernel: rows times weight rows against 256 times the reduction (65 to 256 rows); backward:
# a reduction from 2048 on with fewer than 40 tiles of 256 x 128
@pytest.mark.parametrize("R,N,K", [(64, 520, 64), (65, 520, 128), (65, 520, 136), (256, 256, 256), (256, 248, 256), (255, 1000, 1000),
                                   (250, 130, 2500), (130, 40, 70000), (2, 8, 70000), (256, 2056, 2048)])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_forward_on_both_sides_of_the_rule(R, N, K, act):
    _forward(R, N, K, act, BF16)


@pytest.mark.parametrize("R,N,K", [(2047, 264, 136), (2048, 264, 136), (40, 2048, 264), (40, 2040, 264), (2304, 600, 1280), (2300, 1300, 1300),
                                   (600, 2100, 1300)])
@pytest.mark.parametrize("act", ["none", "silu", "geglu"])
def test_linear_backward_on_both_sides_of_the_rule(R, N, K, act):
    _backward(R, N, K, act, BF16)


def test_linear_residual_in_place_and_repeatable():
    cuda_device()
    for R in (5, 90, 700):
        x, w, b, res, out, _, ws = _forward(R, 328, 520, "none", BF16, save=False)
        again = torch.empty_like(out)
        m.moe_linear_forward(x, w, again, ws, bias=b, residual=res)
        assert torch.equal(again, out)
        m.moe_linear_forward(x, w, res, ws, bias=b, residual=res)
        assert torch.equal(res, out)


def test_linear_nan_and_infinity_stay_in_their_row():
    cuda_device()
    g = _gen(3)
    for R, N, K, act in ((9, 96, 200, "swiglu"), (9, 96, 200, "swiglu_clamp"), (9, 96, 200, "srelu"), (300, 200, 136, "gelu"),
                         (300, 200, 136, "swiglu_clamp"), (300, 200, 136, "none")):
        x, w = _rows(g, R, K, BF16), _rows(g, D.halves(act) * N, K, BF16, std=K ** -0.5)
        ws = _ws(R, D.halves(act) * N, K)
        want, out = (torch.empty(R, N, dtype=BF16, device="cuda") for _ in range(2))
        m.moe_linear_forward(x, w, want, ws, act=act, alpha=ALPHA, limit=LIMIT)
        bad = x.clone()
        bad[4, K - 1] = NAN
        bad[7, 0] = math.inf
        m.moe_linear_forward(torch.nn.functional.pad(bad, (0, 8 - K % 8 if K % 8 else 0))[:, :K], w, out, ws, act=act, alpha=ALPHA,
                             limit=LIMIT)
        keep = [r for r in range(R) if r not in (4, 7)]
        assert torch.equal(out[keep], want[keep])
        assert bool(torch.isnan(out[4].float()).all())


def _backward(R, N, K, act, dtype, wdtype=F32, pad=0):
    cuda_device()
    g = _gen(R * 5 + N + K * 3)
    rows = D.halves(act) * N
    x, w = _rows(g, R, K, dtype), _rows(g, rows, K, dtype, std=K ** -0.5)
    plain = act == "none"
    dout = _rows(g, R, N, dtype) if plain else P.strided(_randn(g, R, N, dtype=dtype), pad)[0]
    z = None if plain else P.strided(_randn(g, R, rows, dtype=dtype, std=1.5), pad)[0]
    dz, zbuf = (None, None) if plain else P.strided(torch.zeros(R, rows, dtype=dtype, device="cuda"), pad and 8, whole=8)
    dx, xbuf = P.strided(torch.zeros(R, K, dtype=dtype, device="cuda"), pad)
    dw, wbuf = P.strided(torch.zeros(rows, K, dtype=dtype, device="cuda"), pad)
    db = torch.full((rows,), NAN, dtype=wdtype, device="cuda")
    ws = _ws(R, rows, K, True)
    m.moe_linear_backward(dout, x, w, z, dz, dx, dw, db, ws, act=act, alpha=ALPHA, limit=LIMIT)
    rz, bz = D.linear_dz(dout, z, act, ALPHA, LIMIT)
    if not plain:
        P.assert_within(dz, rz, bz, "dz")
        if pad:
            _canary(zbuf, rows, "dz")
    P.assert_within(db, rz.sum(0), bz.sum(0) + (R + 8) * P.EPS32 * (rz.abs() + bz).sum(0), "db")
    # the products, of dz as it was rounded
    d = dout.double() if plain else dz.double()
    P.assert_within(dx, d @ w.double(), (rows + 8) * P.EPS32 * (d.abs() @ w.double().abs()), "dx")
    P.assert_within(dw, d.t() @ x.double(), (R + 8) * P.EPS32 * (d.abs().t() @ x.double().abs()), "dw")
    if pad:
        _canary(xbuf, K, "dx")
        _canary(wbuf, K, "dw")
    assert m.moe_mm_read_status(ws) == 0
    return x, w, dout, z, dz, dx, dw, db, ws


BACK = [(1, 1, 1), (1, 264, 72), (3, 40, 129), (64, 264, 200), (130, 257, 1000), (257, 256, 640), (700, 100, 65), (1100, 640, 128)]


@pytest.mark.parametrize("R,N,K", BACK)
@pytest.mark.parametrize("act", D.ACTS)
@pytest.mark.parametrize("dtype,wdtype,pad", [(BF16, F32, 0), (F16, F16, 3)])
def test_linear_backward(R, N, K, act, dtype, wdtype, pad):
    _backward(R, N, K, act, dtype, wdtype, pad)


@pytest.mark.parametrize("R,N,K", [(16384, 128, 96), (4096, 1440, 720), (2051, 2881, 264)])
@pytest.mark.parametrize("act", ["none", "swiglu", "gelu"])
def test_linear_backward_of_many_rows(R, N, K, act):
    _backward(R, N, K, act, BF16)


def test_linear_backward_parts_and_repeatable():
    """Each gradient alone has the same bits as all together, and as again."""
    x, w, dout, z, dz, dx, dw, db, ws = _backward(333, 200, 264, "swiglu", BF16)
    kw = dict(act="swiglu", alpha=ALPHA, limit=LIMIT)
    for i in range(3):
        got = [torch.full_like(t, NAN) for t in (dx, dw, db)]
        m.moe_linear_backward(dout, x, w, z, torch.empty_like(dz), *[t if i == j else None for j, t in enumerate(got)], ws, **kw)
        assert torch.equal(got[i], (dx, dw, db)[i])
        assert all(bool(torch.isnan(got[j].float()).all()) for j in range(3) if j != i)


def test_linear_no_rows():
    cuda_device()
    w = torch.randn(48, 64, device="cuda").to(BF16)
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    ws = _ws(0, 48, 64)
    m.moe_linear_forward(x, w, torch.empty(0, 24, dtype=BF16, device="cuda"), ws, act="swiglu")
    dw, db = torch.full((48, 64), NAN, dtype=BF16, device="cuda"), torch.full((48,), NAN, device="cuda")
    z = torch.empty(0, 48, dtype=BF16, device="cuda")
    m.moe_linear_backward(z[:, :24], x, w, z, z.clone(), x.clone(), dw, db, _ws(0, 48, 64, True), act="swiglu")
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("act", D.ACTS)
def test_linear_gradient_by_differences(act):
    """dx, dw and db of L = sum(c out) against central differences of the 64-bit forward."""
    cuda_device()
    g = _gen(11)
    R, N, K = 5, 24, 40
    rows = D.halves(act) * N
    x, w, b = _rows(g, R, K, F16), _rows(g, rows, K, F16, std=K ** -0.5), _randn(g, rows, std=0.2)
    c = _randn(g, R, N, dtype=F16)
    out, z = torch.empty(R, N, dtype=F16, device="cuda"), torch.empty(R, rows, dtype=F16, device="cuda")
    m.moe_linear_forward(x, w, out, _ws(R, rows, K), bias=b, z=z, act=act, alpha=ALPHA, limit=LIMIT)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    plain = act == "none"
    m.moe_linear_backward(c, x, w, None if plain else z, None if plain else torch.empty_like(z), dx, dw, db, _ws(R, rows, K, True),
                          act=act, alpha=ALPHA, limit=LIMIT)

    def loss(x_, w_, b_):
        return (c.double() * D.linear(x_, w_, b_, None, act, ALPHA, LIMIT)[0]).sum()

    args = [x.double(), w.double(), b.double()]
    if act in ("swiglu_clamp", "srelu"):       # away from the corners, where the difference means nothing
        zz = D.product(*args)[0]
        edge = zz.abs() if act == "srelu" else (zz.abs() - LIMIT).abs()
        assert float(edge.min()) > 1e-5
    h = 1e-6
    # z in 16 bits shifts the derivative by |act''| 2^-11 |z|, dz's rounding by 2^-11: of |c| (1 + |z|^2) at most, summed
    zz = D.product(*args)[0].abs()
    wide = (c.double().abs().repeat(1, D.halves(act)) * (2 + zz) ** 2 * 4 * 2.0 ** -11) * (1 + zz.max())
    bounds = [wide @ w.double().abs(), wide.t() @ x.double().abs(), wide.sum(0)]
    for i, got in enumerate((dx, dw, db)):
        flat = args[i].flatten()
        for at in range(0, flat.numel(), max(1, flat.numel() // 40)):
            lo, hi = args[i].clone().flatten(), args[i].clone().flatten()
            lo[at] -= h
            hi[at] += h
            diff = [loss(*[v.view_as(args[i]) if j == i else args[j] for j in range(3)]) for v in (lo, hi)]
            want = float(diff[1] - diff[0]) / (2 * h)
            lim = float(bounds[i].flatten()[at]) + 1e-4 + 2.0 ** -11 * abs(want)
            assert abs(float(got.flatten()[at]) - want) <= lim, (act, i, at)


def test_linear_on_another_stream_and_in_graphs_that_share_a_workspace():
    cuda_device()
    g = _gen(5)
    N, K = 328, 640
    ws = _ws(400, 2 * N, K)
    sets = []
    for R in (7, 400):
        x, w = _rows(g, R, K, BF16), _rows(g, 2 * N, K, BF16, std=K ** -0.5)
        want, out = torch.empty(R, N, dtype=BF16, device="cuda"), torch.zeros(R, N, dtype=BF16, device="cuda")
        m.moe_linear_forward(x, w, want, ws, act="swiglu")
        sets.append((x, w, want, out))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x, w, want, out in sets:
            m.moe_linear_forward(x, w, out, ws, act="swiglu")
    side.synchronize()
    graphs = []
    for x, w, want, out in sets:
        assert torch.equal(out, want)
        out.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.moe_linear_forward(x, w, out, ws, act="swiglu")
        graphs.append(graph)
    for _ in range(3):
        for graph, (x, w, want, out) in zip(graphs, sets):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_linear_backward_on_another_stream_and_in_graphs_that_share_a_workspace():
    """Sizes whose products take different kernels, their partial sums in the same places."""
    cuda_device()
    sizes = ((20, 2048, 264, "silu"), (2100, 300, 136, "swiglu"), (700, 520, 640, "none"))
    ws = torch.zeros(max(m.moe_linear_workspace_size(R, D.halves(act) * N, K, True) for R, N, K, act in sizes), dtype=torch.uint8,
                     device="cuda")
    sets, graphs = [], []
    for R, N, K, act in sizes:
        x, w, dout, z, dz, *want, _ = _backward(R, N, K, act, BF16)
        sets.append(((dout, x, w, z, dz), want, [torch.zeros_like(t) for t in want], act))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def each(i):
        args, want, got, act = sets[i]
        for t in got:
            t.fill_(NAN)
        yield
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))

    def call(i):
        args, _, got, act = sets[i]
        m.moe_linear_backward(*args, *got, ws, act=act, alpha=ALPHA, limit=LIMIT)

    for i in range(len(sets)):
        for _ in each(i):
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                call(i)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(i)
        graphs.append(graph)
    for _ in range(2):
        for i, graph in enumerate(graphs):
            for _ in each(i):
                graph.replay()
            for _ in each(i):
                call(i)


def _needs_gb(n):
    if torch.cuda.get_device_properties(0).total_memory < n << 30:
        pytest.skip(f"needs {n} GB")


@pytest.mark.parametrize("R", [33, 600])
def test_linear_elements_past_32_bits(R):
    """Rows so far apart that the last one's offset passes 2^31 elements, of x, residual, z and out."""
    cuda_device()
    _needs_gb(60)
    g = _gen(8)
    N, K = 48, 64
    ld = (2 ** 31 // (R - 1) + 64) // 8 * 8
    buf = torch.zeros(R, ld, dtype=BF16, device="cuda")
    obuf, zbuf = torch.zeros_like(buf), torch.zeros_like(buf)
    x = buf[:, :K]
    x.copy_(_randn(g, R, K))
    res = buf[:, K:K + N]
    res.copy_(_randn(g, R, N))
    w = _rows(g, 2 * N, K, BF16, std=K ** -0.5)
    m.moe_linear_forward(x, w, obuf[:, :N], _ws(R, 2 * N, K), residual=res, z=zbuf[:, :2 * N], act="swiglu")
    ro, bo, rz, bz = D.linear(x, w, None, res, "swiglu", ALPHA, LIMIT)
    P.assert_within(obuf[:, :N], ro, bo, "out")
    P.assert_within(zbuf[:, :2 * N], rz, bz, "z")
    obuf[:, N:N + 96].zero_()
    dz = obuf[:, N:N + 2 * N]
    dx = zbuf[:, 128:128 + K]
    dw, db = torch.empty_like(w), torch.empty(2 * N, device="cuda")
    if N % 8 == 0:
        m.moe_linear_backward(res, x, w, zbuf[:, :2 * N], dz, dx, dw, db, _ws(R, 2 * N, K, True), act="swiglu")
        d = dz.double()
        rdz, bdz = D.linear_dz(res, zbuf[:, :2 * N], "swiglu", ALPHA, LIMIT)
        P.assert_within(dz, rdz, bdz, "dz")
        P.assert_within(dx, d @ w.double(), (2 * N + 8) * P.EPS32 * (d.abs() @ w.double().abs()), "dx")


@pytest.mark.parametrize("act", [a for a in D.ACTS if a != "none"])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_linear_derivative_by_differences(act, dtype):
    """dz against central differences of the activation alone, in 64 bits at the very z that the kernel reads: only dz's
    own rounding and the kernel's error are between the two. A derivative that lacks a term is outside."""
    cuda_device()
    g = _gen(12)
    R, N = 37, 200
    hv = D.halves(act)
    z, d = _randn(g, R, hv * N, dtype=dtype, std=1.5), _randn(g, R, N, dtype=dtype)
    x, w = _rows(g, R, 8, dtype), _rows(g, hv * N, 8, dtype)
    dz = torch.empty_like(z)
    m.moe_linear_backward(d, x, w, z, dz, None, None, None, _ws(R, hv * N, 8, True), act=act, alpha=ALPHA, limit=LIMIT)
    h = 1e-4
    zs = list(z.double().chunk(hv, 1))
    bound = D.linear_dz(d, z, act, ALPHA, LIMIT)[1].chunk(hv, 1)
    for i, got in enumerate(dz.chunk(hv, 1)):
        f = [D.act([v + s * h if j == i else v for j, v in enumerate(zs)], act, ALPHA, LIMIT)[0] for s in (1, -1)]
        want = d.double() * (f[0] - f[1]) / (2 * h)
        # the difference's own error: h^2 / 6 of a third derivative below 4 (1 + |other half|), at srelu's corner h
        other = 1 + (zs[1 - i].abs() if hv == 2 else 0)
        lim = bound[i] + d.double().abs() * other * (4 * h * h + (h if act == "srelu" else 0))
        lim = lim + P.HALF_STEP[dtype] * (want.abs() + lim) + P.TINY[dtype]
        smooth = torch.ones_like(want, dtype=torch.bool)
        if act == "swiglu_clamp":         # a corner has no difference
            smooth = (zs[i].abs() - LIMIT).abs() > 2 * h
        assert float(smooth.double().mean()) > 0.95
        assert bool(((got.double() - want).abs() <= lim)[smooth].all()), (act, i)
        # without f's own slope in v s(v), or without the derivative at all
        live = smooth & (want != 0)
        value = D.act(zs, act, ALPHA, LIMIT)[0]
        less = want / 2 if act == "srelu" else d.double() * value / zs[0] if i == 0 else d.double() * value / zs[1] * 0.5
        for wrong in (less, want * 0):
            assert float(((wrong - want).abs() > lim)[live].double().mean()) > 0.9, (act, i)


@pytest.mark.parametrize("R,N,K,act", [(300, 200, 136, "silu"), (300, 200, 136, "swiglu"), (300, 200, 136, "swiglu_clamp"), (40, 2048, 264, "gelu"),
                                       (2304, 40, 136, "geglu"), (300, 200, 136, "none")])
def test_linear_backward_nan_stays_in_its_row(R, N, K, act):
    """A NaN in a row of dout or of z leaves the other rows of dz and dx alone, in either kind of product kernel; dw and db
    hold it where dz's column does."""
    x, w, dout, z, dz, dx, dw, db, ws = _backward(R, N, K, act, BF16)
    dout[4, N - 1] = NAN
    if z is not None:
        z[7, 3] = NAN
    got_z = None if dz is None else torch.zeros_like(dz)
    got_x, got_w, got_b = torch.zeros_like(dx), torch.zeros_like(dw), torch.zeros_like(db)
    m.moe_linear_backward(dout, x, w, z, got_z, got_x, got_w, got_b, ws, act=act, alpha=ALPHA, limit=LIMIT)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[4], keep[7] = False, act == "none"
    assert torch.equal(got_x[keep], dx[keep])
    assert bool(torch.isnan(got_x[~keep].float()).all())
    d = dout if dz is None else got_z
    if dz is not None:
        assert torch.equal(got_z[keep], dz[keep])
    bad = torch.isnan(d.float()).any(0)
    assert bool(bad.any()) and not bool(bad.all())
    assert torch.equal(torch.isnan(got_b.float()), bad) and torch.equal(got_b[~bad], db[~bad])
    assert torch.equal(torch.isnan(got_w.float()), bad[:, None].expand_as(got_w)) and torch.equal(got_w[~bad], dw[~bad])
    assert m.moe_mm_read_status(ws) == 0


@pytest.mark.parametrize("R,N,K,act", [(33, 48, 64, "swiglu"), (600, 48, 64, "swiglu"), (2200, 40, 72, "silu"), (600, 48, 64, "none")])
def test_linear_backward_elements_past_32_bits(R, N, K, act):
    """Rows so far apart that the last one's offset passes 2^31 elements, of every matrix of the backward; few and many
    rows, and a split reduction of dw."""
    cuda_device()
    _needs_gb(80)
    g = _gen(9)
    rows = D.halves(act) * N

    def far(n, cols):
        ld = (2 ** 31 // (n - 1) + 64) // 8 * 8
        return torch.zeros(n, ld, dtype=BF16, device="cuda")[:, :cols]

    x, dout, dx, dw, w = far(R, K), far(R, N), far(R, K), far(rows, K), far(rows, K)
    x.copy_(_randn(g, R, K))
    dout.copy_(_randn(g, R, N))
    w.copy_(_randn(g, rows, K, std=K ** -0.5))
    z = dz = None
    if act != "none":
        z, dz = far(R, rows), far(R, rows)
        z.copy_(_randn(g, R, rows, std=1.5))
    db = torch.full((rows,), NAN, device="cuda")
    ws = _ws(R, rows, K, True)
    m.moe_linear_backward(dout, x, w, z, dz, dx, dw, db, ws, act=act, alpha=ALPHA, limit=LIMIT)
    rz, bz = D.linear_dz(dout, z, act, ALPHA, LIMIT)
    d = dout.double()
    if z is not None:
        P.assert_within(dz, rz, bz, "dz")
        d = dz.double()
    P.assert_within(db, rz.sum(0), bz.sum(0) + (R + 8) * P.EPS32 * (rz.abs() + bz).sum(0), "db")
    P.assert_within(dx, d @ w.double(), (rows + 8) * P.EPS32 * (d.abs() @ w.double().abs()), "dx")
    P.assert_within(dw, d.t() @ x.double(), (R + 8) * P.EPS32 * (d.abs().t() @ x.double().abs()), "dw")
    assert m.moe_mm_read_status(ws) == 0


FIRST_CALL = '''
import torch
import quantized_grouped_gemm_topk_gb300 as m

torch.manual_seed(0)
bf = torch.bfloat16
dev = dict(device="cuda")


def randn(*shape):
    return torch.randn(*shape, **dev).to(bf) * 0.2


def zeros(n):
    return torch.zeros(n, dtype=torch.uint8, **dev)


T, H, I, E, k = 7, 320, 192, 9, 3
layer = [randn(T, H), torch.randn(H, E, **dev), None, randn(E, 2 * I, H), randn(E, H, I), torch.zeros(T, H, dtype=bf, **dev),
         torch.zeros(T, k, dtype=torch.int32, **dev), torch.zeros(T, k, **dev), zeros(m.moe_layer16_workspace_size(T, H, I, E, k))]
outs = [layer[5]]
calls = [lambda: m.moe_layer16_forward(*layer)]
for R, N, K in ((5, 200, 264), (400, 200, 264), (40, 2048, 264)):
    x, w, d = randn(R, K), randn(2 * N, K), randn(R, N)
    out, z, dz, dx, dw = (torch.zeros(*s, dtype=bf, **dev) for s in ((R, N), (R, 2 * N), (R, 2 * N), (R, K), (2 * N, K)))
    db = torch.zeros(2 * N, **dev)
    fws, bws = (zeros(m.moe_linear_workspace_size(R, 2 * N, K, b)) for b in (False, True))
    calls.append(lambda x=x, w=w, out=out, ws=fws, z=z: m.moe_linear_forward(x, w, out, ws, z=z, act="swiglu"))
    calls.append(lambda d=d, x=x, w=w, z=z, dz=dz, dx=dx, dw=dw, db=db, ws=bws: m.moe_linear_backward(d, x, w, z, dz, dx, dw, db, ws, act="swiglu"))
    outs += [out, z, dz, dx, dw, db]
torch.cuda.synchronize()
stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=stream):
    for call in calls:
        call()
torch.cuda.synchronize()
assert not any(bool(o.any()) for o in outs)             # captured, not run
graph.replay()
torch.cuda.synchronize()
got = [o.clone() for o in outs]
assert all(bool(o.any()) for o in outs)
for o in outs:
    o.zero_()
for call in calls:
    call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
print("same")
'''


def test_first_calls_of_a_process_in_a_graph():
    """The layer's and the dense products' first calls in a process are captured, on a stream of their own: what the library
    asks the driver once (attributes, residency) may be asked during a capture."""
    import os
    import subprocess
    import sys
    cuda_device()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["same"], r.stdout + r.stderr


@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_fp32_weight_gradient_of_the_grouped_products(act):
    """dw in fp32: the grouped products' weight gradient of dz, with one group of all rows."""
    R, N, K = 700, 200, 264
    x, w, dout, z, dz, _, dw, _, _ = _backward(R, N, K, act, BF16)
    d = dout if dz is None else dz
    rows = d.shape[1]
    off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
    got = torch.full((1, rows, K), NAN, device="cuda")
    ws = torch.zeros(m.moe_mm_workspace_size(m.MOE_MM_WGRAD, R, rows, K, 1), dtype=torch.uint8, device="cuda")
    m.moe_grouped_mm_wgrad(d, x, off, got, ws)
    ref, mag = d.double().t() @ x.double(), d.double().abs().t() @ x.double().abs()
    P.assert_within(got[0], ref, (R + 8) * P.EPS32 * mag, "dw")
    # one rounding less than the 16-bit one
    assert float((got[0].double() - ref).norm()) < 0.01 * float((dw.double() - ref).norm())
