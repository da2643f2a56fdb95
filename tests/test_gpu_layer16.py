"""The layer for a few tokens with 16-bit experts on the GPU, against its 64-bit form."""
import math

import pytest
import torch

import dense_ref as D
import ops_ref as P
import quantized_grouped_gemm_topk_gb300 as m

from util import cuda_device

pytestmark = pytest.mark.gpu

BF16, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
NAN, INF = float("nan"), math.inf
ALPHA, LIMIT = 1.702, 2.0


def _gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=F32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _inputs(T, H, I, E, k, S, act, dtype, bias, pad, seed=0):
    g = _gen(seed + T * 11 + H * 3 + I + E)
    G = E + S
    c = dict(x=P.strided(_randn(g, T, H, dtype=dtype), pad, whole=8)[0],
             W_r=_randn(g, H, E, std=H ** -0.5),
             w1=P.strided(_randn(g, G, D.halves(act) * I, H, dtype=dtype, std=1.5 * H ** -0.5), pad, whole=8)[0],
             w2=P.strided(_randn(g, G, H, I, dtype=dtype, std=I ** -0.5), pad, whole=8)[0],
             b1=_randn(g, G, 2 * I, std=0.3) if bias else None,
             ids=torch.zeros(T, k, dtype=I32, device="cuda"), wts=torch.zeros(T, k, device="cuda"),
             ws=torch.zeros(m.moe_layer16_workspace_size(T, H, I, E, k, S), dtype=torch.uint8, device="cuda"))
    c["out"], c["obuf"] = P.strided(torch.zeros(T, H, dtype=dtype, device="cuda"), pad and 3)
    return c


def _run(c, act, S=0, W_r=None, logits=None, scale=1.0, out=None):
    m.moe_layer16_forward(c["x"], W_r, logits, c["w1"], c["w2"], c["out"] if out is None else out, c["ids"], c["wts"], c["ws"],
                          b1=c["b1"], n_shared=S, act=act, alpha=ALPHA, limit=LIMIT, routed_scale=scale)


def _check_out(c, act, S):
    ref, bound = D.layer(c["x"], c["w1"], c["w2"], c["b1"], c["ids"].long(), c["wts"], S, act, ALPHA, LIMIT)
    P.assert_within(c["out"], ref, bound, "out")


def _layer(T, H, I, E, k, S=0, act="swiglu", dtype=BF16, bias=False, pad=0, scale=1.0):
    cuda_device()
    c = _inputs(T, H, I, E, k, S, act, dtype, bias, pad)
    _run(c, act, S, W_r=c["W_r"], scale=scale)
    x, r = c["x"].double(), c["W_r"].double()
    logits, b = x @ r, (H + 8) * P.EPS32 * (x.abs() @ r.abs()).amax(1, keepdim=True)
    want, _ = D.routing(logits, k, scale)
    ids = c["ids"].long()
    assert bool((ids >= 0).all()) and bool((ids < E).all())
    assert all(len(set(row)) == k for row in ids.tolist())
    # ids may differ only where two logits are nearer than their sums' error
    assert bool(((logits.gather(1, ids) - logits.gather(1, want)).abs() <= 2 * b).all())
    p = torch.exp(logits.gather(1, ids) - logits.gather(1, ids).amax(1, keepdim=True))
    w = p / p.sum(1, keepdim=True) * scale
    # exp of a difference of two logits, twice (CUDA's expf: 2 units); k additions, a division and two products
    P.assert_within(c["wts"], w, w * (4 * b + (k + 12) * P.EPS32), "weights")
    _check_out(c, act, S)
    if pad:
        assert bool(torch.isnan(c["obuf"][:, H:].float()).all())
    assert m.moe_mm_read_status(c["ws"]) == 0
    return c


@pytest.mark.parametrize("T,H,I,E,k,S", [
    (1, 256, 128, 8, 2, 0), (1, 8, 8, 1, 1, 0), (2, 1, 1, 3, 2, 1), (3, 72, 40, 5, 5, 0), (5, 1999, 1001, 24, 3, 1), (8, 520, 264, 16, 4, 0),
    (16, 640, 384, 160, 8, 1), (17, 300, 65, 7, 3, 0), (31, 129, 200, 40, 6, 0), (32, 1024, 512, 16, 4, 1), (33, 200, 129, 12, 2, 0),
    (48, 264, 320, 3, 1, 0), (64, 576, 448, 64, 8, 0), (64, 128, 64, 2048, 32, 0), (64, 2880, 360, 32, 4, 0), (63, 64, 1031, 2, 2, 1),
    (1, 7168, 256, 64, 8, 0), (4, 100, 3001, 2, 1, 0), (1, 17, 4096, 300, 31, 1)])
@pytest.mark.parametrize("act,dtype,bias,pad", [("swiglu", BF16, False, 0), ("swiglu_clamp", F16, True, 8), ("geglu", BF16, True, 8),
                                                ("srelu", F16, False, 0)])
def test_layer16(T, H, I, E, k, S, act, dtype, bias, pad):
    _layer(T, H, I, E, k, S, act, dtype, bias, pad, scale=2.5 if S else 1.0)


@pytest.mark.parametrize("T", [1, 2, 16, 64])
@pytest.mark.parametrize("H,I,E,k,S", [(2880, 2880, 16, 4, 0), (6144, 1536, 12, 8, 1), (7168, 2048, 9, 8, 0)])
def test_layer16_of_model_widths(T, H, I, E, k, S):
    _layer(T, H, I, E, k, S)


@pytest.mark.parametrize("T,E,k", [(1, 8, 3), (9, 100, 8), (64, 33, 32), (5, 2047, 6)])
def test_layer16_from_logits_ties_masks_and_nan(T, E, k):
    """Ready logits: ties go to the lower id; -inf masks an expert, NaN ranks as -inf and is flagged; a token without a
    finite logit has weights 0; a masked expert's weights may hold anything."""
    cuda_device()
    g = _gen(T + E)
    c = _inputs(T, 72, 40, E, k, 0, "swiglu", BF16, False, 0)
    logits = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    logits[0] = torch.where(logits[0] == 0, torch.tensor(-0.0, device="cuda"), logits[0])
    _run(c, "swiglu", logits=logits)
    ids, w = D.routing(logits.double(), k, 1.0)
    assert torch.equal(c["ids"].long(), ids)
    P.assert_within(c["wts"], w, w * (k + 12) * P.EPS32, "weights")
    _check_out(c, "swiglu", 0)
    assert m.moe_mm_read_status(c["ws"]) == 0

    logits[:, 1:] = torch.where(torch.rand(T, E - 1, generator=g, device="cuda") < 0.7, torch.tensor(-INF, device="cuda"), logits[:, 1:])
    logits[:, E - 1] = -INF           # nobody's
    logits[T - 1] = -INF
    c["w1"][E - 1], c["w2"][E - 1] = NAN, INF
    c["out"].fill_(NAN)
    _run(c, "swiglu", logits=logits)
    ids, w = D.routing(logits.double(), k, 1.0)
    assert torch.equal(c["ids"].long(), ids)
    assert torch.equal(c["wts"] == 0, w == 0) and not bool(c["wts"][T - 1].any())
    assert not bool(c["out"][T - 1].any())
    safe = {**c, "w1": c["w1"].clone(), "w2": c["w2"].clone()}
    safe["w1"][E - 1], safe["w2"][E - 1] = 0, 0
    _check_out(safe, "swiglu", 0)

    logits[0, 0] = NAN
    _run(c, "swiglu", logits=logits)
    ids, w = D.routing(logits.double(), k, 1.0)
    assert torch.equal(c["ids"].long(), ids)
    assert m.moe_mm_read_status(c["ws"]) == m.MOE_DEV_NAN_LOGIT
    assert m.moe_mm_read_status(c["ws"]) == 0


def test_layer16_from_given_ids():
    """Ids and weights of the caller: an id may repeat, its weights add up; one out of range is skipped and flagged; weights
    are taken as they are (negative ones too)."""
    cuda_device()
    g = _gen(4)
    T, E, k, S = 21, 6, 5, 1
    c = _inputs(T, 200, 136, E, k, S, "geglu", F16, True, 8)
    c["ids"].copy_(torch.randint(0, E, (T, k), generator=g, device="cuda"))
    c["wts"].copy_(_randn(g, T, k))
    c["wts"][3] = 0
    before = c["ids"].clone(), c["wts"].clone()
    _run(c, "geglu", S)
    _check_out(c, "geglu", S)
    assert torch.equal(c["ids"], before[0]) and torch.equal(c["wts"], before[1])
    assert m.moe_mm_read_status(c["ws"]) == 0
    c["ids"][2, 1], c["ids"][20, 4] = -1, E
    _run(c, "geglu", S)
    _check_out(c, "geglu", S)
    assert m.moe_mm_read_status(c["ws"]) == m.MOE_DEV_BAD_EXPERT_ID


def test_layer16_tokens_do_not_reach_each_other():
    """A NaN or infinity in one token, or in an expert that only it chose, leaves the others' bits alone."""
    cuda_device()
    T, H, I, E, k = 19, 328, 200, 8, 2
    c = _inputs(T, H, I, E, k, 0, "swiglu", BF16, False, 0)
    g = _gen(2)
    c["ids"].copy_(torch.stack([torch.randperm(E - 1, generator=g, device="cuda")[:k] for _ in range(T)]))
    c["wts"].copy_(torch.rand(T, k, generator=g, device="cuda") + 0.1)
    c["ids"][5, 1] = E - 1
    _run(c, "swiglu")
    want = c["out"].clone()
    others = [t for t in range(T) if t != 5]
    c["w1"][E - 1, 3, 7] = INF
    c["w2"][E - 1] = NAN
    _run(c, "swiglu")
    assert torch.equal(c["out"][others], want[others]) and bool(torch.isnan(c["out"][5].float()).all())
    c["w1"][E - 1], c["w2"][E - 1] = 0, 0
    c["x"][5, H - 1] = NAN
    _run(c, "swiglu")
    assert torch.equal(c["out"][others], want[others]) and bool(torch.isnan(c["out"][5].float()).all())


def test_layer16_repeats_streams_graphs_and_a_shared_workspace():
    cuda_device()
    big = _inputs(64, 640, 384, 24, 4, 1, "swiglu", BF16, False, 0)
    sets = [(big, 1)]
    small = _inputs(3, 640, 384, 24, 4, 1, "swiglu", BF16, False, 0, seed=9)
    small["ws"] = big["ws"]           # one for the largest batch serves a smaller one
    sets.append((small, 1))
    wants = []
    for c, S in sets:
        _run(c, "swiglu", S, W_r=c["W_r"])
        wants.append(c["out"].clone())
    for _ in range(4):
        for (c, S), want in zip(sets, wants):
            c["out"].fill_(NAN)
            _run(c, "swiglu", S, W_r=c["W_r"])
            assert torch.equal(c["out"], want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, S in sets:
            c["out"].fill_(NAN)
            _run(c, "swiglu", S, W_r=c["W_r"])
    side.synchronize()
    graphs = []
    for (c, S), want in zip(sets, wants):
        assert torch.equal(c["out"], want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _run(c, "swiglu", S, W_r=c["W_r"])
        graphs.append(graph)
    for _ in range(3):
        for graph, (c, S), want in zip(graphs, sets, wants):
            c["out"].fill_(NAN)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(c["out"], want)
    assert m.moe_mm_read_status(big["ws"]) == 0


def test_layer16_of_two_streams_at_once():
    """Two calls that may run at the same time, each with its own workspace."""
    cuda_device()
    cs = [_inputs(40, 1024, 512, 16, 4, 0, "swiglu", BF16, False, 0, seed=s) for s in (1, 2)]
    wants = []
    for c in cs:
        _run(c, "swiglu", W_r=c["W_r"])
        wants.append(c["out"].clone())
        c["out"].fill_(NAN)
    streams = [torch.cuda.Stream() for _ in cs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                _run(c, "swiglu", W_r=c["W_r"])
    torch.cuda.synchronize()
    for c, want in zip(cs, wants):
        assert torch.equal(c["out"], want)
        assert m.moe_mm_read_status(c["ws"]) == 0


def test_layer16_weights_past_32_bits():
    """Experts whose matrices lie beyond 2^31 elements."""
    cuda_device()
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    T, H, I, E, k = 3, 4096, 2048, 140, 2
    w1 = torch.zeros(E, 2 * I, H, dtype=BF16, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=BF16, device="cuda")
    assert w1.numel() > 2 ** 31
    c = _inputs(T, H, I, 2, k, 0, "swiglu", BF16, False, 0)
    w1[0], w1[E - 1], w2[0], w2[E - 1] = c["w1"][0], c["w1"][1], c["w2"][0], c["w2"][1]
    ids = torch.tensor([[0, E - 1]] * T, dtype=I32, device="cuda")
    c["wts"].fill_(0.5)
    out = torch.empty(T, H, dtype=BF16, device="cuda")
    ws = torch.zeros(m.moe_layer16_workspace_size(T, H, I, E, k), dtype=torch.uint8, device="cuda")
    m.moe_layer16_forward(c["x"], None, None, w1, w2, out, ids, c["wts"], ws)
    ref, bound = D.layer(c["x"], c["w1"], c["w2"], None, torch.tensor([[0, 1]] * T, device="cuda"), c["wts"], 0, "swiglu", 1.0, 0.0)
    P.assert_within(out, ref, bound, "out")


@pytest.mark.parametrize("T,H,I,E,k,S", [(3, 40008, 72, 3, 2, 0), (64, 20001, 40, 5, 3, 1), (2, 72, 30001, 2, 2, 0), (20, 16, 9000, 40, 2, 0)])
def test_layer16_wide(T, H, I, E, k, S):
    """Wider than a tile for every SM, in the second product and in the first."""
    _layer(T, H, I, E, k, S, "swiglu_clamp", BF16, True)


def test_layer16_first_call_in_a_graph_on_another_stream():
    """Captured without a call before it, in the same process or not: nothing is allocated or waited for."""
    cuda_device()
    c = _inputs(7, 320, 192, 9, 3, 0, "geglu", F16, False, 0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(c, "geglu", W_r=c["W_r"])
    for _ in range(2):
        c["out"].fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        _check_out(c, "geglu", 0)


def test_layer16_of_a_trained_block():
    """The experts that the example's grouped products train, served: the same layer, token by token and in a batch."""
    cuda_device()
    T, H, I, E, k = 24, 256, 128, 8, 2
    c = _inputs(T, H, I, E, k, 0, "swiglu", BF16, False, 0)
    _run(c, "swiglu", W_r=c["W_r"])
    whole, ids, wts = c["out"].clone(), c["ids"].clone(), c["wts"].clone()
    # the same tokens by the grouped products, sorted by expert
    order = torch.argsort(ids.flatten().long(), stable=True)
    off = torch.zeros(E + 1, dtype=I32, device="cuda")
    off[1:] = torch.bincount(ids.flatten().long(), minlength=E).cumsum(0)
    rows = T * k
    xg = c["x"][order // k].contiguous()
    h, y, z = (torch.empty(rows, n, dtype=BF16, device="cuda") for n in (2 * I, I, H))
    ws = torch.zeros(max(m.moe_mm_workspace_size(m.MOE_MM_ROWS, rows, n, q, E) for n, q in ((2 * I, H), (H, I))), dtype=torch.uint8,
                     device="cuda")
    m.moe_grouped_mm(xg, c["w1"].contiguous(), off, h, ws)
    q, s = torch.empty(rows, 2 * I, dtype=torch.uint8, device="cuda"), torch.empty(rows, 2 * -(-I // 128), device="cuda")
    m.moe_act_ckpt_forward(h, wts.flatten()[order].contiguous(), y, q, s)
    m.moe_grouped_mm(y, c["w2"].contiguous(), off, z, ws)
    other = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, order // k, z.double())
    # h and z of the grouped way are rounded to bf16 too: h's half step moves act by 2^-8 (|g| act'_g + |u| act'_u) <= 2^-8 * 3
    # |act| and a little, z's is 2^-8 |z| a slot
    ref, bound = D.layer(c["x"], c["w1"], c["w2"], None, ids.long(), wts, 0, "swiglu", 1.0, 0.0)
    mag = z.double().abs()
    slack = torch.zeros_like(other).index_add_(0, order // k, 2.0 ** -8 * mag)
    a = torch.cat([v.double() for v in (h,)], 1)
    g, u = a[:, :I], a[:, I:]
    dact = 2.0 ** -8 * (g.abs() * (1.2 * u.abs()) + u.abs() * g.abs()) * wts.flatten()[order].double()[:, None]
    for e in range(E):
        sl = slice(int(off[e]), int(off[e + 1]))
        slack.index_add_(0, order[sl] // k, dact[sl] @ c["w2"][e].double().abs().t())
    assert bool(((other - ref).abs() <= bound + slack + 1e-6).all())
    P.assert_within(whole, ref, bound, "out")
    # one token at a time: its own weights, whose logits may be summed in another order, and the same bound
    for t in (0, 11, 23):
        out = torch.empty(1, H, dtype=BF16, device="cuda")
        m.moe_layer16_forward(c["x"][t:t + 1], c["W_r"], None, c["w1"], c["w2"], out, c["ids"][:1], c["wts"][:1], c["ws"])
        assert torch.equal(c["ids"][0], ids[t])
        one = D.layer(c["x"][t:t + 1], c["w1"], c["w2"], None, c["ids"][:1].long(), c["wts"][:1], 0, "swiglu", 1.0, 0.0)
        P.assert_within(out, *one, "one token")


# the second product's groups whole, in halves and in quarters, with one to all tokens a group
@pytest.mark.parametrize("T,H,I,E,k,S", [(16, 4096, 512, 24, 8, 0), (64, 1024, 256, 16, 8, 1), (64, 4096, 64, 4, 2, 0), (64, 7168, 264, 6, 4, 0),
                                         (3, 2048, 768, 40, 8, 1), (40, 2880, 520, 9, 3, 0), (64, 300, 72, 2, 2, 1), (17, 512, 2056, 60, 6, 0)])
@pytest.mark.parametrize("act,dtype", [("swiglu", BF16), ("srelu", F16)])
def test_layer16_narrow_experts(T, H, I, E, k, S, act, dtype):
    _layer(T, H, I, E, k, S, act, dtype, False, 8)


# the router in one CTA and in slices: eight rows a thread, 4096 values of x
@pytest.mark.parametrize("T,H,E,k", [(1, 2048, 8, 2), (1, 2049, 8, 2), (1, 4096, 3, 3), (2, 2048, 4, 1), (2, 2056, 4, 1), (3, 1024, 13, 5),
                                     (4, 1025, 13, 5), (8, 512, 30, 4), (9, 513, 30, 4), (33, 64, 256, 8), (64, 65, 256, 8), (64, 64, 257, 8),
                                     (5, 8, 100, 32), (64, 1, 1, 1)])
def test_layer16_routers(T, H, E, k):
    _layer(T, H, 24, E, k, 0, "swiglu", BF16, False)


@pytest.mark.parametrize("T", [1, 3, 20, 64])
def test_layer16_shares_its_workspace(T):
    """Behind the status word's block the workspace holds nothing between calls: what another product left there does no harm."""
    cuda_device()
    c = _inputs(T, 264, 136, 12, 3, 1, "swiglu", BF16, False, 0)
    _run(c, "swiglu", 1, W_r=c["W_r"])
    first = c["out"].clone()
    for v in (0x7f, 0xff, 1):
        c["ws"][256:] = v
        c["out"].fill_(NAN)
        _run(c, "swiglu", 1, W_r=c["W_r"])
        assert torch.equal(c["out"], first)
        assert m.moe_mm_read_status(c["ws"]) == 0


def test_layer16_no_tokens():
    cuda_device()
    c = _inputs(1, 64, 64, 4, 2, 0, "swiglu", BF16, False, 0)
    m.moe_layer16_forward(c["x"][:0], c["W_r"], None, c["w1"], c["w2"], c["out"][:0], c["ids"][:0], c["wts"][:0], c["ws"])
    assert m.moe_last_launch_count() == 0


def test_decode_block_of_the_operators():
    """A decode step as it is used: norm, the routed layer beside a dense shared part that adds to it, and the residual."""
    cuda_device()
    T, H, I, E, k = 6, 512, 256, 16, 4
    c = _inputs(T, H, I, E, k, 0, "swiglu", BF16, False, 0)
    g = _gen(77)
    h = _randn(g, T, H, dtype=BF16)
    gamma = _randn(g, H) * 0.1 + 1
    m.moe_layer_norm_forward(h, gamma, None, 1e-5, c["x"])
    P.assert_within(c["x"], P.norm_fwd(h, gamma, None, 1e-5)[0], torch.full((T, H), 1e-4, dtype=torch.float64, device="cuda"), "norm")
    _run(c, "swiglu", W_r=c["W_r"])
    _check_out(c, "swiglu", 0)
    u, d = _randn(g, 2 * I, H, dtype=BF16, std=H ** -0.5), _randn(g, H, I, dtype=BF16, std=I ** -0.5)
    a = torch.empty(T, I, dtype=BF16, device="cuda")
    ws = torch.zeros(max(m.moe_linear_workspace_size(T, 2 * I, H), m.moe_linear_workspace_size(T, H, I)), dtype=torch.uint8, device="cuda")
    m.moe_linear_forward(c["x"], u, a, ws, act="swiglu")
    ra, ba, _, _ = D.linear(c["x"], u, None, None, "swiglu", 1.0, 0.0)
    P.assert_within(a, ra, ba, "shared part")
    routed = c["out"].clone()
    m.moe_linear_forward(a, d, c["out"], ws, residual=c["out"])
    ro, bo, _, _ = D.linear(a, d, None, routed, "none", 1.0, 0.0)
    P.assert_within(c["out"], ro, bo, "out")


# sizes whose second product splits its groups in halves and in quarters
@pytest.mark.parametrize("T,H,I,E,k", [(16, 4096, 512, 24, 8), (64, 1024, 256, 64, 8), (3, 2048, 768, 40, 8), (17, 512, 264, 60, 6)])
def test_layer16_fewer_groups_than_parts(T, H, I, E, k):
    """No token with an expert, or all of them with the same few: parts without a group have nothing to compute and are
    joined all the same."""
    cuda_device()
    c = _inputs(T, H, I, E, k, 0, "swiglu", BF16, False, 0)
    for live in (0, 1, 2, 3, 5):
        c["ids"].copy_(torch.arange(k, device="cuda").expand(T, k) * 3 % E)
        c["wts"].copy_((torch.arange(k, device="cuda") < live).float() * 0.25)
        want = None
        for _ in range(20 if live < 2 else 3):
            c["out"].fill_(NAN)
            _run(c, "swiglu")
            if want is None:
                want = c["out"].clone()
                _check_out(c, "swiglu", 0)
            assert torch.equal(c["out"], want)
        if not live:
            assert not bool(want.any())
        assert m.moe_mm_read_status(c["ws"]) == 0


def _check_out_in_parts(c, act, S):
    """The bound of y in two parts, which dense_ref.layer knows for up to 32 tokens, at any number of them."""
    parts = [D.layer(c["x"][t:t + 32], c["w1"], c["w2"], c["b1"], c["ids"][t:t + 32].long(), c["wts"][t:t + 32], S, act, ALPHA, LIMIT)
             for t in range(0, c["x"].shape[0], 32)]
    P.assert_within(c["out"], torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts]), "out")


# few values to sum, so that a rounding of y is seen; groups of a few tokens, of up to 32, and of more
@pytest.mark.parametrize("T,H,I,E,k,S", [(32, 264, 40, 4, 2, 0), (33, 264, 40, 40, 2, 0), (33, 520, 72, 4, 2, 1), (48, 1024, 64, 2, 1, 0),
                                         (64, 300, 24, 3, 2, 1), (64, 2048, 128, 24, 4, 0), (64, 7168, 72, 2, 2, 0), (64, 1024, 136, 64, 8, 1),
                                         (50, 20001, 40, 3, 3, 0), (64, 128, 1, 5, 2, 0)])
@pytest.mark.parametrize("act,dtype,bias", [("swiglu", BF16, False), ("geglu", F16, True), ("srelu", BF16, False)])
def test_layer16_is_as_exact_for_many_tokens(T, H, I, E, k, S, act, dtype, bias):
    """A token's result is as exact in a batch of 64 as in one of 32: y is in two parts at any number of tokens."""
    cuda_device()
    c = _inputs(T, H, I, E, k, S, act, dtype, bias, 8)
    _run(c, act, S, W_r=c["W_r"])
    _check_out_in_parts(c, act, S)
    assert m.moe_mm_read_status(c["ws"]) == 0


@pytest.mark.parametrize("T,H,I,E,k,S", [(1, 264, 136, 4, 2, 0), (16, 264, 136, 40, 2, 0), (30, 1024, 256, 4, 2, 1), (64, 520, 72, 3, 2, 1),
                                         (64, 1024, 256, 64, 4, 0)])
@pytest.mark.parametrize("act", ["srelu", "swiglu"])
def test_layer16_f16_activations_past_its_range(T, H, I, E, k, S, act):
    """Activations that an f16 number cannot hold, of results that it can; and, past what y holds, an infinity of one token."""
    cuda_device()
    c = _inputs(T, H, I, E, k, S, act, F16, False, 8)
    c["w1"] *= 160
    c["w2"] *= 2.0 ** -8
    _run(c, act, S, W_r=c["W_r"])
    largest = 0.0
    for e in range(E):
        w = (c["wts"].double() * (c["ids"] == e)).sum(1)
        y = D.linear(c["x"], c["w1"][e], None, None, act, ALPHA, LIMIT)[0] * w[:, None]
        largest = max(largest, float(y.abs().max()))
    assert largest > 65520
    assert bool(torch.isfinite(c["out"].float()).all())
    _check_out_in_parts(c, act, S)
    if T == 1 or S:
        return
    want = c["out"].clone()
    c["x"][T // 2] *= 500
    _run(c, act, S)             # with the ids and weights of before
    keep = [t for t in range(T) if t != T // 2]
    assert torch.equal(c["out"][keep], want[keep]) and not bool(torch.isfinite(c["out"][T // 2].float()).all())
    assert m.moe_mm_read_status(c["ws"]) == 0


@pytest.mark.parametrize("T,k", [(2, 2), (16, 3), (17, 2), (40, 2), (64, 5)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_layer16_tokens_do_not_reach_each_other_at_any_number(T, k, dtype):
    """As above with each way through the epilogues (up to 16 tokens, up to 32, more) and with groups of many tokens: a NaN
    or an infinity of a token, of its weight, or of an expert that only it chose."""
    cuda_device()
    H, I, E = 328, 200, 6
    c = _inputs(T, H, I, E, k, 0, "swiglu", dtype, False, 0)
    g = _gen(3)
    c["ids"].copy_(torch.stack([torch.randperm(E - 1, generator=g, device="cuda")[:k] for _ in range(T)]))
    c["wts"].copy_(torch.rand(T, k, generator=g, device="cuda") + 0.1)
    t = T // 2
    c["ids"][t, 1] = E - 1
    _run(c, "swiglu")
    want = c["out"].clone()
    others = [i for i in range(T) if i != t]

    def check(alone=NAN):
        c["out"].fill_(7)
        _run(c, "swiglu")
        assert torch.equal(c["out"][others], want[others])
        mine = c["out"][t].float()
        assert bool((torch.isnan(mine) if alone != alone else ~torch.isfinite(mine)).all())

    w1, w2, x = c["w1"][E - 1].clone(), c["w2"][E - 1].clone(), c["x"][t].clone()
    c["w1"][E - 1, 3, 7] = INF
    c["w2"][E - 1] = NAN
    check()
    c["w1"][E - 1], c["w2"][E - 1] = w1, w2
    for v in (NAN, INF, -INF):
        c["x"][t, H - 1] = v
        check()
    c["x"][t] = x
    c["wts"][t, 0] = NAN
    check()
    c["wts"][t, 0] = INF
    check(INF)
    c["wts"][t, 0] = 0.5
    c["out"].fill_(7)
    _run(c, "swiglu")
    assert torch.equal(c["out"][others], want[others]) and bool(torch.isfinite(c["out"][t].float()).all())
    assert m.moe_mm_read_status(c["ws"]) == 0


def test_layer16_of_many_wide_experts():
    """As many experts and slots as there can be, whose tables take most of what the ring of weights has, and ranges of H of
    more than 64 features: only the experts that a token chose hold anything else than NaN."""
    cuda_device()
    if torch.cuda.get_device_properties(0).total_memory < 60 << 30:
        pytest.skip("needs 60 GB")
    T, I, E, S, dtype = 64, 72, 2047, 1, BF16
    for H, k in ((20008, 31), (8200, 8)):
        g = _gen(H)
        few = 40
        live = torch.randperm(E, generator=g, device="cuda")[:few]
        kept = torch.cat([live, torch.tensor([E], device="cuda")])
        w1 = torch.full((E + S, 2 * I, H), NAN, dtype=dtype, device="cuda")
        w2 = torch.full((E + S, H, I), NAN, dtype=dtype, device="cuda")
        w1[kept] = _randn(g, few + 1, 2 * I, H, dtype=dtype, std=H ** -0.5)
        w2[kept] = _randn(g, few + 1, H, I, dtype=dtype, std=I ** -0.5)
        at = torch.stack([torch.randperm(few, generator=g, device="cuda")[:k] for _ in range(T)])
        c = dict(x=_randn(g, T, H, dtype=dtype), w1=w1, w2=w2, b1=None, ids=live[at].int().contiguous(),
                 wts=torch.rand(T, k, generator=g, device="cuda"), out=torch.empty(T, H, dtype=dtype, device="cuda"),
                 ws=torch.zeros(m.moe_layer16_workspace_size(T, H, I, E, k, S), dtype=torch.uint8, device="cuda"))
        _run(c, "swiglu", S)
        small = {**c, "w1": w1[kept], "w2": w2[kept], "ids": at}
        _check_out_in_parts(small, "swiglu", S)
        assert m.moe_mm_read_status(c["ws"]) == 0
