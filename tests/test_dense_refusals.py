"""The dense product and the layer for a few tokens refuse what they cannot
compute, on the host, before any device work (no GPU needed: a call that reached
the CUDA runtime here would return the CUDA error code)."""
import ctypes

import pytest

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from quantized_grouped_gemm_topk_gb300 import build as b
    b.build()
    from quantized_grouped_gemm_topk_gb300 import binding
    return binding.load()


def _call(fn, base, **kw):
    unknown = set(kw) - set(base)
    assert not unknown, unknown
    return fn(*{**base, **kw}.values())


FWD = dict(x=P(0x1000), ldx=64, w=P(0x2000), ldw=64, bias=P(0x3000), res=P(0x4000), ldr=32, R=4, N=32, K=64, act=0, alpha=1.0,
           limit=0.0, dtype=0, wdtype=2, z=P(0x5000), ldz=64, out=P(0x6000), ldo=32, ws=P(0x7000), ws_bytes=1 << 30, stream=None)
BWD = dict(dout=P(0x1000), lddout=32, x=P(0x2000), ldx=64, w=P(0x3000), ldw=64, z=P(0x4000), ldz=64, R=4, N=32, K=64, act=0,
           alpha=1.0, limit=0.0, dtype=0, wdtype=2, dz=P(0x5000), lddz=64, dx=P(0x6000), lddx=64, dw=P(0x7000), lddw=64,
           db=P(0x8000), ws=P(0x9000), ws_bytes=1 << 30, stream=None)
LAYER = dict(x=P(0x1000), ldx=64, W_r=P(0x2000), logits=None, w1=P(0x3000), g1=4096, ld1=64, b1=P(0x4000), w2=P(0x5000), g2=2048,
             ld2=32, T=4, H=64, I=32, E=3, k=2, S=1, act=0, alpha=1.0, limit=0.0, rs=1.0, dtype=0, out=P(0x6000), ldo=64,
             ids=P(0x7000), wts=P(0x8000), ws=P(0x9000), ws_bytes=1 << 30, stream=None)

BAD = {
    "moe_linear_forward": (FWD, [
        dict(x=None), dict(w=None), dict(out=None), dict(ws=None), dict(x=P(0x1008)), dict(w=P(0x2002)), dict(ws=P(0x7008)),
        dict(bias=P(0x3002)), dict(bias=P(0x3001), wdtype=0), dict(res=P(0x4001)), dict(z=P(0x5001)), dict(out=P(0x6001)),
        dict(ldx=63), dict(ldx=68), dict(ldw=56), dict(ldw=68), dict(ldr=31), dict(ldz=63), dict(ldo=31), dict(R=-1), dict(N=0),
        dict(K=0), dict(act=7), dict(act=-1), dict(act=1), dict(dtype=2), dict(wdtype=1), dict(dtype=1, wdtype=0),
        dict(res=P(0x6000), ldr=40), dict(N=2 ** 30, ldo=2 ** 31, ldr=2 ** 31, ldz=2 ** 32)]),
    "moe_linear_backward": (BWD, [
        dict(dout=None), dict(z=None), dict(dz=None), dict(x=None), dict(w=None), dict(ws=None), dict(dz=P(0x5008)), dict(x=P(0x2008)),
        dict(w=P(0x3008)), dict(lddout=31), dict(ldx=68), dict(ldw=68), dict(ldz=63), dict(lddz=68), dict(lddz=56), dict(lddx=63),
        dict(lddw=63), dict(db=P(0x8002)), dict(dx=P(0x6001)), dict(dw=P(0x7001)), dict(act=4, lddout=36), dict(act=4, dout=P(0x1008)),
        dict(act=9), dict(dtype=2), dict(wdtype=1), dict(R=-1), dict(N=0), dict(K=-4)]),
    "moe_layer16_forward": (LAYER, [
        dict(x=None), dict(w1=None), dict(w2=None), dict(out=None), dict(ids=None), dict(wts=None), dict(ws=None),
        dict(logits=P(0xa000)), dict(x=P(0x1008)), dict(w1=P(0x3008)), dict(w2=P(0x5008)), dict(ws=P(0x9008)), dict(W_r=P(0x2001)),
        dict(b1=P(0x4002)), dict(ids=P(0x7001)), dict(wts=P(0x8002)), dict(out=P(0x6001)), dict(ldx=63), dict(ldx=68), dict(ld1=56),
        dict(ld1=68), dict(ld2=24), dict(ld2=36), dict(ldo=63), dict(g1=4088), dict(g1=4100), dict(g2=2040), dict(g2=2052), dict(T=-1),
        dict(H=0), dict(I=0), dict(E=0), dict(k=0), dict(k=4), dict(S=2), dict(S=-1), dict(E=2048, S=1), dict(E=40, k=32, S=1),
        dict(act=3), dict(act=4), dict(act=1), dict(rs=0.0), dict(rs=float("nan")), dict(dtype=2), dict(H=2 ** 20 + 1, ldx=2 ** 21),
        dict(I=2 ** 20 + 1)]),
}


@pytest.mark.parametrize("fn,i", [(f, i) for f, (_, bad) in BAD.items() for i in range(len(bad))])
def test_bad_arguments(lib, fn, i):
    base, bad = BAD[fn]
    assert _call(getattr(lib, fn), base, **bad[i]) == INVALID, bad[i]


def test_too_many_tokens(lib):
    assert _call(lib.moe_layer16_forward, LAYER, T=65) == UNSUPPORTED
    n = ctypes.c_size_t()
    assert lib.moe_layer16_workspace_size(65, 64, 64, 4, 2, 0, ctypes.byref(n)) == UNSUPPORTED
    assert lib.moe_layer16_workspace_size(64, 64, 64, 4, 2, 0, ctypes.byref(n)) == OK


def test_no_rows_launch_nothing(lib):
    assert _call(lib.moe_linear_forward, FWD, R=0, x=None, out=None, res=None, z=None) == OK
    assert _call(lib.moe_linear_backward, BWD, R=0, dout=None, x=None, z=None, dz=None, dx=None, dw=None, db=None) == OK
    assert _call(lib.moe_layer16_forward, LAYER, T=0, x=None, out=None, ids=None, wts=None) == OK
    assert lib.moe_last_launch_count() == 0


def test_workspaces(lib):
    from quantized_grouped_gemm_topk_gb300 import binding as m
    assert _call(lib.moe_linear_forward, FWD, ws_bytes=16) == WORKSPACE
    assert _call(lib.moe_linear_backward, BWD, ws_bytes=m.moe_linear_workspace_size(4, 64, 64, True) - 1) == WORKSPACE
    assert _call(lib.moe_layer16_forward, LAYER, ws_bytes=m.moe_layer16_workspace_size(4, 64, 32, 3, 2, 1) - 1) == WORKSPACE
    for rows, K in ((1, 1), (64, 7168), (7168, 64), (14336, 7168), (100000, 8), (8, 100000)):
        for back in (False, True):
            sizes = [m.moe_linear_workspace_size(R, rows, K, back) for R in (0, 1, 2, 7, 64, 65, 128, 256, 257, 1000, 2048, 65536, 10 ** 7)]
            assert sizes == sorted(sizes) and sizes[0] >= 256
            assert sizes[-1] <= (96 << 20) + 4 * 256 * rows
    for E, k, S in ((1, 1, 0), (8, 2, 1), (256, 8, 0), (2047, 31, 1)):
        sizes = [m.moe_layer16_workspace_size(T, 7168, 2048, E, k, S) for T in range(65)]
        assert sizes == sorted(sizes)
        assert sizes[-1] <= (96 << 20) + 8 * 64 * (k + 1) * (7168 + 2048)
    for bad in ((-1, 8, 8, 0), (1, 0, 8, 0), (1, 8, 0, 1), (2 ** 30 + 1, 8, 8, 0), (1, 8, 8, 2)):
        n = ctypes.c_size_t()
        assert lib.moe_linear_workspace_size(*bad, ctypes.byref(n)) == INVALID


def test_tensors_that_do_not_fit_are_refused(lib, monkeypatch):
    """The binding checks shapes, types and strides (the device check is switched off: there is no GPU here)."""
    import torch
    from quantized_grouped_gemm_topk_gb300 import binding as m

    class Fake:
        """A CPU tensor that says it is on the current CUDA device."""

        def __init__(self, t):
            self.t = t

        def __getattr__(self, k):
            return getattr(self.t, k)

        def get_device(self):
            return 0

    monkeypatch.setattr(m, "_require_cuda", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(m, "_stream", lambda s=None: None)
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32

    def z(*shape, dtype=bf):
        return Fake(torch.zeros(*shape, dtype=dtype))

    ws = z(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="shape"):       # a gated act has two rows of weights for a column
        m.moe_linear_forward(z(4, 64), z(32, 64), z(4, 32), ws, act="swiglu")
    with pytest.raises(ValueError, match="shape"):
        m.moe_linear_forward(z(4, 64), z(64, 64), z(4, 32), ws, act="swiglu", bias=z(32, dtype=f32))
    with pytest.raises(ValueError, match="shape"):
        m.moe_linear_forward(z(4, 64), z(64, 64), z(4, 32), ws, act="swiglu", z=z(4, 32))
    with pytest.raises(ValueError, match="type"):
        m.moe_linear_forward(z(4, 64), z(32, 64), z(4, 32), ws, residual=z(4, 32, dtype=f32))
    with pytest.raises(ValueError, match="type"):
        m.moe_linear_forward(z(4, 64), z(32, 64), z(4, 32), ws, bias=z(32, dtype=torch.float16))
    with pytest.raises(ValueError, match="type"):
        m.moe_linear_forward(z(4, 64), z(32, 64), z(4, 32, dtype=f32), ws)
    with pytest.raises(KeyError):
        m.moe_linear_forward(z(4, 64), z(32, 64), z(4, 32), ws, act="relu")
    with pytest.raises(ValueError, match="takes no z"):
        m.moe_linear_backward(z(4, 32), z(4, 64), z(32, 64), z(4, 32), z(4, 32), None, None, None, ws)
    with pytest.raises(ValueError, match="shape"):
        m.moe_linear_backward(z(4, 32), z(4, 64), z(32, 64), z(4, 32), z(4, 32), None, z(32, 32), None, ws, act="gelu")
    with pytest.raises(m.MoEError):                      # no z to a gated act
        m.moe_linear_backward(z(4, 32), z(4, 64), z(64, 64), None, z(4, 64), None, None, None, z(1 << 24, dtype=torch.uint8), act="swiglu")
    args = dict(x=z(4, 64), W_r=z(64, 3, dtype=f32), logits=None, w1=z(4, 64, 64), w2=z(4, 64, 32), out=z(4, 64),
                topk_ids=z(4, 2, dtype=i32), topk_w=z(4, 2, dtype=f32), ws=ws, n_shared=1)
    for kw, what in ((dict(W_r=z(64, 4, dtype=f32)), "shape"), (dict(W_r=z(64, 3)), "type"), (dict(w1=z(4, 32, 64)), "shape"),
                     (dict(w2=z(4, 64, 32, dtype=torch.float16)), "type"), (dict(topk_ids=z(4, 2, dtype=torch.int64)), "type"),
                     (dict(topk_w=z(4, 3, dtype=f32)), "shape"), (dict(b1=z(4, 32, dtype=f32)), "shape"), (dict(x=z(4, 64, dtype=f32)), "type"),
                     (dict(logits=z(3, 4, dtype=f32), W_r=None), "shape"), (dict(w1=z(3, 64, 64)), "shape")):
        with pytest.raises(ValueError, match=what):
            m.moe_layer16_forward(**{**args, **kw})
    with pytest.raises(m.MoEError):
        m.moe_layer16_forward(**args)                    # the workspace is too small
