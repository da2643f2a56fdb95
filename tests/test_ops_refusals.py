"""The training-side operators refuse what they cannot compute, on the host,
before any device work (no GPU needed: a call that reached the CUDA runtime
here would return the CUDA error code)."""
import ctypes

import pytest

P = ctypes.c_void_p
OK, INVALID, WORKSPACE = 0, 1, 3


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


NORM_F = dict(x=P(0x1000), ldx=64, gamma=P(0x2000), beta=P(0x3000), eps=1e-5, T=4, H=64, dtype=0, wdtype=2,
              y=P(0x4000), ldy=64, mean=None, rstd=None, stream=None)
NORM_B = dict(dy=P(0x1000), lddy=64, x=P(0x2000), ldx=64, gamma=P(0x3000), mean=P(0x4000), rstd=P(0x5000), T=4, H=64,
              dtype=0, wdtype=2, dx=P(0x6000), lddx=64, dgamma=P(0x7000), dbeta=P(0x8000), ws=P(0x9000),
              ws_bytes=1 << 20, stream=None)
CKPT_F = dict(h=P(0x1000), ldh=128, w=None, R=4, I=64, dtype=0, act=0, alpha=1.0, limit=0.0, y=P(0x2000), ldy=64,
              q=P(0x3000), ldq=128, s=P(0x4000), stream=None)
CKPT_B = dict(dy=P(0x1000), lddy=64, q=P(0x2000), ldq=128, s=P(0x3000), w=None, R=4, I=64, dtype=0, act=0, alpha=1.0,
              limit=0.0, dh=P(0x4000), lddh=128, dw=None, y=None, ldy=0, stream=None)
MM = dict(x=P(0x1000), ldx=64, w=P(0x2000), wg=4096, ldw=64, trans=0, off=P(0x3000), R=8, N=64, K=64, G=2, dtype=0,
          out=P(0x4000), ldo=64, out_dtype=0, ws=P(0x5000), ws_bytes=1 << 27, stream=None)
WGRAD = dict(dy=P(0x1000), lddy=64, x=P(0x2000), ldx=64, off=P(0x3000), R=8, N=64, K=64, G=2, dtype=0, dw=P(0x4000),
             dwg=4096, lddw=64, out_dtype=2, ws=P(0x5000), ws_bytes=1 << 27, stream=None)
QR = dict(x=P(0x1000), ldx=256, R=4, C=256, dtype=0, q=P(0x2000), ldq=256, s=P(0x3000), lds=2, stream=None)
QW = dict(w=P(0x1000), wg=4096, ldw=64, G=2, N=64, K=64, dtype=0, q=P(0x2000), qg=4096, ldq=64, s=P(0x3000),
          qt=P(0x4000), qtg=4096, ldqt=64, st=P(0x5000), stream=None)
FP8 = dict(xq=P(0x1000), ldx=64, xs=P(0x2000), ldxs=1, wq=P(0x3000), wg=4096, ldw=64, wsc=P(0x4000), off=P(0x5000),
           R=8, N=64, K=64, G=2, out=P(0x6000), ldo=64, out_dtype=0, ws=P(0x7000), ws_bytes=1 << 27, stream=None)

BAD = {
    "moe_layer_norm_forward": (NORM_F, [
        dict(x=None), dict(x=P(0x1001)), dict(y=None), dict(T=-1), dict(H=0), dict(ldx=63), dict(ldy=63), dict(dtype=3),
        dict(wdtype=1), dict(eps=-1.0), dict(eps=float("nan")), dict(gamma=P(0x2002)), dict(mean=P(0x4002))]),
    "moe_layer_norm_backward": (NORM_B, [
        dict(dy=None), dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(ws=None), dict(lddy=1),
        dict(lddx=63), dict(dtype=-1), dict(wdtype=1), dict(H=-4), dict(ws=P(0x9004)), dict(dgamma=P(0x7001))]),
    "moe_act_ckpt_forward": (CKPT_F, [
        dict(h=None), dict(y=None), dict(q=None), dict(s=None), dict(R=-1), dict(I=0), dict(dtype=2), dict(act=4),
        dict(act=1, limit=0.0), dict(act=1, limit=float("nan")), dict(ldh=127), dict(ldq=127), dict(ldy=63),
        dict(I=2 ** 31 - 1), dict(w=P(0x1002))]),
    "moe_act_ckpt_backward": (CKPT_B, [
        dict(dy=None), dict(q=None), dict(s=None), dict(dh=None), dict(dtype=2), dict(act=-1), dict(lddh=127),
        dict(lddy=63), dict(y=P(0x6000), ldy=63), dict(dw=P(0x6002)), dict(R=-1)]),
    "moe_grouped_mm": (MM, [
        dict(x=None), dict(w=None), dict(out=None), dict(off=None), dict(ws=None), dict(R=-1), dict(N=0), dict(K=0),
        dict(G=0), dict(G=2049), dict(dtype=2), dict(out_dtype=1), dict(trans=2), dict(ldx=63), dict(ldx=68),
        dict(ldw=68), dict(ldw=56), dict(wg=4088), dict(wg=4100), dict(ldo=63), dict(x=P(0x1008)), dict(w=P(0x2002)),
        dict(off=P(0x3002)), dict(out=P(0x4001)), dict(ws=P(0x5008)), dict(trans=1, ldw=56)]),
    "moe_grouped_mm_wgrad": (WGRAD, [
        dict(dy=None), dict(x=None), dict(dw=None), dict(off=None), dict(ws=None), dict(lddy=60), dict(lddy=68),
        dict(ldx=68), dict(lddw=63), dict(dwg=4000), dict(dtype=2), dict(out_dtype=1), dict(dw=P(0x4002)), dict(N=-1),
        dict(dy=P(0x1002))]),
    "moe_fp8_quant_rows": (QR, [
        dict(x=None), dict(q=None), dict(s=None), dict(ldx=255), dict(ldq=255), dict(lds=1), dict(C=0), dict(R=-1),
        dict(dtype=5), dict(s=P(0x3002))]),
    "moe_fp8_quant_weights": (QW, [
        dict(w=None), dict(q=None), dict(s=None), dict(qt=None), dict(st=None), dict(wg=4095), dict(qg=64),
        dict(qtg=64), dict(ldw=63), dict(ldq=63), dict(ldqt=63), dict(G=0), dict(dtype=-2)]),
    "moe_fp8_mm": (FP8, [
        dict(xq=None), dict(xs=None), dict(wq=None), dict(wsc=None), dict(out=None), dict(off=None), dict(ws=None),
        dict(ldx=56), dict(ldx=72), dict(ldw=72), dict(wg=4104), dict(wg=64), dict(ldxs=0), dict(ldo=63),
        dict(out_dtype=3), dict(xq=P(0x1008)), dict(G=2049), dict(K=-1)]),
}


@pytest.mark.parametrize("fn,i", [(f, i) for f, (_, bad) in BAD.items() for i in range(len(bad))])
def test_bad_arguments(lib, fn, i):
    base, bad = BAD[fn]
    assert _call(getattr(lib, fn), base, **bad[i]) == INVALID, bad[i]


def test_workspaces_too_small(lib):
    assert _call(lib.moe_layer_norm_backward, NORM_B, ws_bytes=4 * 2 * 64 * 4 - 1) == WORKSPACE
    for fn, base in ((lib.moe_grouped_mm, MM), (lib.moe_grouped_mm_wgrad, WGRAD), (lib.moe_fp8_mm, FP8)):
        assert _call(fn, base, ws_bytes=16) == WORKSPACE


def test_no_rows_launch_nothing(lib):
    """Zero rows are legal, also with NULL row buffers; nothing is enqueued (here: no CUDA error)."""
    assert _call(lib.moe_layer_norm_forward, NORM_F, T=0, x=None, y=None) == OK
    assert _call(lib.moe_layer_norm_backward, NORM_B, T=0, x=None, dy=None, dx=None, mean=None, rstd=None, ws=None,
                 dgamma=None, dbeta=None) == OK
    assert _call(lib.moe_act_ckpt_forward, CKPT_F, R=0, h=None, y=None, q=None, s=None) == OK
    assert _call(lib.moe_act_ckpt_backward, CKPT_B, R=0, dy=None, q=None, s=None, dh=None) == OK
    assert _call(lib.moe_grouped_mm, MM, R=0, x=None, out=None) == OK
    assert _call(lib.moe_fp8_mm, FP8, R=0, xq=None, xs=None, out=None) == OK
    assert _call(lib.moe_fp8_quant_rows, QR, R=0, x=None, q=None, s=None) == OK
    assert lib.moe_last_launch_count() == 0


def test_workspace_sizes(lib):
    from quantized_grouped_gemm_topk_gb300 import binding as m
    assert m.moe_layer_norm_workspace_size(4, 64) == 4 * 2 * 64 * 4
    assert m.moe_layer_norm_workspace_size(10 ** 6, 64) == 1024 * 2 * 64 * 4
    for kind in (m.MOE_MM_ROWS, m.MOE_MM_WGRAD, m.MOE_MM_FP8):
        for R in (0, 1, 3, 64, 1000, 65536, 10 ** 7):
            for N, K in ((1, 1), (64, 7168), (7168, 64), (7168, 7168), (100000, 8), (8, 100000)):
                for G in (1, 2, 256, 2048):
                    assert 256 <= m.moe_mm_workspace_size(kind, R, N, K, G) <= 256 + (64 << 20)
    with pytest.raises(m.MoEError):
        m.moe_mm_workspace_size(3, 1, 1, 1, 1)
    with pytest.raises(m.MoEError):
        m.moe_mm_workspace_size(0, 1, 1, 1, 2049)
    with pytest.raises(m.MoEError):
        m.moe_layer_norm_workspace_size(1, 0)


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

    with pytest.raises(ValueError, match="shape"):
        m.moe_layer_norm_forward(z(4, 64), z(32), None, 1e-5, z(4, 64))
    with pytest.raises(ValueError, match="type"):
        m.moe_layer_norm_forward(z(4, 64), z(64, dtype=torch.float16), None, 1e-5, z(4, 64))
    with pytest.raises(ValueError, match="type"):
        m.moe_layer_norm_forward(z(4, 64, dtype=torch.float64), None, None, 1e-5, z(4, 64, dtype=torch.float64))
    with pytest.raises(ValueError, match="contiguous"):
        m.moe_layer_norm_forward(Fake(torch.zeros(64, 4, dtype=bf).t()), None, None, 1e-5, z(4, 64))
    with pytest.raises(ValueError, match="overlap"):
        m.moe_layer_norm_forward(Fake(torch.zeros(1, 64, dtype=bf).expand(4, 64)), None, None, 1e-5, z(4, 64))
    with pytest.raises(ValueError, match="axes"):
        m.moe_layer_norm_forward(z(64), None, None, 1e-5, z(64))
    off = z(3, dtype=i32)
    with pytest.raises(ValueError, match="shape"):
        m.moe_grouped_mm(z(4, 64), z(2, 32, 72), off, z(4, 32), z(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="type"):
        m.moe_grouped_mm(z(4, 64), z(2, 32, 64), z(3, dtype=torch.int64), z(4, 32), z(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        m.moe_grouped_mm(z(4, 64), z(2, 32, 64), z(2, dtype=i32), z(4, 32), z(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="type"):
        m.moe_grouped_mm_wgrad(z(4, 64, dtype=f32), z(4, 64), off, z(2, 64, 64), z(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        m.moe_act_ckpt_forward(z(4, 64), None, z(4, 64), z(4, 64, dtype=torch.uint8), z(4, 2, dtype=f32))
    with pytest.raises(KeyError):
        m.moe_act_ckpt_forward(z(4, 128), None, z(4, 64), z(4, 128, dtype=torch.uint8), z(4, 2, dtype=f32), act="relu")
    with pytest.raises(ValueError, match="shape"):
        m.moe_fp8_mm(z(4, 256, dtype=torch.uint8), z(4, 1, dtype=f32), z(1, 64, 256, dtype=torch.uint8),
                     z(1, 1, 2, dtype=f32), z(4, 64), z(256, dtype=torch.uint8))
    cpu = torch.zeros(4, 64, dtype=bf)
    with pytest.raises(ValueError, match="device"):
        m.moe_layer_norm_forward(cpu, None, None, 1e-5, cpu)


BIG = 2 ** 30 + 1       # one past the longest row; 2^31 - 100: rounding up to a block of 128 leaves 32 bits


@pytest.mark.parametrize("n", [BIG, 2 ** 31 - 100])
def test_rows_too_long(lib, n):
    """Refused like the products' sizes: the kernels round up to blocks and step past the end in 32 bits."""
    wide = dict(ldx=n, ldy=n)
    assert _call(lib.moe_layer_norm_forward, NORM_F, H=n, **wide) == INVALID
    assert _call(lib.moe_layer_norm_backward, NORM_B, H=n, lddy=n, ldx=n, lddx=n, ws_bytes=1 << 40) == INVALID
    need = ctypes.c_size_t()
    assert lib.moe_layer_norm_workspace_size(4, n, ctypes.byref(need)) == INVALID
    assert _call(lib.moe_act_ckpt_forward, CKPT_F, act=3, I=n, ldh=n, ldy=n, ldq=n) == INVALID
    assert _call(lib.moe_act_ckpt_backward, CKPT_B, act=3, I=n, lddy=n, ldq=n, lddh=n) == INVALID
    assert _call(lib.moe_fp8_quant_rows, QR, C=n, ldx=n, ldq=n, lds=n) == INVALID
    assert _call(lib.moe_fp8_quant_weights, QW, K=n, ldw=n, ldq=n, wg=64 * n, qg=64 * n, qtg=64 * n) == INVALID
    assert _call(lib.moe_fp8_quant_weights, QW, N=n, ldqt=n, wg=64 * n, qg=64 * n, qtg=64 * n) == INVALID


@pytest.mark.parametrize("G", [1, 8, 64])
@pytest.mark.parametrize("N,K", [(64, 8192), (128, 4096), (2880, 2880), (7168, 2048), (4096, 7168), (129, 1024)])
def test_a_workspace_for_the_largest_batch_serves_every_batch(lib, N, K, G):
    """Sized for many rows, used with few (which are cut into more pieces): never MOE_ERR_WORKSPACE. Each call stops at
    another argument behind the workspace's check, so nothing is enqueued."""
    from quantized_grouped_gemm_topk_gb300 import binding as m
    small = [*range(1, 130), 200, 255, 256, 257, 500, 1000, 2047, 2048, 4097, 9000, 20000, 65536]
    for kind, fn, base, kw in (
            (m.MOE_MM_ROWS, lib.moe_grouped_mm, MM, dict(ldx=K, wg=N * K, ldw=K, ldo=N, dtype=9)),
            (m.MOE_MM_WGRAD, lib.moe_grouped_mm_wgrad, WGRAD, dict(lddy=N, ldx=K, dwg=N * K, lddw=K, dtype=9)),
            (m.MOE_MM_FP8, lib.moe_fp8_mm, FP8, dict(ldx=K, ldw=K, ldxs=64, ldo=N, wg=N * K, out_dtype=9))):
        sizes = [m.moe_mm_workspace_size(kind, R, N, K, G) for R in small]
        assert sizes == sorted(sizes)
        for most in (20000, 65536):
            have = m.moe_mm_workspace_size(kind, most, N, K, G)
            for R in small:
                if R <= most:
                    assert _call(fn, base, R=R, N=N, K=K, G=G, ws_bytes=have, **kw) == INVALID, (kind, R)
