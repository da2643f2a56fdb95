"""The training example's block: its gradients against autograd in 64 bits on
the same routing, and a falling loss."""
import importlib.util
import os

import pytest
import torch

from util import cuda_device, rel_l2

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_block_gradients():
    """Two 8-bit roundings (relative 2^-4 each at most) stand between the block and the 64-bit one."""
    cuda_device()
    ex = _example()
    T, H, I, E, k = 300, 256, 192, 8, 3
    b = ex.Block(T, H, I, E, k, seed=3)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    out = b.forward(x)
    v = b.saved[4]
    ids, tw = v["topk_ids"].long().clone(), v["topk_w"].double().clone()
    grads = b.backward(dout)

    p = {n: getattr(b, n).double().requires_grad_() for n in ("gamma", "beta", "w1", "w2", "wp")}
    x64 = x.double().requires_grad_()
    mu = x64.mean(1, keepdim=True)
    xn = (x64 - mu) / torch.sqrt((x64 - mu).pow(2).mean(1, keepdim=True) + ex.EPS) * p["gamma"] + p["beta"]
    ref = xn @ p["wp"][0].t()
    for j in range(k):
        h = torch.einsum("th,tnh->tn", xn, p["w1"][ids[:, j]])
        a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        ref = ref + tw[:, j:j + 1] * torch.einsum("ti,thi->th", a, p["w2"][ids[:, j]])
    (ref * dout.double()).sum().backward()
    assert rel_l2(out.double().cpu().numpy(), ref.detach().cpu().numpy()) < 2 * 2.0 ** -4
    for n, want in (("x", x64.grad), *((n, t.grad) for n, t in p.items())):
        assert rel_l2(grads[n].double().cpu().numpy(), want.cpu().numpy()) < 2 * 2.0 ** -4, n


def test_training_lowers_the_loss():
    cuda_device()
    losses = _example().train(steps=12, tokens=512, hidden=256, inner=128, experts=8, k=2)
    assert losses[-1] < 0.8 * losses[0] and all(l == l for l in losses), losses


@pytest.mark.parametrize("T,H,I,E,k", [(300, 256, 192, 8, 3), (257, 128, 320, 5, 2)])
def test_block_gradients_through_the_router(T, H, I, E, k):
    """The routing weights are functions of x and of the router here, only the choice of experts is held fixed. Bound as
    above; dw_row is a sum over columns of one 8-bit rounding's errors, and the router's gradient a combination of them."""
    cuda_device()
    b = _example().Block(T, H, I, E, k, seed=4)
    g = torch.Generator(device="cuda").manual_seed(10)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    dout = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    b.forward(x)
    v = b.saved[4]
    ids, inv = v["topk_ids"].long().clone(), v["inv"].long().clone()
    grads = b.backward(dout, router=True)
    fixed = b.backward(dout)

    p = {n: getattr(b, n).double().requires_grad_() for n in ("gamma", "beta", "router", "w1", "w2", "wp")}
    x64 = x.double().requires_grad_()
    mu = x64.mean(1, keepdim=True)
    xn = (x64 - mu) / torch.sqrt((x64 - mu).pow(2).mean(1, keepdim=True) + 1e-5) * p["gamma"] + p["beta"]
    tw = torch.softmax((xn @ p["router"]).gather(1, ids), 1)
    tw.retain_grad()
    ref = xn @ p["wp"][0].t()
    for j in range(k):
        h = torch.einsum("th,tnh->tn", xn, p["w1"][ids[:, j]])
        a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
        ref = ref + tw[:, j:j + 1] * torch.einsum("ti,thi->th", a, p["w2"][ids[:, j]])
    (ref * dout.double()).sum().backward()
    dw = torch.empty(T * k, dtype=torch.float64, device="cuda")
    dw[inv] = tw.grad.reshape(-1)
    for n, want in (("x", x64.grad), ("dw_row", dw), *((n, t.grad) for n, t in p.items())):
        assert rel_l2(grads[n].double().cpu().numpy(), want.cpu().numpy()) < 2 * 2.0 ** -4, n
    # without the router: the same but for that path
    assert "router" not in fixed
    for n in ("w1", "w2", "wp", "dw_row"):
        assert torch.equal(grads[n], fixed[n]), n
    assert not torch.equal(grads["x"], fixed["x"])


def test_training_moves_the_router():
    cuda_device()
    ex = _example()
    b = ex.Block(128, 128, 64, 4, 2, seed=1)
    x = torch.randn(128, 128, device="cuda").bfloat16()
    before = b.router.clone()
    b.forward(x)
    b.step(b.backward(x, router=True), 0.1)
    assert bool(torch.isfinite(b.router).all()) and not torch.equal(b.router, before)
