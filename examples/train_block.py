"""Trains one Mixture-of-Experts block with 16-bit experts on synthetic data.

The block is  out = experts(norm(x)) + norm(x) . Wp^T : a layer norm, top-k
routing and dispatch, the experts' two grouped products with SwiGLU between
them, the combine, and next to the experts an always-on FP8 projection with a
scale for each block of 128. The backward pass recomputes the experts'
activation from its 8-bit checkpoint, and the router is trained through the
routing weights. The products, the norm, the activation and the routing run in
the library's kernels; PyTorch holds the memory, gathers rows by index, takes
the routing weights back to the router (as the layer's backward, which leaves
the router's two dense products to its caller) and applies the update.

    python examples/train_block.py [--steps 30] [--tokens 2048] [--hidden 1024]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_grouped_gemm_topk_gb300 as m  # noqa: E402

E4M3 = torch.float8_e4m3fn
EPS = 1e-5


class Block:
    """Weights, workspaces and one step's saved tensors."""

    def __init__(self, T, H, I, E, k, seed=0, device="cuda"):
        self.T, self.H, self.I, self.E, self.k = T, H, I, E, k
        g = torch.Generator(device=device).manual_seed(seed)

        def w(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).bfloat16()

        self.gamma, self.beta = torch.ones(H, device=device), torch.zeros(H, device=device)
        self.router = torch.randn(H, E, generator=g, device=device) * H ** -0.5
        self.w1, self.w2 = w(E, 2 * I, H, std=H ** -0.5), w(E, H, I, std=I ** -0.5)
        self.wp = w(1, H, H, std=H ** -0.5)
        # routing and dispatch of the layer; its expert products are not used here
        self.cfg = m.make_config(H, I, E, k, T_max=T, wfmt="mxfp8")
        self.ws = torch.zeros(m.moe_workspace_size(self.cfg), dtype=torch.uint8, device=device)
        R = self.R = T * k
        sizes = [m.moe_mm_workspace_size(m.MOE_MM_ROWS, R, n, c, E) for n, c in ((2 * I, H), (H, I), (I, H), (H, 2 * I))]
        sizes += [m.moe_mm_workspace_size(m.MOE_MM_WGRAD, R, n, c, E) for n, c in ((H, I), (2 * I, H))]
        sizes += [m.moe_mm_workspace_size(m.MOE_MM_WGRAD, T, H, H, 1), m.moe_mm_workspace_size(m.MOE_MM_FP8, T, H, H)]
        self.mm_ws = torch.zeros(max(sizes), dtype=torch.uint8, device=device)
        self.norm_ws = torch.empty(m.moe_layer_norm_workspace_size(T, H), dtype=torch.uint8, device=device)
        self.all_rows = torch.tensor([0, T], dtype=torch.int32, device=device)

    def _new(self, *shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=self.w1.device)

    def _quant_rows(self, x):
        q, s = self._new(*x.shape, dtype=E4M3), self._new(x.shape[0], -(-x.shape[1] // 128), dtype=torch.float32)
        m.moe_fp8_quant_rows(x, q, s)
        return q, s

    def forward(self, x):
        """x [T, H] bf16 -> out [T, H] bf16; keeps what backward() needs, the experts' h in 8 bits."""
        T, H, I, R = self.T, self.H, self.I, self.R
        xn, mean, rstd = self._new(T, H), self._new(T, dtype=torch.float32), self._new(T, dtype=torch.float32)
        m.moe_layer_norm_forward(x, self.gamma, self.beta, EPS, xn, mean, rstd)

        logits = self._new(T, self.E, dtype=torch.float32)
        m.moe_router_logits(self.cfg, xn, self.router, T, logits, self.ws)
        v = m.ws_tensor_views(self.cfg, self.ws, T)
        m.moe_route_dispatch(self.cfg, logits, xn, T, m.dispatch_struct(v), self.ws)
        src = torch.div(v["perm_src"], self.k, rounding_mode="floor")
        xg = xn.index_select(0, src)

        h, y, z = self._new(R, 2 * I), self._new(R, I), self._new(R, H)
        m.moe_grouped_mm(xg, self.w1, v["offsets"], h, self.mm_ws)
        q, s = self._new(R, 2 * I, dtype=E4M3), self._new(R, 2 * -(-I // 128), dtype=torch.float32)
        m.moe_act_ckpt_forward(h, v["w_row"], y, q, s)
        m.moe_grouped_mm(y, self.w2, v["offsets"], z, self.mm_ws)
        out = self._new(T, H)
        m.moe_combine(self.cfg, z, v["inv"], None, T, out)

        # the projection beside the experts: weights quantised once a step, with the transposed copy for backward
        nb = -(-H // 128)
        wq, wtq = self._new(1, H, H, dtype=E4M3), self._new(1, H, H, dtype=E4M3)
        wsc, wtsc = self._new(1, nb, nb, dtype=torch.float32), self._new(1, nb, nb, dtype=torch.float32)
        m.moe_fp8_quant_weights(self.wp, wq, wsc, wtq, wtsc)
        p = self._new(T, H)
        m.moe_fp8_mm(*self._quant_rows(xn), wq, wsc, p, self.mm_ws)
        self.saved = (x, xn, mean, rstd, v, src, xg, q, s, wtq, wtsc)
        return out + p

    def backward(self, dout, router=False):
        """Gradients of L = sum(dout * forward(x)) by name. The routing weights count as constants, and dw_row is L's
        gradient by them (by dispatched row); with router=True they are functions of x and of the router (the choice of
        experts stays fixed): "router" is returned too, and x, gamma and beta include that path."""
        x, xn, mean, rstd, v, src, xg, q, s, wtq, wtsc = self.saved
        T, H, I, R, off = self.T, self.H, self.I, self.R, v["offsets"]
        dz = dout.index_select(0, src)
        dy = self._new(R, I)
        m.moe_grouped_mm(dz, self.w2, off, dy, self.mm_ws, trans_w=True)
        dh, dw_row, y = self._new(R, 2 * I), self._new(R, dtype=torch.float32), self._new(R, I)
        m.moe_act_ckpt_backward(dy, q, s, v["w_row"], dh, dw_row, y)
        dw2, dw1 = torch.empty_like(self.w2), torch.empty_like(self.w1)
        m.moe_grouped_mm_wgrad(dz, y, off, dw2, self.mm_ws)
        m.moe_grouped_mm_wgrad(dh, xg, off, dw1, self.mm_ws)
        dxg, dxn = self._new(R, H), self._new(T, H)
        m.moe_grouped_mm(dh, self.w1, off, dxg, self.mm_ws, trans_w=True)
        m.moe_combine(self.cfg, dxg, v["inv"], None, T, dxn)

        dp, dwp = self._new(T, H), torch.empty_like(self.wp)
        m.moe_fp8_mm(*self._quant_rows(dout), wtq, wtsc, dp, self.mm_ws)
        m.moe_grouped_mm_wgrad(dout, xn, self.all_rows, dwp, self.mm_ws)

        dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(self.gamma), torch.empty_like(self.beta)
        grads = {"x": dx, "gamma": dgamma, "beta": dbeta, "w1": dw1, "w2": dw2, "wp": dwp, "dw_row": dw_row}
        dxn = dxn + dp
        if router:
            dlogits = self._dlogits(v, dw_row)
            grads["router"] = xn.float().t() @ dlogits
            dxn = (dxn.float() + dlogits @ self.router.t()).bfloat16()
        m.moe_layer_norm_backward(dxn, x, self.gamma, mean, rstd, dx, dgamma, dbeta, self.norm_ws)
        return grads

    def _dlogits(self, v, dw_row):
        """The routing weights are the softmax p of a token's chosen logits: d logit_j = p_j (d p_j - sum_i p_i d p_i)."""
        p, dp = v["topk_w"], dw_row[v["inv"].long()].view(self.T, self.k)
        d = p * (dp - (p * dp).sum(1, keepdim=True))
        return torch.zeros(self.T, self.E, device=d.device).scatter_(1, v["topk_ids"].long(), d)

    def step(self, grads, lr):
        for name in ("gamma", "beta", "router", "w1", "w2", "wp"):
            if name in grads:
                getattr(self, name).add_(grads[name], alpha=-lr)


def train(steps=30, tokens=2048, hidden=1024, inner=512, experts=16, k=4, lr=0.1, seed=0):
    """Mean squared error against a fixed target map, by step."""
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    block = Block(tokens, hidden, inner, experts, k, seed)
    target_w = torch.randn(hidden, hidden, generator=g, device="cuda") * hidden ** -0.5
    losses = []
    x = torch.randn(tokens, hidden, generator=g, device="cuda").bfloat16()
    target = x.float() @ target_w
    for _ in range(steps):
        err = block.forward(x).float() - target
        losses.append(float(err.square().mean()))
        block.step(block.backward((err * (2.0 / tokens)).bfloat16(), router=True), lr)
    status = m.moe_mm_read_status(block.mm_ws) | m.moe_read_status(block.cfg, block.ws)
    if status:
        raise RuntimeError(f"device status {status:#x}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=1024)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.steps, a.tokens, a.hidden)):
        print(f"step {i:3d}  loss {loss:.4f}")
