"""Trains a layer of experts on a GB300 with this library: a router, the grouping
of rows by expert, the experts' two products with a ReLU between them, the weighted
sum, all their gradients, and AdamW.  PyTorch only allocates memory, draws the
synthetic data and multiplies by the router's matrix.

    python examples/experts.py [--tokens 4096] [--width 512] [--hidden 1024]
                               [--experts 16] [--chosen 2] [--steps 20]

The layer learns a fixed random map of its input; the router's bias is moved
after each step against the experts' load, so that it stays even.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_gemm_layouts_gb300 as tg  # noqa: E402


class Experts:
    """Router [E, D] and the experts' matrices [E, F, D] and [E, D, F] in 16 bits, with
    fp32 master copies and AdamW states; workspaces and activations for T tokens."""

    def __init__(self, tokens, width, hidden, experts, chosen, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes = tokens, width, hidden, experts, chosen
        self.code = {torch.bfloat16: tg.TG_BF16, torch.float16: tg.TG_F16}[dtype]
        draw = lambda *s: torch.randn(*s, device="cuda", generator=gen) * s[-1]**-0.5  # noqa: E731
        self.master = [draw(experts, width), draw(experts, hidden, width), draw(experts, width, hidden)]
        self.params = self.router, self.w1, self.w2 = [p.to(dtype) for p in self.master]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.states = [[torch.zeros_like(p) for p in self.master] for _ in range(2)]
        self.tensors = tg.make_adamw_tensors(self.params, self.grads, *self.states, master=self.master)
        self.bias = torch.zeros(experts, device="cuda")
        new = lambda *s, like=dtype: torch.empty(*s, device="cuda", dtype=like)  # noqa: E731
        rows = tokens * chosen
        self.index, self.weight = new(tokens, chosen, like=torch.int32), new(tokens, chosen, like=torch.float32)
        self.offset, self.row = new(experts + 1, like=torch.int32), new(rows, like=torch.int32)
        self.place, self.dweight = new(tokens, chosen, like=torch.int32), new(tokens, chosen, like=torch.float32)
        self.logits, self.dlogits = new(tokens, experts), new(tokens, experts)
        self.h, self.dh = new(rows, hidden), new(rows, hidden)
        self.y, self.dy, self.dxg = new(rows, width), new(rows, width), new(rows, width)
        self.out, self.dx = new(tokens, width), new(tokens, width)
        self.options = tg.make_route_options(chosen, tg.TG_ROUTE_SIGMOID, renormalise=True)
        self.workspace = new(max(1, tg.tg_group_rows_workspace_size(rows, experts)), like=torch.uint8)

    def forward(self, x):
        t, d, f, e, k = self.sizes
        s = torch.cuda.current_stream()
        torch.mm(x, self.router.T, out=self.logits)
        tg.route(t, e, self.logits, e, self.bias, self.index, self.weight, self.code, self.options, s)
        tg.group_rows(t * k, e, self.index, self.offset, self.row, self.place, self.workspace, self.workspace.numel(), s)
        tg.grouped_gemm(t * k, f, d, e, x, t, d, self.row, k, self.w1, d, f * d, tg.TG_OP_T, self.offset, self.h, f, self.code,
                        tg.make_group_epilogue(relu=True), s)
        tg.grouped_gemm(t * k, d, f, e, self.h, t * k, f, None, 1, self.w2, f, d * f, tg.TG_OP_T, self.offset, self.y, d,
                        self.code, stream=s)
        tg.combine(t, k, d, self.y, t * k, d, self.place, self.weight, self.out, d, self.code, s)
        return self.out

    def backward(self, x, dout):
        """Gradients of the parameters (in .grads) and of x (returned)."""
        t, d, f, e, k = self.sizes
        r, code, s = t * k, self.code, torch.cuda.current_stream()
        tg.combine_grad(t, k, d, dout, d, self.y, r, d, self.place, self.weight, self.dy, d, self.dweight, code, s)
        tg.route_grad(t, e, self.logits, e, self.index, self.dweight, self.dlogits, e, code, self.options, s)
        tg.grouped_gemm_grad(r, d, f, e, self.dy, d, self.h, r, f, None, 1, self.offset, self.grads[2], f, d * f, tg.TG_OP_T, code, s)
        tg.grouped_gemm(r, f, d, e, self.dy, r, d, None, 1, self.w2, f, d * f, tg.TG_OP_N, self.offset, self.dh, f, code,
                        tg.make_group_epilogue(relu_of=self.h, ld_relu=f), s)
        tg.grouped_gemm_grad(r, f, d, e, self.dh, f, x, t, d, self.row, k, self.offset, self.grads[1], d, f * d, tg.TG_OP_T, code, s)
        tg.grouped_gemm(r, d, f, e, self.dh, r, f, None, 1, self.w1, d, f * d, tg.TG_OP_N, self.offset, self.dxg, d, code, stream=s)
        tg.combine(t, k, d, self.dxg, r, d, self.place, None, self.dx, d, code, s)
        torch.mm(self.dlogits.T, x, out=self.grads[0])
        return self.dx + self.dlogits @ self.router

    def step(self, number, lr=1e-3, rate=1e-3):
        tg.adamw(self.tensors, tg.make_adamw_options(lr, 0.9, 0.99, 1e-8, 0.0, number, self.code), torch.cuda.current_stream())
        load = self.offset.diff().float()  # experts with more than their share come later
        self.bias -= rate * torch.sign(load - load.mean())


def main():
    ap = argparse.ArgumentParser()
    for name, default in (("tokens", 4096), ("width", 512), ("hidden", 1024), ("experts", 16), ("chosen", 2), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=default)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    layer = Experts(a.tokens, a.width, a.hidden, a.experts, a.chosen)
    target = torch.randn(a.width, a.width, device="cuda", generator=gen).bfloat16() * a.width**-0.5
    for step in range(1, a.steps + 1):
        x = torch.randn(a.tokens, a.width, device="cuda", generator=gen).bfloat16()
        off = layer.forward(x) - x @ target
        layer.backward(x, (off * (2 / off.numel() * 1e3)).contiguous())
        layer.step(step)
        print(f"step {step}: loss {off.float().square().mean().item():.4f}, "
              f"largest load {layer.offset.diff().max().item() * a.experts / (a.tokens * a.chosen):.2f} of even")
    status, detail = tg.tg_debug_status()
    if status != tg.TG_OK:
        raise RuntimeError(f"device watchdog fired: {detail:#x}")


if __name__ == "__main__":
    main()
