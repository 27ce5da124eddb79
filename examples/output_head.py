"""Trains the output head of a language model on a GB300 with this library:
layer norm, projection onto the vocabulary with softmax cross entropy (the
logits are never kept), both gradients, and AdamW on all parameters at once.
PyTorch only allocates memory and draws the synthetic data.

    python examples/output_head.py [--tokens 2048] [--width 1024] [--vocab 32768]
                                   [--steps 20] [--state-bits 8] [--dtype bf16]

The "hidden states" are noisy copies of one direction per target, so that a
head can learn them: the loss falls from log(vocab) towards zero.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_gemm_layouts_gb300 as tg  # noqa: E402


class OutputHead:
    """norm weight and bias [D] and projection [V, D] in 16 bits, with fp32
    master copies and AdamW states."""

    EPS = 1e-5

    def __init__(self, vocab, width, dtype=torch.bfloat16, state_bits=32, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.width, self.state_bits = vocab, width, state_bits
        self.code = {torch.bfloat16: tg.TG_BF16, torch.float16: tg.TG_F16}[dtype]
        self.master = [torch.ones(width, device="cuda"), torch.zeros(width, device="cuda"),
                       torch.randn(vocab, width, device="cuda", generator=gen) * 0.02]
        self.weight, self.bias, self.proj = self.params = [p.to(dtype) for p in self.master]
        self.grads = [torch.empty_like(p) for p in self.params]
        state = torch.float32 if state_bits == 32 else torch.uint8
        self.m, self.v = ([torch.zeros_like(p, dtype=state) for p in self.params] for _ in range(2))
        blocks = [(p.numel() + 255) // 256 for p in self.params]
        self.m_scale, self.v_scale = ([torch.zeros(b, device="cuda") for b in blocks] for _ in range(2))
        self.tensors = tg.make_adamw_tensors(
            self.params, self.grads, self.m, self.v, master=self.master, m_scale=self.m_scale,
            v_scale=self.v_scale)
        self.steps = 0
        self.space = {}

    def _buffers(self, x):
        """What a batch of this size needs, made once per size."""
        rows = x.shape[0]
        if rows not in self.space:
            d, v, c = self.width, self.vocab, self.code
            y, dy, dx = (torch.empty(rows, d, device="cuda", dtype=x.dtype) for _ in range(3))
            size = max(tg.tg_linear_ce_workspace_size(rows, v, d, y, d, self.proj, d, c),
                       tg.tg_linear_ce_grad_workspace_size(rows, v, d, y, d, self.proj, d, dy, d,
                                                           self.grads[2], d, c),
                       tg.tg_layernorm_grad_workspace_size(rows, d, c))
            stats = torch.empty(4, rows, device="cuda")
            self.space[rows] = y, dy, dx, stats, torch.empty(size, device="cuda", dtype=torch.uint8)
        return self.space[rows]

    def loss_and_gradients(self, x, target):
        """Mean loss over the targets inside the vocabulary (a tensor), and the
        gradient for x; the parameters' gradients are left in self.grads."""
        rows, d, v, c = x.shape[0], self.width, self.vocab, self.code
        y, dy, dx, stats, ws = self._buffers(x)
        mean, rstd, loss, lse = stats
        stream = torch.cuda.current_stream()
        tg.layernorm(rows, d, x, x.stride(0), self.weight, self.bias, self.EPS, y, d, mean, rstd, c, stream)
        tg.linear_ce(rows, v, d, y, d, self.proj, d, target, loss, lse, c, ws, ws.numel(), stream)
        share = 1.0 / ((target >= 0) & (target < v)).sum().clamp(min=1).float()
        dloss = share.expand(rows).contiguous()
        tg.linear_ce_grad(rows, v, d, y, d, self.proj, d, target, lse, dloss, dy, d, self.grads[2], d, c, ws,
                          ws.numel(), stream)
        tg.layernorm_grad(rows, d, dy, d, x, x.stride(0), self.weight, mean, rstd, dx, d, self.grads[0],
                          self.grads[1], c, ws, ws.numel(), stream)
        return loss.sum() * share, dx

    def update(self, lr, decay=0.01):
        self.steps += 1
        tg.adamw(self.tensors, tg.make_adamw_options(lr, 0.9, 0.95, 1e-8, decay, self.steps, self.code,
                                                     state_bits=self.state_bits, seed=self.steps),
                 torch.cuda.current_stream())


def batch(directions, tokens, gen, ignored=0.1):
    """Noisy directions of random targets; some tokens are not to be learned."""
    vocab = directions.shape[0]
    target = torch.randint(0, vocab, (tokens,), device="cuda", generator=gen)
    x = directions[target] + 0.5 * torch.randn(tokens, directions.shape[1], device="cuda", generator=gen)
    target[torch.rand(tokens, device="cuda", generator=gen) < ignored] = -100
    return x.to(torch.bfloat16), target


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32768)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--dtype", choices=("bf16", "f16"), default="bf16")
    a = ap.parse_args()
    dtype = {"bf16": torch.bfloat16, "f16": torch.float16}[a.dtype]
    gen = torch.Generator(device="cuda").manual_seed(1)
    directions = torch.randn(a.vocab, a.width, device="cuda", generator=gen)
    head = OutputHead(a.vocab, a.width, dtype, a.state_bits)
    for step in range(a.steps):
        x, target = batch(directions, a.tokens, gen)
        loss, _ = head.loss_and_gradients(x.to(dtype), target)
        head.update(lr=2e-2)
        print(f"step {step + 1:3d}  loss {float(loss):.4f}")


if __name__ == "__main__":
    main()
