"""The example of a layer of experts: it runs, and its gradients are those of automatic
differentiation in 64 bits."""
import os
import subprocess
import sys

import pytest
import torch

from rows_reference import HALF_ULP

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_runs():
    run = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "experts.py"), "--tokens", "300", "--width", "72", "--hidden",
                          "136", "--experts", "6", "--chosen", "3", "--steps", "3"], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr
    assert run.stdout.count("loss") == 3 and "nan" not in run.stdout


@pytest.mark.parametrize("tokens,chosen", [(1, 2), (515, 2), (64, 1)])
def test_gradients(tg, tokens, chosen):
    import experts
    width, hidden, count = 64, 96, 5
    layer = experts.Experts(tokens, width, hidden, count, chosen)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(tokens, width, device="cuda", generator=gen).bfloat16()
    dout = torch.randn(tokens, width, device="cuda", generator=gen).bfloat16()
    out = layer.forward(x)
    dx = layer.backward(x, dout)
    leaves = [v.double().requires_grad_() for v in (x, *layer.params)]
    xx, router, w1, w2 = leaves
    # the logits as they were rounded, with the exact ones' derivative
    exact = xx @ router.T
    logits = exact + (layer.logits.double() - exact).detach()
    index = layer.index.long()
    s = torch.sigmoid(logits).gather(1, index)
    weight = s / s.sum(1, keepdim=True)
    want = torch.zeros(tokens, width, device="cuda", dtype=torch.float64)
    for j in range(chosen):
        hid = torch.relu(torch.einsum("td,tfd->tf", xx, w1[index[:, j]]))
        want = want + weight[:, j, None] * torch.einsum("tf,tdf->td", hid, w2[index[:, j]])
    grads = torch.autograd.grad((want * dout.double()).sum(), leaves)
    # a chain of at most five tensors in 16 bits on the way, each off by 2^-8 of a value, and
    # sums over products of either sign of them, six deviations wide.  With one expert per
    # token its renormalised weight is s / s = 1: the router's gradient is 0, and what the
    # 64-bit form has in its place is its own rounding, 2^-53 of terms below 1000
    for got, exact_grad in zip((out, dx, *layer.grads), (want, *grads)):
        size = exact_grad.square().mean().sqrt()
        assert ((got.double() - exact_grad).abs() <= 5 * HALF_ULP[torch.bfloat16] * (exact_grad.abs() + 6 * size) + 1000 * 2.0**-53).all()
