"""A token whose upstream gradient is infinite leaves the others' rows of dH alone."""
import math

import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d", [(50, 900, 72), (2500, 600, 64)])
def test_an_infinite_upstream_gradient(tg, t, v, d, dt, bad):
    g = torch.Generator(device="cuda").manual_seed(t)
    code = tg.TG_BF16 if dt == torch.bfloat16 else tg.TG_F16
    h, w = ref.rows(g, t, d, 0, dt), ref.rows(g, v, d, 0, dt, 2 / math.sqrt(d))
    target = torch.randint(0, v, (t,), device="cuda", generator=g)
    lse = ref.linear_ce(h, w, target)[1].float()
    dloss = 512 * (0.5 + torch.rand(t, device="cuda", generator=g))  # a loss scale
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    size = tg.tg_linear_ce_grad_workspace_size(t, v, d, h, d, w, d, dh, d, dw, d, code)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    wh, _, bh, _ = ref.linear_ce_grad(h, w, target, lse, dloss)
    dloss[7] = bad
    tg.linear_ce_grad(t, v, d, h, d, w, d, target, lse, dloss, dh, d, dw, d, code, ws, size)
    torch.cuda.synchronize()
    others = torch.arange(t, device="cuda") != 7
    assert not torch.isfinite(dh[7]).any()
    ref.assert_within(dh[others], wh[others], bh[others], "dh")
