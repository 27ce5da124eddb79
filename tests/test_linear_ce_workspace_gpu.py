"""The workspace of linear cross entropy's gradient grows with the tokens, and
nothing is written past it."""
import math

import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t", [1, 8, 63, 64, 65, 128, 129, 256])
def test_few_tokens(tg, t, dt):
    v, d = 20000, 200
    g = torch.Generator(device="cuda").manual_seed(t)
    code = tg.TG_BF16 if dt == torch.bfloat16 else tg.TG_F16
    h, w = ref.rows(g, t, d, 0, dt), ref.rows(g, v, d, 0, dt, 2 / math.sqrt(d))
    target = torch.randint(0, v, (t,), device="cuda", generator=g)
    if t > 8:
        target[::5] = -1
    lse = ref.linear_ce(h, w, target)[1].float()
    dloss = torch.rand(t, device="cuda", generator=g) + 0.1
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    size = tg.tg_linear_ce_grad_workspace_size(t, v, d, h, d, w, d, dh, d, dw, d, code)
    # G in whole K-blocks of 64 tokens up to 128, then in whole tiles; splits of dH's
    # contraction, 8 K-blocks deep at least; the gathered rows of H (twice in fp16)
    rows = 64 if t <= 64 else 128 if t <= 128 else 256
    most = rows * (v + 256) * 2 + (v / 64 / 8) * t * d * 4 + 2 * rows * 256 * 2 + 4096 + 64 * t
    assert size <= most, (size, most)
    whole = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    whole[:size] = 0xFF
    tg.linear_ce_grad(t, v, d, h, d, w, d, target, lse, dloss, dh, d, dw, d, code, whole, size)
    torch.cuda.synchronize()
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)
    assert (whole[size:] == 0xA5).all()
    wh, ww, bh, bw = ref.linear_ce_grad(h, w, target, lse, dloss)
    ref.assert_within(dh, wh, bh, "dh")
    ref.assert_within(dw, ww, bw, "dw")
