"""Vocabulary entries that W masks out with infinities: rows of the gathered H
that hold no token must not meet them."""
import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu

BOTH = [torch.float16, torch.bfloat16]


def call(tg, h, w, target, lse, dloss, want_h):
    t, v, d = h.shape[0], w.shape[0], h.shape[1]
    code = tg.TG_BF16 if h.dtype == torch.bfloat16 else tg.TG_F16
    if lse is None:
        loss, lse = torch.empty(2, t, device="cuda").unbind(0)
        size = tg.tg_linear_ce_workspace_size(t, v, d, h, d, w, d, code)
        tg.linear_ce(t, v, d, h, d, w, d, target, loss, lse, code, torch.empty(size, dtype=torch.uint8, device="cuda"),
                     size)
    dh, dw = torch.full_like(h, 7.0) if want_h else None, torch.full_like(w, 7.0)
    size = tg.tg_linear_ce_grad_workspace_size(t, v, d, h, d, w, d, dh, d, dw, d, code)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    tg.linear_ce_grad(t, v, d, h, d, w, d, target, lse, dloss, dh, d, dw, d, code, ws, size)
    torch.cuda.synchronize()
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)
    return lse, dh, dw


@pytest.mark.parametrize("dt", BOTH, ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d", [(5, 600, 80), (300, 10001, 72), (70, 300, 1200)])
def test_no_token_counts_and_w_is_not_finite(tg, t, v, d, dt):
    g = torch.Generator(device="cuda").manual_seed(t)
    h = torch.randn(t, d, device="cuda", generator=g).to(dt)
    w = torch.randn(v, d, device="cuda", generator=g).to(dt)
    w[3, 0], w[v // 2], w[v - 1, d - 1] = float("inf"), float("nan"), -float("inf")
    target = torch.full((t,), -1, device="cuda")
    _, dh, dw = call(tg, h, w, target, torch.zeros(t, device="cuda"), torch.ones(t, device="cuda"), True)
    assert (dh == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("dt", BOTH, ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d", [(40, 500, 64), (300, 10001, 72), (70, 300, 1200)])
def test_entries_masked_by_minus_infinity(tg, t, v, d, dt):
    """H's first column is positive: a masked entry's logit is -inf, its
    probability and its row of dW are 0."""
    g = torch.Generator(device="cuda").manual_seed(t + 1)
    h = torch.randn(t, d, device="cuda", generator=g).to(dt)
    h[:, 0] = 1.0
    w = (torch.randn(v, d, device="cuda", generator=g) / d**0.5).to(dt)
    masked = torch.arange(v, device="cuda") % 7 == 3
    w[masked, 0] = -float("inf")
    target = (torch.randint(0, v // 7, (t,), device="cuda", generator=g)) * 7
    target[::3] = -1
    dloss = torch.full((t,), 8.0, device="cuda")
    lse, _, dw = call(tg, h, w, target, None, dloss, False)
    kept = w[~masked]
    place = torch.cumsum(~masked, 0) - 1  # of a kept entry among them
    inner = torch.where(target >= 0, place[target.clamp(min=0)], -1)
    _, want = ref.linear_ce(h, kept, inner)
    ref.assert_within(lse, want, ref.lse_bound(h, kept, want), "lse")
    _, ww, _, bw = ref.linear_ce_grad(h, kept, inner, lse, dloss)
    assert (dw[masked] == 0).all()
    ref.assert_within(dw[~masked], ww, bw, "dw")
