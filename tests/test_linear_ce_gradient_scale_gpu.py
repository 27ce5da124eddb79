"""Gradients of linear cross entropy where tokens weigh very differently: each
row of dH is as exact as fp16 or bf16 allow for its own upstream gradient."""
import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu

WEIGHTS = [1.0, 2.0**-8 * 1.1, 2.0**-12 * 1.3, -(2.0**-16) * 1.7, 2.0**-20 * 1.3, 0.0, -0.75]


def gradients(tg, h, w, target, lse, dloss, want=(True, True)):
    t, v, d = h.shape[0], w.shape[0], h.shape[1]
    code = tg.TG_BF16 if h.dtype == torch.bfloat16 else tg.TG_F16
    dh, dw = torch.empty_like(h) if want[0] else None, torch.empty_like(w) if want[1] else None
    size = tg.tg_linear_ce_grad_workspace_size(t, v, d, h, d, w, d, dh, d, dw, d, code)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    tg.linear_ce_grad(t, v, d, h, d, w, d, target, lse, dloss, dh, d, dw, d, code, ws, size)
    torch.cuda.synchronize()
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)
    return dh, dw


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
# by one block's compaction and by every block's; a single tile's and a pair's products
@pytest.mark.parametrize("t,v,d", [(40, 40000, 72), (300, 20000, 264), (2500, 5000, 64)])
def test_tokens_of_very_different_weight(tg, t, v, d, dt):
    """W's entries are of one sign and the probabilities nearly equal, so that
    what is lost of them adds up."""
    g = torch.Generator(device="cuda").manual_seed(t)
    h = torch.randn(t, d, device="cuda", generator=g).to(dt)
    w = (0.5 + torch.rand(v, d, device="cuda", generator=g) / 64).to(dt)
    target = torch.randint(0, v, (t,), device="cuda", generator=g)
    target[::9] = -1
    target[0], target[-1] = 5, v - 1
    # times a loss scale: the light rows of dH are normal fp16 numbers
    dloss = torch.tensor(WEIGHTS, device="cuda").repeat(t // len(WEIGHTS) + 1)[:t] * 512.0
    dloss[0], dloss[-1] = 512.0, 512.0 * 2.0**-20
    logits = h.double() @ w.double().T
    lse = torch.logsumexp(logits, 1).float()
    dh, dw = gradients(tg, h, w, target, lse, dloss)

    u, ok = ref.HALF_ULP[dt] * 1.01, target >= 0
    up = torch.where(ok, dloss, 0.0).double()
    p = torch.exp(logits - lse.double()[:, None])
    slack = ref.logit_bound(h, w)[:, None] + 16 * ref.EPS32 * (1 + lse.abs().max().double()) + 2.0**-20
    off = p * slack
    p[torch.arange(t, device="cuda"), target.clamp(min=0)] -= 1
    # G to 16 bits; in fp16 full precision down to probabilities of 2^-18
    off = (off + u * p.abs() + (2.0**-29 if dt == torch.float16 else 0.0)) * up.abs()[:, None]
    gg = p * up[:, None]
    want_h, want_w = gg @ w.double(), gg.T @ h.double()
    acc = 2 * ref.EPS32
    bound_h = off @ w.double().abs() + (v / 16 + 8) * acc * (gg.abs() @ w.double().abs()) + u * want_h.abs() + ref.TINY[dt]
    # fp16: a light token's row of H is an fp16 number times a power of two, 2^-10 at least
    rows = h.double().abs() * (1 + u) + (2.0**-15 if dt == torch.float16 else 0.0)
    bound_w = off.T @ rows + (gg.abs().T @ torch.full_like(rows, 2.0**-15) if dt == torch.float16 else 0.0)
    bound_w = bound_w + (t / 16 + 8) * acc * (gg.abs().T @ rows) + u * want_w.abs() + ref.TINY[dt]
    ref.assert_within(dh, want_h, bound_h, "dh")
    ref.assert_within(dw, want_w, bound_w, "dw")
    # the bound is small beside the light tokens' own gradients
    light = ok & (dloss.abs() < 512.0 * 2.0**-15) & (dloss != 0)
    if dt == torch.float16 and t < 1000:
        size = off[light] @ w.double().abs()
        assert light.any() and float((size / (up[light].abs()[:, None] * 0.5)).max()) < 0.01
    only_h, _ = gradients(tg, h, w, target, lse, dloss, (True, False))
    _, only_w = gradients(tg, h, w, target, lse, dloss, (False, True))
    assert torch.equal(only_h, dh) and torch.equal(only_w, dw)


def test_one_weight_for_all_is_as_before(tg):
    """Gradients scale with a power of two bit for bit."""
    t, v, d, dt = 200, 3000, 136, torch.float16
    g = torch.Generator(device="cuda").manual_seed(8)
    h = torch.randn(t, d, device="cuda", generator=g).to(dt)
    w = (torch.randn(v, d, device="cuda", generator=g) / d**0.5).to(dt)
    target = torch.randint(0, v, (t,), device="cuda", generator=g)
    lse = torch.logsumexp(h.double() @ w.double().T, 1).float()
    one = gradients(tg, h, w, target, lse, torch.full((t,), 512.0, device="cuda"))
    two = gradients(tg, h, w, target, lse, torch.full((t,), 1024.0, device="cuda"))
    for a, b in zip(one, two):
        normal = a.abs() >= 2.0**-14
        assert normal.any() and torch.equal((a * 2)[normal], b[normal])
