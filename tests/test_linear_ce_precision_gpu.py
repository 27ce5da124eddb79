"""How exact the logits of linear cross entropy are: data whose sums no rounding
touches, and products of one sign, on which an accumulator that truncates is
furthest off.  No bound here is fitted to a distribution."""
import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu

DEPTH = 1024  # products that the tensor core sums before a part is added in fp32
# single tiles and (from 76 tiles of 256 x 256 on) tiles of CTA pairs; one part
# to sixteen, and a last one that is not whole
SHAPES = [(1, 300, 64), (1, 300, 4096), (130, 600, 1024), (3, 1000, 16384), (200, 700, 4136), (300, 10001, 4096),
          (520, 9800, 2112)]


def forward(tg, h, w, target):
    t, v, d = h.shape[0], w.shape[0], h.shape[1]
    code = tg.TG_BF16 if h.dtype == torch.bfloat16 else tg.TG_F16
    size = tg.tg_linear_ce_workspace_size(t, v, d, h, d, w, d, code)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(2, t, device="cuda").unbind(0)
    tg.linear_ce(t, v, d, h, d, w, d, target, loss, lse, code, ws, size)
    torch.cuda.synchronize()
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)
    return loss, lse


def sums_bound(v, lse):
    """Of everything behind exact logits: 2^x (2^-22 relative, and the argument's
    rounding), the sums' additions, and the result's roundings in log2 units."""
    return 2.0**-21 + (96 + v / 128 + 1) * ref.EPS32 + 8 * ref.EPS32 * (1 + lse.abs())


def check(tg, h, w, target, logits_off):
    want_loss, want = ref.linear_ce(h, w, target)
    loss, lse = forward(tg, h, w, target)
    bound = sums_bound(w.shape[0], want) + logits_off
    ref.assert_within(lse, want, bound, "lse")
    # the target's logit may be larger than lse is
    hit = (want - want_loss).abs()
    ref.assert_within(loss, want_loss, 2 * bound + 8 * ref.EPS32 * hit, "loss")


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d", SHAPES)
def test_one_product_per_logit(tg, t, v, d, dt):
    """Rows of H with one entry: a logit is one product, whatever the order."""
    g = torch.Generator(device="cuda").manual_seed(t + d)
    h = torch.zeros(t, d, device="cuda", dtype=dt)
    at = torch.randint(0, d, (t, 1), device="cuda", generator=g)
    h.scatter_(1, at, (2.0 ** torch.randint(-1, 2, (t, 1), device="cuda", generator=g).float()).to(dt))
    w = (torch.randint(-120, 121, (v, d), device="cuda", generator=g) / 4).to(dt)
    check(tg, h, w, torch.randint(0, v, (t,), device="cuda", generator=g), 0.0)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d", SHAPES)
def test_small_integers(tg, t, v, d, dt):
    """Sixteenths below 2^15 in sum: every partial sum is an fp32 number."""
    g = torch.Generator(device="cuda").manual_seed(t + d + 1)
    h = torch.randint(-1, 3, (t, d), device="cuda", generator=g).to(dt)
    w = (torch.randint(-16, 17, (v, d), device="cuda", generator=g) / 16).to(dt)
    check(tg, h, w, torch.randint(0, v, (t,), device="cuda", generator=g), 0.0)


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d", SHAPES)
def test_products_of_one_sign(tg, t, v, d, dt):
    """Logits of about 32.  Every 16 products one addition, off by at most 2^-23
    of the part's sum so far; then the parts' additions, rounded to nearest."""
    g = torch.Generator(device="cuda").manual_seed(t + d + 2)
    h = (0.5 + torch.rand(t, d, device="cuda", generator=g)).to(dt)
    w = ((0.5 + torch.rand(v, d, device="cuda", generator=g)) * (32 / d)).to(dt)
    largest = (h.double() @ w.double().T).amax(1)
    parts = -(-d // DEPTH)
    off = (min(d, DEPTH) / 16 * 2.0**-23 + (parts - 1) * ref.EPS32) * largest
    check(tg, h, w, torch.randint(0, v, (t,), device="cuda", generator=g), off)
