"""Rows that lie more than 2^31 elements apart: the output head's operators
give what they give on rows side by side."""
import pytest
import torch

pytestmark = pytest.mark.gpu

STEP = (1 << 31) + 64  # elements from one row to the next


def far(x, extra=0):
    """A copy of x (a few rows) whose rows are STEP + extra elements apart."""
    flat = torch.empty((x.shape[0] - 1) * (STEP + extra) + x.shape[1], dtype=x.dtype, device="cuda")
    view = flat.as_strided(x.shape, (STEP + extra, 1))
    view.copy_(x)
    return view


@pytest.mark.parametrize("extra", [0, 1], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("d", [512, 5000, 20000])
def test_layernorm(tg, d, extra):
    g = torch.Generator(device="cuda").manual_seed(d)
    draw = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()  # noqa: E731
    x, dy, w, b = draw(3, d), draw(3, d), draw(d), draw(d)
    size = tg.tg_layernorm_grad_workspace_size(3, d, tg.TG_BF16)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    ends = []
    for place in (lambda t: t.clone(), lambda t: far(t, extra)):
        a, e, y, dx = place(x), place(dy), place(torch.zeros_like(x)), place(torch.zeros_like(x))
        mean, rstd = torch.empty(2, 3, device="cuda").unbind(0)
        dw, db = torch.empty_like(w), torch.empty_like(b)
        tg.layernorm(3, d, a, a.stride(0), w, b, 1e-5, y, y.stride(0), mean, rstd, tg.TG_BF16)
        tg.layernorm_grad(3, d, e, e.stride(0), a, a.stride(0), w, mean, rstd, dx, dx.stride(0), dw, db, tg.TG_BF16, ws, size)
        torch.cuda.synchronize()
        ends.append([t.double().contiguous() for t in (y, mean, rstd, dx, dw, db)])
        del a, e, y, dx
    for p, q in zip(*ends):
        # another path may add in another order: a rounding to 16 bits apart at most
        assert ((p - q).abs() <= 2.0**-7 * p.abs() + 2.0**-12 * p.abs().max()).all()
        assert p.abs().max() > 0
    torch.cuda.empty_cache()


@pytest.mark.parametrize("extra", [0, 1], ids=["aligned", "unaligned"])
def test_linear_ce(tg, extra):
    t, v, d = 3, 5, 200
    g = torch.Generator(device="cuda").manual_seed(3)
    h, w = torch.randn(t, d, device="cuda", generator=g).half(), torch.randn(v, d, device="cuda", generator=g).half()
    target, dloss = torch.tensor([4, -1, 0], device="cuda"), torch.ones(t, device="cuda")
    ends = []
    for place in (lambda x: x.clone(), lambda x: far(x, extra)):
        a, b, dh, dw = place(h), place(w), place(torch.zeros_like(h)), place(torch.zeros_like(w))
        loss, lse = torch.empty(2, t, device="cuda").unbind(0)
        size = tg.tg_linear_ce_workspace_size(t, v, d, a, a.stride(0), b, b.stride(0), tg.TG_F16)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        tg.linear_ce(t, v, d, a, a.stride(0), b, b.stride(0), target, loss, lse, tg.TG_F16, ws, size)
        size = tg.tg_linear_ce_grad_workspace_size(t, v, d, a, a.stride(0), b, b.stride(0), dh, dh.stride(0), dw,
                                                   dw.stride(0), tg.TG_F16)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        tg.linear_ce_grad(t, v, d, a, a.stride(0), b, b.stride(0), target, lse, dloss, dh, dh.stride(0), dw,
                          dw.stride(0), tg.TG_F16, ws, size)
        torch.cuda.synchronize()
        st, detail = tg.tg_debug_status()
        assert st == tg.TG_OK, hex(detail)
        ends.append([x.contiguous() for x in (loss, lse, dh, dw)])
        del a, b, dh, dw
        torch.cuda.empty_cache()
    for p, q in zip(*ends):
        assert torch.equal(p, q) and p.abs().max() > 0
