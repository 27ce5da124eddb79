"""Layer norm and its gradient over rows that start anywhere: every operand
with its own offset and row stride, buffers that end with their last element,
against the 64-bit forms.  The bounds are those of the library's roundings."""
import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu

GUARD = 77.0


def rows_at(n, d, offset, extra, dt, gen=None):
    """n x d rows of stride d + extra, `offset` elements into a buffer that
    ends with the last of them; the places between them hold NaN (inputs) or a
    guard value (outputs)."""
    ld = d + extra
    fill = float("nan") if gen is not None else GUARD
    flat = torch.full((offset + (n - 1) * ld + d,), fill, dtype=dt, device="cuda")
    view = flat.as_strided((n, d), (ld, 1), offset)
    if gen is not None:
        view.copy_(torch.randn(n, d, device="cuda", generator=gen))
    return flat, view, ld


def untouched(flat, view):
    inside = torch.zeros_like(flat, dtype=torch.bool)
    inside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool((flat[~inside] == GUARD).all())


CASES = [  # rows, columns, (offset, extra) of x, dy and the output
    (1, 1, (3, 0), (5, 0), (1, 0)), (30, 1, (1, 0), (0, 0), (3, 0)), (5, 3, (0, 0), (1, 0), (2, 0)),
    (41, 8, (1, 0), (7, 1), (0, 3)), (9, 15, (7, 2), (0, 0), (1, 0)), (700, 63, (0, 0), (0, 0), (0, 0)),
    (2500, 250, (1, 1), (2, 3), (3, 0)), (100, 256, (4, 0), (4, 4), (4, 8)), (640, 511, (6, 0), (1, 5), (2, 1)),
    (33, 1017, (0, 0), (0, 7), (0, 0)), (400, 1018, (5, 0), (3, 0), (7, 0)), (2000, 1000, (0, 3), (0, 0), (0, 0)),
    (70, 2047, (1, 0), (1, 0), (1, 0)), (1300, 2050, (0, 0), (2, 0), (6, 2)), (500, 4089, (3, 0), (0, 0), (0, 0)),
    (350, 4090, (7, 0), (6, 1), (1, 0)), (330, 8185, (0, 0), (0, 0), (0, 0)), (310, 8186, (2, 4), (5, 0), (3, 1)),
    (170, 9001, (0, 0), (1, 0), (4, 0)), (340, 16377, (7, 0), (0, 2), (1, 1)), (5, 16378, (1, 0), (0, 0), (0, 0)),
]


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("n,d,at_x,at_dy,at_out", CASES)
def test_rows_that_start_anywhere(tg, n, d, at_x, at_dy, at_out, dt):
    g = torch.Generator(device="cuda").manual_seed(n * 31 + d)
    code = tg.TG_BF16 if dt == torch.bfloat16 else tg.TG_F16
    _, x, ldx = rows_at(n, d, *at_x, dt, g)
    _, dy, lddy = rows_at(n, d, *at_dy, dt, g)
    _, w, _ = rows_at(1, d, 1, 0, dt, g)
    _, b, _ = rows_at(1, d, 2, 0, dt, g)
    w, b = w[0], b[0]
    u, tiny, eps = ref.HALF_ULP[dt] * 1.01, ref.TINY[dt], ref.EPS32
    adds = d / 32 + 48  # of one row's sum over its threads

    full, y, ldy = rows_at(n, d, *at_out, dt)
    mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    tg.layernorm(n, d, x, ldx, w, b, 1e-5, y, ldy, mean, rstd, code)
    torch.cuda.synchronize()
    assert untouched(full, y)
    wy, wm, wr = ref.layernorm(x, w, b, 1e-5)
    bm = adds * eps * 2 * x.double().abs().mean(1)
    ref.assert_within(mean, wm, bm, "mean")
    br = wr * (adds * eps + 4 * eps + bm**2 * wr**2)
    ref.assert_within(rstd, wr, br, "rstd")
    xh = (x.double() - wm[:, None]) * wr[:, None]
    by = (bm * wr)[:, None] + xh.abs() * ((br / wr)[:, None] + 8 * eps)
    by = by * w.double().abs() + u * wy.abs() + 4 * eps * (xh * w.double()).abs() + tiny
    ref.assert_within(y, wy, by, "y")

    mean, rstd = wm.float(), wr.float()
    full, dx, lddx = rows_at(n, d, *at_out, dt)
    full_w, dw, _ = rows_at(1, d, 1, 0, dt)
    full_b, db, _ = rows_at(1, d, 3, 0, dt)
    size = tg.tg_layernorm_grad_workspace_size(n, d, code)
    ws = torch.full((max(1, size),), 0xFF, dtype=torch.uint8, device="cuda")
    tg.layernorm_grad(n, d, dy, lddy, x, ldx, w, mean, rstd, dx, lddx, dw, db, code, ws, size)
    torch.cuda.synchronize()
    assert untouched(full, dx) and untouched(full_w, dw) and untouched(full_b, db)
    wx, ww, wb = ref.layernorm_grad(dy, x, w, mean, rstd)
    r = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    gg = dy.double() * w.double()
    c1 = adds * eps * gg.abs().mean(1, keepdim=True)
    c2 = (adds + 8) * eps * (gg * xh).abs().mean(1, keepdim=True)
    m2 = (gg * xh).mean(1, keepdim=True).abs()
    xh, gg = xh.abs(), gg.abs()
    bx = r * (c1 + xh * c2 + 8 * eps * (gg + gg.mean(1, keepdim=True) + xh * m2))
    ref.assert_within(dx, wx, bx + u * wx.abs() + tiny, "dx")
    adds = n + 64  # of a column's sum
    ref.assert_within(dw[0], ww, (adds + 4) * eps * (dy.double().abs() * xh).sum(0) + u * ww.abs() + tiny, "dweight")
    ref.assert_within(db[0], wb, adds * eps * dy.double().abs().sum(0) + u * wb.abs() + tiny, "dbias")
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)


@pytest.mark.parametrize("d", [37, 600, 5001, 9001])
def test_a_row_of_infinities_stays_alone(tg, d):
    """Neighbours of a row share 16-byte units with it; nothing of it may reach them."""
    n, dt = 12, torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(d)
    flat, x, ld = rows_at(n, d, 1, 0, dt, g)
    _, dy, _ = rows_at(n, d, 1, 0, dt, g)
    w, b = torch.ones(d, dtype=dt, device="cuda"), torch.zeros(d, dtype=dt, device="cuda")
    out = []
    for bad in (False, True):
        if bad:
            x[5] = float("inf")
            dy[5] = float("nan")
        y, mean, rstd = torch.empty(n, d, dtype=dt, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        tg.layernorm(n, d, x, ld, w, b, 1e-5, y, d, mean, rstd, tg.TG_BF16)
        dx, dw = torch.empty_like(y), torch.empty_like(w)
        size = tg.tg_layernorm_grad_workspace_size(n, d, tg.TG_BF16)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        tg.layernorm_grad(n, d, dy, ld, x, ld, w, mean, rstd, dx, d, dw, None, tg.TG_BF16, ws, size)
        torch.cuda.synchronize()
        out.append((y, mean, rstd, dx))
    keep = torch.arange(n, device="cuda") != 5
    for a, c in zip(*out):
        assert torch.equal(a[keep], c[keep]) and not torch.isfinite(c[5]).all()
