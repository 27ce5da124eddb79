"""The gradients of linear cross entropy into rows that start anywhere hold the
bits that aligned rows get, and nothing beside them is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

GUARD = 77.0


def rows_at(n, d, offset, extra, dt):
    ld = d + extra
    flat = torch.full((offset + (n - 1) * ld + d,), GUARD, dtype=dt, device="cuda")
    return flat, flat.as_strided((n, d), (ld, 1), offset), ld


def untouched(flat, view):
    inside = torch.zeros_like(flat, dtype=torch.bool)
    inside.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(True)
    return bool((flat[~inside] == GUARD).all())


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d", [(1, 3, 5), (9, 70, 8), (40, 300, 64), (70, 1000, 71), (200, 700, 201),
                                   (300, 2100, 130), (130, 20500, 264), (600, 1500, 513)])
def test_gradients_into_rows_that_start_anywhere(tg, t, v, d, dt):
    g = torch.Generator(device="cuda").manual_seed(t + v + d)
    code = tg.TG_BF16 if dt == torch.bfloat16 else tg.TG_F16
    pad = -d % 8  # aligned inputs: only the outputs move
    h = torch.randn(t, d + pad, device="cuda", generator=g).to(dt)[:, :d]
    w = (torch.randn(v, d + pad, device="cuda", generator=g) / d**0.5).to(dt)[:, :d]
    target = torch.randint(-1, v, (t,), device="cuda", generator=g)
    lse = torch.logsumexp(h.float() @ w.float().T, 1)
    dloss = torch.rand(t, device="cuda", generator=g) / t

    def grads(at_h, at_w):
        full_h, dh, ldh = rows_at(t, d, *at_h, dt)
        full_w, dw, ldw = rows_at(v, d, *at_w, dt)
        size = tg.tg_linear_ce_grad_workspace_size(t, v, d, h, h.stride(0), w, w.stride(0), dh, ldh, dw, ldw, code)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        tg.linear_ce_grad(t, v, d, h, h.stride(0), w, w.stride(0), target, lse, dloss, dh, ldh, dw, ldw, code,
                          ws, size)
        torch.cuda.synchronize()
        assert untouched(full_h, dh) and untouched(full_w, dw)
        return dh.clone(), dw.clone()

    want = grads((0, pad), (0, pad))
    assert torch.isfinite(want[0]).all() and want[1].abs().max() > 0
    for at_h, at_w in (((1, 0), (1, 0)), ((0, 1), (3, 1)), ((5, 2), (0, 3)), ((2, 8), (8, 5)), ((7, 3), (6, 2)),
                       ((8, 0), (4, 4))):
        got = grads(at_h, at_w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (at_h, at_w)
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)


# inputs: whole 16-byte units that start inside a 32-byte sector, and any address;
# vocabularies large enough for copies of H alone, and for W's through the ring
@pytest.mark.parametrize("t,v,d", [(100, 41000, 72), (300, 41000, 72), (5, 70001, 129), (70, 4100, 2100),
                                   (300, 9001, 1025), (20, 70001, 500), (3, 3000, 4097)])
def test_inputs_that_start_anywhere(tg, t, v, d):
    dt = torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(t + v + d)
    values_h = torch.randn(t, d, device="cuda", generator=g).to(dt)
    values_w = (torch.randn(v, d, device="cuda", generator=g) / d**0.5).to(dt)
    target = torch.randint(-1, v, (t,), device="cuda", generator=g)
    dloss = torch.rand(t, device="cuda", generator=g) / t

    def run(at_h, at_w):
        full_h, h, ldh = rows_at(t, d, *at_h, dt)
        full_w, w, ldw = rows_at(v, d, *at_w, dt)
        full_h.fill_(float("nan")), full_w.fill_(float("nan"))  # between the rows
        h.copy_(values_h), w.copy_(values_w)
        loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        size = tg.tg_linear_ce_workspace_size(t, v, d, h, ldh, w, ldw, tg.TG_BF16)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        tg.linear_ce(t, v, d, h, ldh, w, ldw, target, loss, lse, tg.TG_BF16, ws, size)
        dh, dw = torch.empty(t, d, dtype=dt, device="cuda"), torch.empty(v, d, dtype=dt, device="cuda")
        size = tg.tg_linear_ce_grad_workspace_size(t, v, d, h, ldh, w, ldw, dh, d, dw, d, tg.TG_BF16)
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        tg.linear_ce_grad(t, v, d, h, ldh, w, ldw, target, lse, dloss, dh, d, dw, d, tg.TG_BF16, ws, size)
        torch.cuda.synchronize()
        return loss, lse, dh, dw

    pad = -d % 64
    want = run((0, pad), (0, pad))
    assert all(torch.isfinite(x).all() for x in want)
    for at_h, at_w in (((0, -d % 16 + 8), (0, pad)), ((8, pad), (8, pad)), ((1, 0), (0, pad)), ((0, pad), (3, 0)),
                       ((5, 2), (7, 1))):
        for a, b in zip(run(at_h, at_w), want):
            assert torch.equal(a, b), (at_h, at_w)
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)
