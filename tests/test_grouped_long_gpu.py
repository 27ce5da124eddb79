"""Contractions of one tile that take longer than the time limit of a single wait."""
import pytest
import torch

from rows_reference import code, offsets

pytestmark = pytest.mark.gpu

LIMIT = 3_000_000  # cycles; the products alone, 64 cycles for 128 x 128 x 16, are more than that below


def whole(gen, *shape, dtype):
    """-1, 0 and 1: their sums are exact in fp32."""
    return torch.randint(-1, 2, shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("listed", [False, True])
def test_one_group_of_many_rows(tg, listed, dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    r, n, k = (1 << 21) - 5, 72, 64
    x, dy = whole(gen, r, k, dtype=dtype), whole(gen, r, n, dtype=dtype)
    row = torch.randperm(r, generator=gen, device="cuda").int() if listed else None
    offset = offsets([0, r])
    db = torch.empty(2, n, k, device="cuda", dtype=dtype)
    assert (r // 64) * 4 * 64 > LIMIT
    tg.tg_debug_configure(LIMIT, -1)
    try:
        tg.grouped_gemm_grad(r, n, k, 2, dy, n, x, r, k, row, 1, offset, db, k, n * k, tg.TG_OP_T, code(tg, dtype))
        assert tg.tg_debug_status()[0] == tg.TG_OK
    finally:
        tg.tg_debug_configure(0, -1)
    want = dy.double().T @ (x[row.long()] if listed else x).double()
    assert (db[0] == 0).all() and torch.equal(db[1], want.to(dtype))


@pytest.mark.parametrize("listed", [False, True])
def test_a_long_inner_dimension(tg, listed):
    gen = torch.Generator(device="cuda").manual_seed(2)
    r, n, k, dtype = 9, 72, (1 << 21) - 8, torch.bfloat16
    x, b = whole(gen, r, k, dtype=dtype), whole(gen, k, n, dtype=dtype)
    row = torch.randperm(r, generator=gen, device="cuda").int() if listed else None
    y = torch.empty(r, n, device="cuda", dtype=dtype)
    tg.tg_debug_configure(LIMIT, -1)
    try:
        tg.grouped_gemm(r, n, k, 1, x, r, k, row, 1, b, n, k * n, tg.TG_OP_N, offsets([r]), y, n, tg.TG_BF16)
        assert tg.tg_debug_status()[0] == tg.TG_OK
    finally:
        tg.tg_debug_configure(0, -1)
    want = (x[row.long()] if listed else x).double() @ b.double()
    assert torch.equal(y, want.to(dtype))
