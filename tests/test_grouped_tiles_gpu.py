"""Every tile of the grouped products (64 and 128 columns on one CTA, 256 x 256 on a pair) with
several tiles of columns, more tiles of rows than share their columns in turn, more K-blocks than
the ring holds, an odd number of them and a part one; rows by a list and one after another, both
orders of the matrices, with and without an epilogue.  Ragged ends beside rows that are no numbers,
and operands that lie far apart."""
import pytest
import torch

from rows_reference import EPS32, assert_within, code, offsets, padded, product, rounded, source, stacked

pytestmark = pytest.mark.gpu

STEP = (1 << 31) + 64  # elements

TILES = {  # rows per group, N, and the tile that the library's rule takes for them on 152 SMs
    "pair": ([2500, 0, 129, 1, 700], 1101),
    "128": ([0] * 17 + [2400, 1, 0, 130] + [0] * 10 + [300] + [3] * 8, 300),
    "64": ([2600, 0, 77], 267),
}
K = 664  # 11 K-blocks, the last of 24


def columns(r, n, g):
    """The rule for a product that is not of few rows."""
    tiles = lambda rows, cols: (min(r, g) + r // rows) * -(-n // cols)  # noqa: E731
    if r >= 128 * g and tiles(256, 256) >= 152 // 2:
        return "pair"
    return "128" if tiles(128, 128) >= 152 else "64"


def sources(gen, r, x_rows, per_row):
    row = torch.randint(0, x_rows * per_row, (r,), generator=gen, device="cuda", dtype=torch.int32)
    row[2], row[5] = -1, x_rows * per_row  # outside: rows of zeros
    return row


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("tile", TILES)
@pytest.mark.parametrize("perm", [0, 1])
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("epilogue", [False, True])
def test_product(tg, tile, perm, listed, epilogue, dtype):
    counts, n = TILES[tile]
    gen = torch.Generator(device="cuda").manual_seed(n)
    g, used = len(counts), sum(counts)
    r = used + 3  # rows of no group behind the last
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert columns(r, n, g) == tile
    per_row, x_rows = (3, r // 3) if listed else (1, r)
    x = padded(gen, x_rows, K, 8, dtype)
    row = sources(gen, r, x_rows, per_row) if listed else None
    b = stacked(gen, g, *((K, n) if perm == 0 else (n, K)), 8, 16, dtype)
    epi = None
    if epilogue:
        bias = (torch.randn(g, n + 1, generator=gen, device="cuda") * 3).to(dtype)[:, :n]
        relu_of = padded(gen, r, n, 8, dtype)
        relu_of[::5], relu_of[1::7], relu_of[2::11, :40] = 0.0, -0.0, float("nan")
        epi = tg.make_group_epilogue(bias, bias.stride(0), True, relu_of, relu_of.stride(0))
    y = torch.full((r, (n + 7) // 8 * 8), 5.0, device="cuda", dtype=dtype)
    tg.grouped_gemm(r, n, K, g, x, x_rows, x.stride(0), row, per_row, b, b.stride(1), b.stride(0), perm, offsets(counts), y,
                    y.stride(0), code(tg, dtype), epi)
    assert tg.tg_debug_status()[0] == tg.TG_OK
    lo = 0
    for q, c in enumerate(counts):
        m = b[q].double() if perm == 0 else b[q].double().T
        want, slack, _ = product(source(x, row, per_row, lo, lo + c), m, dtype)
        if epilogue:
            want = want + bias[q].double()
            slack = slack + EPS32 * want.abs()
            off = (want < 0) | ~(relu_of[lo:lo + c] > 0)
            assert (y[lo:lo + c, :n][~(relu_of[lo:lo + c] > 0)] == 0).all()
            want = torch.where(off, 0.0, want)  # (a sum near 0 may be on its other side, by its slack)
        assert_within(y[lo:lo + c, :n], want, rounded(want, slack, dtype), f"group {q}")
        lo += c
    assert (y[used:] == 5.0).all() and (y[:, n:] == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,m,n", [([700, 0, 65], 2401, 700), ([777], 2300, 203)])  # a pair's tiles, 128 columns
@pytest.mark.parametrize("perm", [0, 1])
@pytest.mark.parametrize("listed", [False, True])
def test_gradient(tg, counts, m, n, perm, listed, dtype):
    """m x n: a matrix as it is stored."""
    gen = torch.Generator(device="cuda").manual_seed(m)
    g, used = len(counts), sum(counts)
    r = used + 3
    inner, outer = (m, n) if perm == 0 else (n, m)  # the product's K and N
    per_row, x_rows = (3, r // 3) if listed else (1, r)
    x, dy = padded(gen, x_rows, inner, 8, dtype), padded(gen, r, outer, 0, dtype, 0.25)
    row = sources(gen, r, x_rows, per_row) if listed else None
    db = stacked(gen, g, m, n, 8, 16, dtype)
    outside = torch.isnan(db.as_strided((db.stride(0) * g,), (1,)))
    tg.grouped_gemm_grad(r, outer, inner, g, dy, dy.stride(0), x, x_rows, x.stride(0), row, per_row, offsets(counts), db, db.stride(1),
                         db.stride(0), perm, code(tg, dtype))
    assert tg.tg_debug_status()[0] == tg.TG_OK
    lo = 0
    for q, c in enumerate(counts):
        want, slack, _ = product(source(x, row, per_row, lo, lo + c).T, dy[lo:lo + c].double(), dtype)
        assert_within(db[q] if perm == 0 else db[q].T, want, rounded(want, slack, dtype), f"group {q}")
        lo += c
    assert torch.isnan(db.as_strided((db.stride(0) * g,), (1,))[outside]).all()


@pytest.mark.parametrize("perm", [0, 1])
@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("wide", [False, True])
def test_ragged_ends_beside_rows_that_are_no_numbers(tg, perm, listed, wide):
    """Groups of 1 to 128 rows, each between two of one row of infinities and NaN."""
    dtype, n, k = torch.bfloat16, 40, 72
    rests = range(1, 129) if wide else range(1, 129, 7)  # (many groups: pairs; few: 128 columns)
    counts = [c for rest in rests for c in (rest, 1)]
    gen = torch.Generator(device="cuda").manual_seed(5)
    g, r = len(counts), sum(counts)
    offset = offsets(counts)
    spoilt = offset[1:-1:2].long()
    x, dy = padded(gen, r, k, 0, dtype), padded(gen, r, n, 0, dtype, 0.25)
    row = torch.randperm(r, generator=gen, device="cuda").int() if listed else None
    x[row[spoilt].long() if listed else spoilt], dy[spoilt] = float("inf"), float("nan")
    db = stacked(gen, g, *((k, n) if perm == 0 else (n, k)), 0, 0, dtype)
    tg.grouped_gemm_grad(r, n, k, g, dy, dy.stride(0), x, r, x.stride(0), row, 1, offset, db, db.stride(1), db.stride(0), perm,
                         tg.TG_BF16)
    assert tg.tg_debug_status()[0] == tg.TG_OK
    lo = 0
    for q, c in enumerate(counts):
        got = db[q] if perm == 0 else db[q].T
        if q % 2:
            assert got.isnan().all()
        else:
            want, slack, _ = product(source(x, row, 1, lo, lo + c).T, dy[lo:lo + c].double(), dtype)
            assert_within(got, want, rounded(want, slack, dtype), f"{c} rows")
        lo += c


def apart(shape, stride, dtype):
    """A stack or matrix whose first dimension's parts lie `stride` elements apart."""
    inner = 1
    for s in shape[1:]:
        inner *= s
    flat = torch.zeros((shape[0] - 1) * stride + inner, device="cuda", dtype=dtype)
    steps = [inner // shape[1] if len(shape) == 3 else 1] + ([1] if len(shape) == 3 else [])
    return flat.as_strided(shape, [stride] + steps)


@pytest.mark.parametrize("rows", [3, 41])  # the kernel of few rows, and tiles
@pytest.mark.parametrize("perm", [0, 1])
def test_matrices_biases_and_masks_far_apart(tg, perm, rows):
    """Matrices, biases and (three rows of) a mask more than 2^31 elements apart, as side by side."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    n, k, dtype = 136, 200, torch.float16
    make = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    x, b, bias, mask = make(rows, k), make(2, *((k, n) if perm == 0 else (n, k))), make(2, n), make(rows, n)
    offset, out = offsets([1, rows - 1]), []
    for far in (False, True):
        def place(v, far=far):
            w = apart(v.shape, STEP if far else v.stride(0), dtype)
            w.copy_(v)
            return w
        m, beside, z = place(b), place(bias), place(mask) if rows == 3 else mask
        y = torch.empty(rows, n, device="cuda", dtype=dtype)
        epi = tg.make_group_epilogue(beside, beside.stride(0), False, z, z.stride(0))
        tg.grouped_gemm(rows, n, k, 2, x, rows, k, None, 1, m, m.stride(1), m.stride(0), perm, offset, y, n, tg.TG_F16, epi)
        assert tg.tg_debug_status()[0] == tg.TG_OK
        out.append(y)
        del m, beside, z, epi
        torch.cuda.empty_cache()
    assert torch.equal(*out) and out[0].abs().max() > 0
