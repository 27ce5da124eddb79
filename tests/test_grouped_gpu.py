"""Grouped products, their gradients, combining and adapters against 64 bits."""
import pytest
import torch

from rows_reference import (EPS32, HALF_ULP, TINY, assert_within, code, offsets, padded, product, rounded, source, stacked)

pytestmark = pytest.mark.gpu

# rows per group: tiles of 64 or 128 columns for few rows, pairs of CTAs from 128 rows per group on
SMALL = [1]
FEW = [0, 1, 3, 0, 0, 5, 127, 0]
RAGGED = [128, 1, 0, 130, 4, 255, 31, 129]
LARGE = [256, 257, 511, 0, 128, 700]
MANY = [i % 4 for i in range(300)]  # more groups than a worker looks at at once


def list_of(gen, r, x_rows, per_row):
    """A source for each row; a few outside."""
    row = torch.randint(0, x_rows * per_row, (r,), generator=gen, device="cuda", dtype=torch.int32)
    if r > 6:
        row[2] = -1
        row[5] = x_rows * per_row
    return row


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,n,k", [
    (SMALL, 1, 1), (SMALL, 200, 64), (FEW, 72, 100), (FEW, 129, 513), (RAGGED, 256, 64), (RAGGED, 250, 72), (LARGE, 520, 200),
    (LARGE, 64, 65), (MANY, 100, 40), ([20000, 3], 136, 64), ([0, 0, 0], 64, 64), ([5] * 200, 1000, 24),
    ([16, 0, 9, 17], 264, 1100), ([130] * 140, 72, 136), ([i % 3 for i in range(4096)], 8, 8)])
@pytest.mark.parametrize("perm", [0, 1])
@pytest.mark.parametrize("gathered", [False, True])
def test_grouped_gemm(tg, counts, n, k, perm, gathered, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    g, used = len(counts), sum(counts)
    r = used + 9  # rows of no group behind the last
    per_row, x_rows = (3, max(1, r // 3)) if gathered else (1, r)
    x = padded(gen, x_rows, k, 8, dtype)
    row = list_of(gen, r, x_rows, per_row) if gathered else None
    b = stacked(gen, g, *((k, n) if perm == 0 else (n, k)), 8, 16, dtype)
    y = torch.full((r, (n + 7) // 8 * 8), 5.0, device="cuda", dtype=dtype)
    offset = offsets(counts)
    tg.grouped_gemm(r, n, k, g, x, x_rows, x.stride(0), row, per_row, b, b.stride(1), b.stride(0), perm, offset, y, y.stride(0),
                    code(tg, dtype))
    assert tg.tg_debug_status()[0] == tg.TG_OK
    lo = 0
    for q, c in enumerate(counts):
        m = b[q].double() if perm == 0 else b[q].double().T
        want, slack, _ = product(source(x, row, per_row, lo, lo + c), m, dtype)
        assert_within(y[lo:lo + c, :n], want, rounded(want, slack, dtype), f"group {q}")
        lo += c
    assert (y[used:] == 5.0).all() and (y[:, n:] == 5.0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,n,k", [([2, 0, 3, 1], 75, 200), (FEW, 75, 64), (LARGE, 300, 64)])
def test_epilogue(tg, counts, n, k, dtype):
    gen = torch.Generator(device="cuda").manual_seed(4)
    g, r = len(counts), sum(counts)
    x = padded(gen, r, k, 0, dtype)
    b = stacked(gen, g, n, k, 0, 0, dtype)
    bias = (torch.randn(g, n + 1, generator=gen, device="cuda") * 3).to(dtype)[:, :n]
    relu_of = padded(gen, r, n, 8, dtype)
    relu_of[::5] = 0.0
    relu_of[1::7] = -0.0
    relu_of[2::11, :3] = float("nan")
    offset = offsets(counts)
    y = torch.empty(r, (n + 7) // 8 * 8, device="cuda", dtype=dtype)
    owner = torch.repeat_interleave(torch.arange(g, device="cuda"), offset.diff().long())
    for with_bias, relu, mask in [(True, False, False), (False, True, False), (False, False, True), (True, True, True)]:
        epi = tg.make_group_epilogue(bias if with_bias else None, bias.stride(0), relu, relu_of if mask else None, relu_of.stride(0))
        tg.grouped_gemm(r, n, k, g, x, r, x.stride(0), None, 1, b, b.stride(1), b.stride(0), tg.TG_OP_T, offset, y, y.stride(0),
                        code(tg, dtype), epi)
        want, slack = torch.empty(r, n, dtype=torch.float64, device="cuda"), torch.empty(r, n, dtype=torch.float64, device="cuda")
        for q in range(g):
            at = owner == q
            want[at], slack[at], _ = product(x[at].double(), b[q].double().T, dtype)
        if with_bias:
            want = want + bias.double()[owner]
            slack = slack + EPS32 * want.abs()
        if relu:
            want = want.clamp(min=0.0)
        if mask:
            off = ~(relu_of > 0)
            want[off], slack[off] = 0.0, 0.0
            assert (y[:, :n][off] == 0).all()
        assert_within(y[:, :n], want, rounded(want, slack, dtype), "epilogue")


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,n,k", [
    (SMALL, 1, 1), (FEW, 72, 100), (RAGGED, 129, 65), (LARGE, 520, 200), (MANY, 40, 24), ([20000, 3], 136, 64), ([0, 0], 64, 64),
    ([63, 64, 65] * 12, 600, 520), ([i % 5 for i in range(600)], 40, 24), ([130] * 140, 72, 136)])
@pytest.mark.parametrize("perm", [0, 1])
@pytest.mark.parametrize("gathered", [False, True])
def test_grouped_gemm_grad(tg, counts, n, k, perm, gathered, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    g, used = len(counts), sum(counts)
    r = used + 9
    per_row, x_rows = (3, max(1, r // 3)) if gathered else (1, r)
    x = padded(gen, x_rows, k, 8, dtype)
    row = list_of(gen, r, x_rows, per_row) if gathered else None
    dy = padded(gen, r, n, 0, dtype, 0.25)
    db = stacked(gen, g, *((k, n) if perm == 0 else (n, k)), 8, 16, dtype)
    offset = offsets(counts)
    outside = torch.isnan(db.as_strided((db.stride(0) * g,), (1,)))
    tg.grouped_gemm_grad(r, n, k, g, dy, dy.stride(0), x, x_rows, x.stride(0), row, per_row, offset, db, db.stride(1), db.stride(0),
                         perm, code(tg, dtype))
    assert tg.tg_debug_status()[0] == tg.TG_OK
    lo = 0
    for q, c in enumerate(counts):
        want, slack, _ = product(source(x, row, per_row, lo, lo + c).T, dy[lo:lo + c].double(), dtype)
        got = db[q] if perm == 0 else db[q].T
        assert_within(got, want, rounded(want, slack, dtype), f"group {q}")
        lo += c
    assert torch.isnan(db.as_strided((db.stride(0) * g,), (1,))[outside]).all()


def test_infinities_stay_in_their_group(tg):
    """Rows of one group that hold infinities and NaN, matrices likewise."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    counts, n, k, dtype = [70, 1, 190, 66], 130, 96, torch.bfloat16
    r, g = sum(counts), 4
    x, dy = padded(gen, r, k, 0, dtype), padded(gen, r, n, 0, dtype)
    b = stacked(gen, g, n, k, 0, 0, dtype)
    x[70:71], dy[70:71], b[1] = float("inf"), float("nan"), float("inf")
    offset = offsets(counts)
    y = torch.empty(r, 136, device="cuda", dtype=dtype)
    db = stacked(gen, g, n, k, 0, 0, dtype)
    tg.grouped_gemm(r, n, k, g, x, r, x.stride(0), None, 1, b, b.stride(1), b.stride(0), tg.TG_OP_T, offset, y, 136, tg.TG_BF16)
    tg.grouped_gemm_grad(r, n, k, g, dy, dy.stride(0), x, r, x.stride(0), None, 1, offset, db, db.stride(1), db.stride(0), tg.TG_OP_T,
                         tg.TG_BF16)
    keep = torch.ones(r, dtype=torch.bool, device="cuda")
    keep[70] = False
    assert y[keep][:, :n].isfinite().all() and (y[70, :n] == float("inf")).all()
    assert db[[0, 2, 3]].isfinite().all() and db[1].isnan().all()


def test_results_repeat(tg):
    gen = torch.Generator(device="cuda").manual_seed(2)
    counts, n, k, dtype = [300, 41, 513], 264, 320, torch.float16
    r, g = sum(counts), 3
    x, b = padded(gen, r, k, 0, dtype), stacked(gen, g, k, n, 0, 0, dtype)
    offset = offsets(counts)
    out = []
    for _ in range(3):
        y, db = torch.empty(r, n, device="cuda", dtype=dtype), torch.empty(g, k, n, device="cuda", dtype=dtype)
        tg.grouped_gemm(r, n, k, g, x, r, k, None, 1, b, n, k * n, tg.TG_OP_N, offset, y, n, tg.TG_F16)
        tg.grouped_gemm_grad(r, n, k, g, y, n, x, r, k, None, 1, offset, db, n, k * n, tg.TG_OP_N, tg.TG_F16)
        out.append((y, db))
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(o, out[0]))


# -------------------------------------------------------------- combining

COMBINE = [(1, 1, 1), (1, 8, 4096), (17, 3, 200), (33, 9, 77), (300, 2, 1024), (5, 40, 24)]


def combine_case(gen, t, k, d, aligned, dtype):
    pad = 8 if aligned else 3
    r = t * k + 2
    make = lambda n: padded(gen, n, d, pad, dtype) if aligned else torch.randn(n, d + pad, generator=gen, device="cuda").to(dtype)[:, 1:d + 1]  # noqa: E731
    place = torch.randperm(r, generator=gen, device="cuda")[:t * k].int().view(t, k)
    if t > 2:
        place[1] = -1
        place[2, 0] = r
    weight = torch.randn(t, k, generator=gen, device="cuda")
    return make, r, place, weight


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,k,d", COMBINE)
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(tg, t, k, d, aligned, weighted, dtype):
    gen = torch.Generator(device="cuda").manual_seed(t + d)
    make, r, place, weight = combine_case(gen, t, k, d, aligned, dtype)
    if t > 2:
        weight[1] = float("nan")  # of no place: no part of the sum
    y, out = make(r), make(t)
    tg.combine(t, k, d, y, r, y.stride(0), place, weight if weighted else None, out, out.stride(0), code(tg, dtype))
    there = ((place >= 0) & (place < r))[..., None]
    w = torch.where(there[..., 0], weight.double() if weighted else torch.ones_like(weight, dtype=torch.float64), 0.0)[..., None]
    part = torch.where(there, y[place.long().clamp(0, r - 1)].double(), 0.0) * w
    want = part.sum(1)
    assert_within(out, want, rounded(want, (k + 1) * EPS32 * part.abs().sum(1), dtype), "out")
    if t > 2:
        assert (out[1] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("t,k,d", COMBINE)
@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_grad(tg, t, k, d, aligned, weighted, dtype):
    gen = torch.Generator(device="cuda").manual_seed(t + d)
    make, r, place, weight = combine_case(gen, t, k, d, aligned, dtype)
    y, dout, dy = make(r), make(t), make(r)
    before = dy.clone()
    dweight = torch.full((t, k), float("nan"), device="cuda")
    w = weight if weighted else None
    tg.combine_grad(t, k, d, dout, dout.stride(0), y, r, y.stride(0), place, w, dy, dy.stride(0), dweight, code(tg, dtype))
    there = (place >= 0) & (place < r)
    wide = (weight.double() if weighted else torch.ones_like(weight, dtype=torch.float64))
    named = torch.zeros(r, dtype=torch.bool, device="cuda")
    for j in range(k):
        at = there[:, j]
        p = place[at, j].long()
        named[p] = True
        want = wide[at, j, None] * dout[at].double()
        assert_within(dy[p], want, rounded(want, EPS32 * want.abs(), dtype), "dy")
        terms = dout[at].double() * y[p].double()
        assert_within(dweight[at, j], terms.sum(1), (d / 64 + 16) * EPS32 * terms.abs().sum(1) + 1e-37, "dweight")
    assert (dweight[~there] == 0).all()
    assert torch.equal(dy[~named].view(torch.int16), before[~named].view(torch.int16))
    # one of the two alone
    again, one = make(r), torch.empty(t, k, device="cuda")
    tg.combine_grad(t, k, d, dout, dout.stride(0), None, r, 0, place, w, again, again.stride(0), None, code(tg, dtype))
    tg.combine_grad(t, k, d, dout, dout.stride(0), y, r, y.stride(0), place, w, None, 0, one, code(tg, dtype))
    assert torch.equal(again[named], dy[named]) and torch.equal(one, dweight)


# --------------------------------------------------------------- adapters

def adapters_case(tg, gen, counts, t, n, k, rank, dtype, scaled=True):
    g, used = len(counts), sum(counts)
    x, y = padded(gen, t, k, 8, dtype), padded(gen, t, n, 8, dtype)
    ld = (k + 7) // 8 * 8
    a = torch.full((g, rank, ld), float("nan"), device="cuda", dtype=dtype)
    a[:, :, :k] = (torch.randn(g, rank, k, generator=gen, device="cuda") / k**0.5).to(dtype)
    lb = (rank + 7) // 8 * 8 + 8
    b = torch.full((g, n, lb), float("nan"), device="cuda", dtype=dtype)
    b[:, :, :rank] = torch.randn(g, n, rank, generator=gen, device="cuda").to(dtype)
    scale = torch.rand(g, generator=gen, device="cuda") + 0.5 if scaled else None
    row = torch.full((t,), -1, device="cuda", dtype=torch.int32)
    row[:used] = torch.randperm(t, generator=gen, device="cuda")[:used].int()
    before = y.clone()
    size = tg.tg_adapters_workspace_size(t, n, k, rank, g, code(tg, dtype))
    ws = torch.randint(0, 255, (size,), device="cuda", dtype=torch.uint8)
    offset = offsets(counts)

    def call(stream=None):
        tg.adapters(t, n, k, rank, g, x, x.stride(0), row, offset, a, ld, b, lb, scale, y, y.stride(0), code(tg, dtype), ws, size,
                    stream=stream)

    def check(start):
        touched = torch.zeros(t, dtype=torch.bool, device="cuda")
        lo = 0
        for q, c in enumerate(counts):
            at = row[lo:lo + c].long()
            touched[at] = True
            xs, aq, bq = x[at].double(), a[q, :, :k].double().T, b[q, :, :rank].double().T
            low = xs @ aq
            # fp32 or tensor-core sums of K products; then 22 bits of each value relative to its row's largest
            off = (k / 16 + 34) * 2 * EPS32 * (xs.abs() @ aq.abs()) + 2.0**-15 * low.abs().amax(1, keepdim=True) * (2.0**-6 if dtype == torch.float16 else 1.0)
            s = scale[q].double() if scaled else 1.0
            delta = s * (low @ bq)
            want = start[at].double() + delta
            slack = s * (off @ bq.abs()) + (rank / 8 + 8) * 2 * EPS32 * s * (low.abs() @ bq.abs()) + 2 * EPS32 * (want.abs() + delta.abs())
            assert_within(y[at], want, rounded(want, slack, dtype), f"adapter {q}")
            lo += c
        assert torch.equal(y[~touched].view(torch.int16), start[~touched].view(torch.int16))

    return call, check, before, y


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("counts,spare,n,k,rank", [
    ([1], 0, 1, 1, 1), ([1] * 64, 0, 520, 600, 16), ([0, 3, 0, 1], 2, 77, 100, 4), ([5, 0, 60], 3, 300, 1025, 8),
    ([1] * 300, 1, 40, 64, 24), ([700, 129, 0, 1], 5, 513, 264, 64), ([2500], 0, 264, 72, 128), ([300, 128], 0, 128, 2000, 33),
    ([0], 4, 64, 64, 8)])
def test_adapters(tg, counts, spare, n, k, rank, dtype):
    gen = torch.Generator(device="cuda").manual_seed(n + rank)
    call, check, before, _ = adapters_case(tg, gen, counts, sum(counts) + spare, n, k, rank, dtype, scaled=n % 2 == 0)
    call()
    assert tg.tg_debug_status()[0] == tg.TG_OK
    check(before)


def test_adapters_captured_and_replayed(tg):
    gen = torch.Generator(device="cuda").manual_seed(1)
    call, check, before, y = adapters_case(tg, gen, [3, 200, 1], 210, 136, 128, 16, torch.bfloat16)
    call()
    check(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(torch.cuda.current_stream())
    for _ in range(2):
        start = y.clone()
        graph.replay()
        check(start)


# --------------------------------------------- a layer of experts, as used

def test_layer_of_experts(tg):
    """Router, grouping, two products, the sum, and all gradients, against automatic
    differentiation in 64 bits of the same chosen experts; captured once, replayed on new tokens."""
    t, e, k, d, f, dtype = 130, 8, 2, 96, 136, torch.bfloat16
    dt, r = tg.TG_BF16, 260
    gen = torch.Generator(device="cuda").manual_seed(6)
    new = lambda *n, like=dtype: torch.empty(*n, device="cuda", dtype=like)  # noqa: E731
    x, logits, dout = new(t, d), new(t, e), new(t, d)
    w1 = (torch.randn(e, f, d, generator=gen, device="cuda") / d**0.5).to(dtype)
    w2 = (torch.randn(e, d, f, generator=gen, device="cuda") / f**0.5).to(dtype)
    index, weight = new(t, k, like=torch.int32), new(t, k, like=torch.float32)
    offset, row, place = new(e + 1, like=torch.int32), new(r, like=torch.int32), new(t, k, like=torch.int32)
    h, y, out = new(r, f), new(r, d), new(t, d)
    dy, dh, dxg, dx = new(r, d), new(r, f), new(r, d), new(t, d)
    dw1, dw2, dweight, dlogits = new(e, f, d), new(e, d, f), new(t, k, like=torch.float32), new(t, e)
    opts = tg.make_route_options(k, tg.TG_ROUTE_SIGMOID, renormalise=True)
    ws = new(max(1, tg.tg_group_rows_workspace_size(r, e)), like=torch.uint8)

    def step():
        s = torch.cuda.current_stream()
        tg.route(t, e, logits, e, None, index, weight, dt, opts, stream=s)
        tg.group_rows(r, e, index, offset, row, place, ws, ws.numel(), stream=s)
        tg.grouped_gemm(r, f, d, e, x, t, d, row, k, w1, d, f * d, tg.TG_OP_T, offset, h, f, dt, tg.make_group_epilogue(relu=True), stream=s)
        tg.grouped_gemm(r, d, f, e, h, r, f, None, 1, w2, f, d * f, tg.TG_OP_T, offset, y, d, dt, stream=s)
        tg.combine(t, k, d, y, r, d, place, weight, out, d, dt, stream=s)
        tg.combine_grad(t, k, d, dout, d, y, r, d, place, weight, dy, d, dweight, dt, stream=s)
        tg.route_grad(t, e, logits, e, index, dweight, dlogits, e, dt, opts, stream=s)
        tg.grouped_gemm_grad(r, d, f, e, dy, d, h, r, f, None, 1, offset, dw2, f, d * f, tg.TG_OP_T, dt, stream=s)
        tg.grouped_gemm(r, f, d, e, dy, r, d, None, 1, w2, f, d * f, tg.TG_OP_N, offset, dh, f, dt,
                        tg.make_group_epilogue(relu_of=h, ld_relu=f), stream=s)
        tg.grouped_gemm_grad(r, f, d, e, dh, f, x, t, d, row, k, offset, dw1, d, f * d, tg.TG_OP_T, dt, stream=s)
        tg.grouped_gemm(r, d, f, e, dh, r, f, None, 1, w1, d, f * d, tg.TG_OP_N, offset, dxg, d, dt, stream=s)
        tg.combine(t, k, d, dxg, r, d, place, None, dx, d, dt, stream=s)

    def fill():
        x.copy_(torch.randn(t, d, generator=gen, device="cuda"))
        logits.copy_(torch.randn(t, e, generator=gen, device="cuda"))
        logits[7] = float("-inf")  # a padding token
        dout.copy_(torch.randn(t, d, generator=gen, device="cuda"))

    def check():
        leaves = [v.double().requires_grad_() for v in (x, w1, w2, logits)]
        xx, a, b, ll = leaves
        total = torch.zeros(t, d, device="cuda", dtype=torch.float64)
        chosen = index.long().clamp(min=0)
        there = (index >= 0).double()
        s = torch.sigmoid(torch.where(ll.isfinite(), ll, 0.0)).gather(1, chosen) * there
        ww = s / s.sum(1, keepdim=True).clamp(min=1e-300)
        for j in range(k):
            hid = torch.relu(torch.einsum("td,tfd->tf", xx, a[chosen[:, j]]))
            total = total + (ww[:, j] * there[:, j])[:, None] * torch.einsum("tf,tdf->td", hid, b[chosen[:, j]])
        grads = torch.autograd.grad((total * dout.double()).sum(), leaves)
        # each chain of at most four tensors is rounded to 16 bits on its way, each time by
        # 2^-8 of a value; sums of f or d such terms of either sign, six deviations wide
        for got, want in zip((out, dx, dw1, dw2, dlogits), (total, *grads)):
            size = want.square().mean().sqrt()
            assert_within(got, want, 4 * HALF_ULP[dtype] * (want.abs() + 6 * size), "layer")
        assert (out[7] == 0).all() and (dx[7] == 0).all() and (dlogits[7] == 0).all()

    fill()
    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        fill()
        graph.replay()
        check()
    assert tg.tg_debug_status()[0] == tg.TG_OK
