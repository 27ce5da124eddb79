"""Routing, its gradient and grouping against their 64-bit forms."""
import math

import pytest
import torch

from rows_reference import EPS32, HALF_ULP, TINY, assert_within, code, group_rows, route, route_weights

pytestmark = pytest.mark.gpu


def logits_of(gen, t, e, pad, dtype, scale=1.5):
    full = torch.full((t, e + pad), float("nan"), dtype=dtype, device="cuda")
    full[:, :e] = (torch.randn(t, e, generator=gen, device="cuda") * scale).to(dtype)
    return full[:, :e]


def run(tg, logits, bias, k, sigmoid=False, groups=1, kept=1, top=1, renorm=False, scale=1.0):
    t, e = logits.shape
    index = torch.full((t, k), -7, dtype=torch.int32, device="cuda")
    weight = torch.full((t, k), float("nan"), device="cuda")
    tg.route(t, e, logits, logits.stride(0), bias, index, weight, code(tg, logits.dtype),
             tg.make_route_options(k, tg.TG_ROUTE_SIGMOID if sigmoid else tg.TG_ROUTE_SOFTMAX, groups, kept, top, renorm, scale))
    return index, weight


def weight_bound(want, e):
    """fp32 exponentials within 2 ulp of an argument rounded once (64 steps of 2^-24
    cover |l - max| < 32 and the sums of E terms), the quotient and the scale."""
    return (96 + e / 16) * EPS32 * want.abs() + 1e-37


CASES = [
    # t, e, k, sigmoid, bias, groups, kept, top, renorm, scale
    (1, 1, 1, False, False, 1, 1, 1, False, 1.0),
    (1, 256, 8, True, True, 8, 4, 2, True, 2.5),
    (37, 60, 4, False, False, 1, 1, 1, True, 1.0),
    (5, 33, 32, False, False, 1, 1, 1, False, 1.0),
    (65, 8, 2, True, False, 1, 1, 1, True, 1.0),
    (129, 257, 6, True, True, 1, 1, 1, False, 1.0),
    (70, 1024, 8, False, True, 32, 5, 1, False, 3.0),
    (70, 96, 7, True, False, 3, 2, 2, True, 1.0),
    (33, 40, 8, False, False, 4, 1, 1, True, 1.0),
    (50, 512, 16, False, True, 16, 3, 2, True, 1.0),
    (31, 32, 3, True, True, 32, 9, 2, True, 1.0),   # groups of one expert
    # many tokens: longer runs of experts per lane
    (2100, 16, 2, False, True, 1, 1, 1, True, 1.0),
    (2100, 160, 6, True, True, 4, 2, 2, True, 1.0),
    (2081, 64, 8, False, False, 2, 1, 2, False, 1.0),
    (2049, 1022, 5, True, True, 14, 3, 2, False, 1.0),  # 14 groups of 73: runs of 37
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,e,k,sigmoid,biased,groups,kept,top,renorm,scale", CASES)
def test_route(tg, t, e, k, sigmoid, biased, groups, kept, top, renorm, scale, dtype):
    gen = torch.Generator(device="cuda").manual_seed(e * 7 + k)
    logits = logits_of(gen, t, e, 3, dtype)
    bias = torch.randn(e, generator=gen, device="cuda") * 0.1 if biased else None
    index, weight = run(tg, logits, bias, k, sigmoid, groups, kept, top, renorm, scale)
    want_index, want = route(logits, bias, k, sigmoid, groups, kept, top, renorm, scale)
    assert torch.equal(index, want_index)
    assert_within(weight, want, weight_bound(want, e), "weight")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_equal_keys_go_to_the_lowest_index(tg, sigmoid, groups, kept, top):
    """Few different logits, and a bias of zeros as training starts with: ties everywhere."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randint(-2, 3, (64, 64), generator=gen, device="cuda").to(torch.bfloat16)
    logits[0] = 0.0
    logits[1] = -0.0
    logits[1, ::2] = 0.0
    for bias in (None, torch.zeros(64, device="cuda")):
        index, weight = run(tg, logits, bias, 8, sigmoid, groups, kept, top, True)
        want_index, want = route(logits, bias, 8, sigmoid, groups, kept, top, True, 1.0)
        assert torch.equal(index, want_index)
        assert_within(weight, want, weight_bound(want, 64), "weight")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,kept", [(1, 1), (4, 2)])
def test_keys_nearer_than_fp32_can_tell(tg, sigmoid, groups, kept):
    """Biases that make up for the scores' differences but for a few parts in 2^24 or
    less: only 64 bits rank them."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    logits = torch.randn(1, 64, generator=gen, device="cuda")
    score = torch.sigmoid(logits.double()) if sigmoid else torch.softmax(logits.double(), 1)
    bias = (0.7 - score[0]).float()
    rows = logits.repeat(40, 1)
    index, weight = run(tg, rows, bias, 8, sigmoid, groups, kept, 2, False)
    want_index, want = route(rows, bias, 8, sigmoid, groups, kept, 2, False, 1.0)
    assert torch.equal(index, want_index)
    assert_within(weight, want, weight_bound(want, 64), "weight")


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (4, 2, 2)])
def test_masked_experts(tg, sigmoid, renorm, biased, groups, kept, top):
    """-inf and NaN are never chosen; rows that leave too few, or none."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = logits_of(gen, 12, 32, 0, torch.float32)
    inf = float("inf")
    logits[0] = -inf
    logits[1, 3:] = -inf
    logits[2, ::2] = -inf
    logits[3, 5] = float("nan")
    logits[4] = torch.finfo(torch.float32).min
    logits[5, 7] = inf
    logits[6, :31] = -inf
    logits[7, 8:24] = -inf
    logits[8] = -300.0 - torch.arange(32, device="cuda")
    logits[9] = 90.0 + torch.arange(32, device="cuda")
    logits[10, :] = -inf
    logits[10, 9] = float("nan")
    bias = torch.randn(32, generator=gen, device="cuda") * 0.1 if biased else None
    index, weight = run(tg, logits, bias, 6, sigmoid, groups, kept, top, renorm, 2.0)
    want_index, want = route(logits, bias, 6, sigmoid, groups, kept, top, renorm, 2.0)
    assert torch.equal(index, want_index)
    # (arguments of exponentials up to 400 apart: 2^-24 of them each)
    assert_within(weight, want, 1024 * EPS32 * want.abs() + 1e-37, "weight")
    assert (index[0] == -1).all() and (weight[0] == 0).all()


def test_low_sigmoid_scores_renormalise(tg):
    logits = torch.tensor([[-200.0, -201.0, -400.0, -203.0]], device="cuda")
    index, weight = run(tg, logits, None, 3, True, renorm=True)
    assert index.tolist() == [[0, 1, 3]]
    want = torch.softmax(torch.tensor([-200.0, -201.0, -203.0], dtype=torch.float64), 0)
    assert_within(weight[0].cpu(), want, 64 * EPS32 * want, "weight")


def grad(tg, logits, index, dweight, sigmoid, renorm, scale, pad=0):
    t, e = logits.shape
    k = index.shape[1]
    full = torch.full((t, e + pad), 7.0, dtype=logits.dtype, device="cuda")
    out = full[:, :e]
    tg.route_grad(t, e, logits, logits.stride(0), index, dweight, out, out.stride(0), code(tg, logits.dtype),
                  tg.make_route_options(k, tg.TG_ROUTE_SIGMOID if sigmoid else tg.TG_ROUTE_SOFTMAX, renormalise=renorm, scale=scale))
    assert pad == 0 or (full[:, e:] == 7.0).all()
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 256, 8), (67, 60, 4), (33, 1000, 32), (300, 129, 6)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad(tg, t, e, k, sigmoid, renorm, dtype):
    gen = torch.Generator(device="cuda").manual_seed(t + e)
    logits = logits_of(gen, t, e, 5, dtype)
    index, _ = run(tg, logits, None, k, sigmoid, renorm=renorm)
    if t > 3 and k > 1:
        index[1, 1] = -1      # fewer than k experts
        index[2] = -1         # none
        index[3, 0] = e       # out of range: as -1
    dweight = torch.randn(t, k, generator=gen, device="cuda")
    got = grad(tg, logits, index, dweight, sigmoid, renorm, 1.5, 2)
    wide = logits.double().requires_grad_()
    clean = torch.where((index >= 0) & (index < e), index, -1)
    w = route_weights(wide, clean, sigmoid, renorm, 1.5)
    want = torch.autograd.grad((torch.where(clean >= 0, w, 0.0) * dweight.double()).sum(), wide)[0].nan_to_num()
    # every term of the sums is a weight times an upstream gradient, exponentials as in weight_bound
    size = 1.5 * dweight.abs().amax(1, keepdim=True).double() * 4
    unit = HALF_ULP.get(dtype, EPS32)
    assert_within(got, want, (160 + e / 16) * EPS32 * size + 1.01 * unit * want.abs() + TINY.get(dtype, 0.0), "dlogits")
    if t > 3 and k > 1:
        assert (got[2] == 0).all()


def test_route_grad_against_differences(tg):
    gen = torch.Generator(device="cuda").manual_seed(9)
    logits = logits_of(gen, 3, 12, 0, torch.float32)
    dweight = torch.randn(3, 4, generator=gen, device="cuda")
    for sigmoid in (False, True):
        for renorm in (False, True):
            index, _ = run(tg, logits, None, 4, sigmoid, renorm=renorm)
            got = grad(tg, logits, index, dweight, sigmoid, renorm, 1.0).double()
            step = 1e-5
            for e in range(12):
                move = torch.zeros_like(logits, dtype=torch.float64)
                move[:, e] = step
                diff = [(route_weights(logits.double() + s * move, index, sigmoid, renorm, 1.0) * dweight.double()).sum(1) for s in (1, -1)]
                # central differences are off by step^2 / 6 of a third derivative of at most about 4
                assert_within(got[:, e], (diff[0] - diff[1]) / (2 * step), 1e-6 + 160 * EPS32 * 8, "difference")


def test_route_grad_adds_up_an_expert_named_twice(tg):
    logits = torch.tensor([[0.3, -0.2, 0.9]], device="cuda")
    dweight = torch.tensor([[0.5, 0.25]], device="cuda")
    got = grad(tg, logits, torch.tensor([[1, 1]], dtype=torch.int32, device="cuda"), dweight, True, False, 1.0)
    s = torch.sigmoid(logits.double()[0, 1])
    assert got[0, 0] == 0 and got[0, 2] == 0
    assert_within(got[0, 1], 0.75 * s * (1 - s), torch.tensor(32 * EPS32, dtype=torch.float64), "twice")


def test_masked_rows_have_no_gradient(tg):
    logits = torch.full((2, 40), float("-inf"), device="cuda")
    logits[1, 3] = 0.5
    index = torch.tensor([[-1, -1], [3, -1]], dtype=torch.int32, device="cuda")
    for sigmoid in (False, True):
        for renorm in (False, True):
            got = grad(tg, logits, index, torch.ones(2, 2, device="cuda"), sigmoid, renorm, 1.0)
            assert got.isfinite().all() and (got[0] == 0).all() and (got[1, :3] == 0).all()


# --------------------------------------------------------------- grouping

def group(tg, index, g, with_place=True):
    r = index.numel()
    offset = torch.full((g + 1,), -9, dtype=torch.int32, device="cuda")
    row = torch.full((r,), -9, dtype=torch.int32, device="cuda")
    place = torch.full((r,), -9, dtype=torch.int32, device="cuda") if with_place else None
    size = tg.tg_group_rows_workspace_size(r, g)
    ws = torch.randint(0, 255, (max(1, size),), dtype=torch.uint8, device="cuda")
    tg.group_rows(r, g, index, offset, row, place, ws, size)
    return offset, row, place


@pytest.mark.parametrize("r,g", [(1, 1), (1, 4096), (5, 3), (32, 7), (2047, 60), (2048, 256), (2049, 256), (5000, 1),
                                 (6001, 4096), (70000, 129), (131072, 5), (131073, 300), (400000, 64)])
@pytest.mark.parametrize("kind", ["even", "one", "dropped", "none"])
def test_group_rows(tg, r, g, kind):
    gen = torch.Generator(device="cuda").manual_seed(r + g)
    index = torch.randint(0, g, (r,), generator=gen, device="cuda", dtype=torch.int32)
    if kind == "one":
        index[:] = g - 1
    elif kind == "dropped":
        index[torch.rand(r, generator=gen, device="cuda") < 0.4] = -1
        index[::7] = g
        index[::11] = 2**31 - 1
    elif kind == "none":
        index[:] = -1
    offset, row, place = group(tg, index, g)
    if r <= 7000:
        w_offset, w_row, w_place = group_rows(index, g) if g <= 300 else (None, None, None)
    else:
        w_offset = None
    inside = (index >= 0) & (index < g)
    order = torch.sort(torch.where(inside, index, g).long(), stable=True).indices
    total = int(inside.sum())
    want_row = torch.where(torch.arange(r, device="cuda") < total, order, -1).int()
    want_offset = torch.cat([torch.zeros(1, device="cuda", dtype=torch.long), torch.bincount(index[inside].long(), minlength=g).cumsum(0)])
    assert torch.equal(row, want_row) and torch.equal(offset.long(), want_offset)
    if w_offset is not None:
        assert offset.tolist() == w_offset and row.tolist() == w_row and place.tolist() == w_place
    want_place = torch.full((r,), -1, device="cuda", dtype=torch.int32)
    want_place[order[:total]] = torch.arange(total, device="cuda", dtype=torch.int32)
    assert torch.equal(place, want_place)
    again = group(tg, index, g, with_place=False)
    assert torch.equal(again[0], offset) and torch.equal(again[1], row)


def test_route_and_group_captured_and_replayed(tg):
    """New logits in the same graph; on a stream of its own."""
    t, e, k = 700, 48, 5
    logits = torch.empty(t, e, device="cuda", dtype=torch.bfloat16)
    index = torch.empty(t, k, device="cuda", dtype=torch.int32)
    weight = torch.empty(t, k, device="cuda")
    offset = torch.empty(e + 1, device="cuda", dtype=torch.int32)
    row, place = torch.empty(2, t * k, device="cuda", dtype=torch.int32).unbind(0)
    size = tg.tg_group_rows_workspace_size(t * k, e)
    ws = torch.empty(max(1, size), device="cuda", dtype=torch.uint8)
    opts = tg.make_route_options(k, renormalise=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits.copy_(torch.randn(t, e, generator=gen, device="cuda"))
    stream = torch.cuda.Stream()

    def call():
        tg.route(t, e, logits, e, None, index, weight, tg.TG_BF16, opts, stream=torch.cuda.current_stream())
        tg.group_rows(t * k, e, index, offset, row, place, ws, size, stream=torch.cuda.current_stream())

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        logits.copy_(torch.randn(t, e, generator=gen, device="cuda"))
        graph.replay()
        want_index, want = route(logits, None, k, False, 1, 1, 1, True, 1.0)
        assert torch.equal(index, want_index)
        assert_within(weight, want, weight_bound(want, e), "weight")
        w_offset, w_row, w_place = group_rows(index, e)
        assert offset.tolist() == w_offset and row.tolist() == w_row and place.tolist() == w_place
