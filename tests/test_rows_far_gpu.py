"""Rows and matrices that lie more than 2^31 elements apart, calls on two streams
at once and of two threads, and places that several tokens name."""
import threading

import pytest
import torch

from rows_reference import EPS32, assert_within, code, offsets, rounded, stacked

pytestmark = pytest.mark.gpu

STEP = (1 << 31) + 64  # elements from one row to the next


def far(x):
    """A copy of x (a few rows) whose rows are STEP elements apart."""
    flat = torch.empty((x.shape[0] - 1) * STEP + x.shape[1], dtype=x.dtype, device="cuda")
    view = flat.as_strided(x.shape, (STEP, 1))
    view.copy_(x)
    return view


def side_by_side_and_far(run):
    """Outputs of run(place) with operands side by side and far apart are the same."""
    ends = []
    for place in (lambda x: x.clone(), far):
        out = run(place)
        torch.cuda.synchronize()
        ends.append([x.clone().contiguous() for x in out])
        del out
        torch.cuda.empty_cache()
    for p, q in zip(*ends):
        assert torch.equal(p, q) and p.abs().max() > 0


def test_route(tg):
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(3, 96, generator=gen, device="cuda").bfloat16()
    dweight = torch.randn(3, 4, generator=gen, device="cuda")
    opts = tg.make_route_options(4, tg.TG_ROUTE_SIGMOID, 4, 2, 2, True)

    def run(place):
        x, dx = place(logits), place(torch.zeros_like(logits))
        index, weight = torch.empty(3, 4, dtype=torch.int32, device="cuda"), torch.empty(3, 4, device="cuda")
        tg.route(3, 96, x, x.stride(0), None, index, weight, tg.TG_BF16, opts)
        tg.route_grad(3, 96, x, x.stride(0), index, dweight, dx, dx.stride(0), tg.TG_BF16, opts)
        return index, weight, dx

    side_by_side_and_far(run)


@pytest.mark.parametrize("perm", [0, 1])
@pytest.mark.parametrize("listed", [False, True])
def test_grouped_products(tg, perm, listed):
    gen = torch.Generator(device="cuda").manual_seed(2)
    r, n, k = 3, 136, 72
    x, dy = (torch.randn(r, w, generator=gen, device="cuda").half() for w in (k, n))
    b = torch.randn(2, *((k, n) if perm == 0 else (n, k)), generator=gen, device="cuda").half()
    row = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda") if listed else None
    offset = offsets([1, 2])

    def run(place):
        xx, gg = place(x), place(dy)
        y = place(torch.zeros(r, n, dtype=torch.float16, device="cuda"))
        flat = torch.zeros((b[0].numel() if place is not far else STEP) + b[0].numel(), dtype=torch.float16, device="cuda")
        m = flat.as_strided(b.shape, (flat.numel() - b[0].numel(), b.shape[2], 1))
        m.copy_(b)
        tg.grouped_gemm(r, n, k, 2, xx, r, xx.stride(0), row, 1, m, m.stride(1), m.stride(0), perm, offset, y, y.stride(0), tg.TG_F16)
        first = y.clone()
        tg.grouped_gemm_grad(r, n, k, 2, gg, gg.stride(0), xx, r, xx.stride(0), row, 1, offset, m, m.stride(1), m.stride(0), perm, tg.TG_F16)
        return first, m

    side_by_side_and_far(run)


def test_combine_and_adapters(tg):
    gen = torch.Generator(device="cuda").manual_seed(3)
    y, dout = torch.randn(4, 80, generator=gen, device="cuda").bfloat16(), torch.randn(2, 80, generator=gen, device="cuda").bfloat16()
    place_of = torch.tensor([[3, 0], [1, 2]], dtype=torch.int32, device="cuda")
    weight = torch.randn(2, 2, generator=gen, device="cuda")
    a, b = torch.randn(2, 8, 80, generator=gen, device="cuda").bfloat16(), torch.randn(2, 80, 8, generator=gen, device="cuda").bfloat16()
    row = torch.tensor([3, 1, 0, 2], dtype=torch.int32, device="cuda")
    offset = offsets([1, 3])
    ws = torch.empty(tg.tg_adapters_workspace_size(4, 80, 80, 8, 2, tg.TG_BF16), dtype=torch.uint8, device="cuda")

    def run(place):
        yy, gg = place(y), place(dout)
        out, dy, dweight = place(torch.zeros_like(dout)), place(torch.zeros_like(y)), torch.zeros(2, 2, device="cuda")
        tg.combine(2, 2, 80, yy, 4, yy.stride(0), place_of, weight, out, out.stride(0), tg.TG_BF16)
        tg.combine_grad(2, 2, 80, gg, gg.stride(0), yy, 4, yy.stride(0), place_of, weight, dy, dy.stride(0), dweight, tg.TG_BF16)
        z = place(y)
        tg.adapters(4, 80, 80, 8, 2, yy, yy.stride(0), row, offset, a, 80, b, 8, None, z, z.stride(0), tg.TG_BF16, ws, ws.numel())
        return out, dy, dweight, z

    side_by_side_and_far(run)


def test_a_row_that_several_tokens_name(tg):
    gen = torch.Generator(device="cuda").manual_seed(4)
    y = torch.randn(3, 64, generator=gen, device="cuda").bfloat16()
    place = torch.tensor([[1, 1, 1], [0, 1, 2]], dtype=torch.int32, device="cuda")
    weight = torch.randn(2, 3, generator=gen, device="cuda")
    out, dweight = torch.empty(2, 64, device="cuda", dtype=torch.bfloat16), torch.empty(2, 3, device="cuda")
    tg.combine(2, 3, 64, y, 3, 64, place, weight, out, 64, tg.TG_BF16)
    tg.combine_grad(2, 3, 64, out, 64, y, 3, 64, place, None, None, 0, dweight, tg.TG_BF16)
    part = weight.double()[..., None] * y.double()[place.long()]
    want = part.sum(1)
    assert_within(out, want, rounded(want, 4 * EPS32 * part.abs().sum(1), torch.bfloat16), "out")
    terms = out.double()[:, None] * y.double()[place.long()]
    assert_within(dweight, terms.sum(2), 32 * EPS32 * terms.abs().sum(2), "dweight")


def test_two_streams_at_once(tg):
    """Products, their gradients and adapters of two independent sets of operands, queued on
    two streams, give what each gives alone."""
    dt, sets = torch.float16, []
    for seed in (5, 6):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        counts = [300, 5, 0, 260] if seed == 5 else [64, 129, 1, 40]
        r, n, k, g = sum(counts), 264, 320, 4
        x = torch.randn(r, k, generator=gen, device="cuda").to(dt)
        b = stacked(gen, g, n, k, 0, 0, dt)
        a, c = stacked(gen, g, 16, k, 0, 0, dt, 0.05), stacked(gen, g, n, 16, 0, 0, dt)
        row = torch.randperm(r, generator=gen, device="cuda").int()
        sets.append((r, n, k, g, x, b, a, c, row, offsets(counts)))

    def outputs(s):
        r, n, k, g = s[:4]
        y, db = torch.empty(r, n, device="cuda", dtype=dt), torch.empty(g, n, k, device="cuda", dtype=dt)
        z = torch.ones(r, n, device="cuda", dtype=dt)
        ws = torch.empty(tg.tg_adapters_workspace_size(r, n, k, 16, g, code(tg, dt)), device="cuda", dtype=torch.uint8)
        return y, db, z, ws

    def queue(s, out, stream=None):
        r, n, k, g, x, b, a, c, row, offset = s
        y, db, z, ws = out
        for _ in range(8):
            tg.grouped_gemm(r, n, k, g, x, r, k, row, 1, b, k, n * k, tg.TG_OP_T, offset, y, n, tg.TG_F16, stream=stream)
            tg.grouped_gemm_grad(r, n, k, g, y, n, x, r, k, row, 1, offset, db, k, n * k, tg.TG_OP_T, tg.TG_F16, stream=stream)
            tg.adapters(r, n, k, 16, g, x, k, row, offset, a, k, c, 16, None, z, n, tg.TG_F16, ws, ws.numel(), stream=stream)

    alone, both = [outputs(s) for s in sets], [outputs(s) for s in sets]
    for s, out in zip(sets, alone):
        queue(s, out)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for s, out, stream in zip(sets, both, streams):
        queue(s, out, stream)
    torch.cuda.synchronize()
    for p, q in zip(alone, both):
        assert all(torch.equal(u, v) for u, v in zip(p[:3], q[:3]))
    assert tg.tg_debug_status()[0] == tg.TG_OK


def test_two_threads_at_once(tg):
    """Calls whose kernels want different amounts of shared memory beyond the default, from
    two threads: none is refused for what the other one has set or for being its thread's
    first, and all give what they give alone."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    index = torch.randint(0, 4096, (2000,), generator=gen, device="cuda").int()
    logits = torch.randn(4000, 32, generator=gen, device="cuda")

    def outputs(groups, chosen):
        ints = lambda *shape: torch.empty(*shape, dtype=torch.int32, device="cuda")
        return ints(groups + 1), ints(2000), ints(4000, chosen), torch.empty(4000, chosen, device="cuda")

    def queue(groups, chosen, out, stream=None):
        tg.group_rows(2000, groups, index, out[0], out[1], None, None, 0, stream=stream)
        tg.route(4000, 32, logits, 32, None, out[2], out[3], tg.TG_F32, tg.make_route_options(chosen), stream=stream)

    sizes = [(4096, 32), (2100, 28)]
    alone, both = [outputs(*s) for s in sizes], [outputs(*s) for s in sizes]
    for s, out in zip(sizes, alone):
        queue(*s, out)
    torch.cuda.synchronize()
    refused = []

    def worker(s, out, stream):
        try:
            for _ in range(300):
                queue(*s, out, stream)
        except Exception as e:
            refused.append(e)

    threads = [threading.Thread(target=worker, args=(s, out, torch.cuda.Stream())) for s, out in zip(sizes, both)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused
    for p, q in zip(alone, both):
        assert all(torch.equal(u, v) for u, v in zip(p, q))
