"""Layer norm, linear cross entropy, their gradients and AdamW on the GPU,
against plain 64-bit forms.  Every tolerance is the bound that head_reference
derives from the library's roundings."""
import math

import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu

BOTH = [torch.float16, torch.bfloat16]


def code(tg, dt):
    return {torch.float16: tg.TG_F16, torch.bfloat16: tg.TG_BF16, torch.float32: tg.TG_F32}[dt]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ok(tg):
    torch.cuda.synchronize()
    st, detail = tg.tg_debug_status()
    assert st == tg.TG_OK, hex(detail)


def workspace(n):
    # old bytes are NaN patterns: nothing may depend on them
    return torch.full((max(1, n),), 0xFF, dtype=torch.uint8, device="cuda")


def padded(n, d, pad, dt):
    full = torch.full((n, d + pad), 77.0, dtype=dt, device="cuda")
    return full, full[:, :d]


# ------------------------------------------------------------- layer norm

LN = [(1, 1, 0), (1, 7, 1), (3, 64, 0), (5, 100, 3), (17, 255, 0), (9, 256, 8), (4, 1000, 24),
      (33, 1024, 0), (2, 1026, 2), (6, 3001, 0), (7, 4096, 0), (3, 8200, 0), (2, 8193, 0), (2, 16384, 0),
      (2, 16386, 0), (3, 32768, 0), (2, 40001, 0), (1500, 72, 0), (700, 2048, 8)]


@pytest.mark.parametrize("dt", BOTH, ids=["f16", "bf16"])
@pytest.mark.parametrize("n,d,pad", LN)
def test_layernorm(tg, n, d, pad, dt):
    g = gen(n * 1000 + d)
    x = ref.rows(g, n, d, pad, dt, 1.5) + 0.5
    x = ref.rows(g, n, d, pad, dt).copy_(x)
    w, b = ref.rows(g, 1, d, 0, dt)[0], ref.rows(g, 1, d, 0, dt)[0]
    for bias in (b, None):
        full, y = padded(n, d, pad, dt)
        mean, rstd = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        tg.layernorm(n, d, x, x.stride(0), w, bias, 1e-5, y, y.stride(0), mean, rstd, code(tg, dt))
        ok(tg)
        wy, wm, wr = ref.layernorm(x, w, bias, 1e-5)
        # a sum of d terms over at most 1024 threads: each adds at most d/32 + 48 times
        adds = d / 32 + 48
        size = x.double().abs().mean(1)
        bm = adds * ref.EPS32 * 2 * size
        ref.assert_within(mean, wm, bm, "mean")
        # variance off relatively by adds/2^24, and by what the mean is off, squared (below that)
        var = wr**-2
        br = wr * (adds * ref.EPS32 + 4 * ref.EPS32 + bm**2 / var)
        ref.assert_within(rstd, wr, br, "rstd")
        xh = (x.double() - wm[:, None]) * wr[:, None]
        by = (bm * wr)[:, None] + xh.abs() * ((br / wr)[:, None] + 8 * ref.EPS32)
        by = by * w.double().abs() + ref.HALF_ULP[dt] * 1.01 * wy.abs() + 4 * ref.EPS32 * (
            xh * w.double()).abs() + ref.TINY[dt]
        ref.assert_within(y, wy, by, "y")
        assert (full[:, d:] == 77).all()


@pytest.mark.parametrize("dt", BOTH, ids=["f16", "bf16"])
@pytest.mark.parametrize("n,d,pad", LN)
def test_layernorm_grad(tg, n, d, pad, dt):
    g = gen(n * 1000 + d + 1)
    x, dy = ref.rows(g, n, d, pad, dt), ref.rows(g, n, d, pad, dt)
    w = ref.rows(g, 1, d, 0, dt)[0]
    _, mean, rstd = (t.float() for t in ref.layernorm(x, w, None, 1e-5))
    wx, ww, wb = ref.layernorm_grad(dy, x, w, mean, rstd)
    size = tg.tg_layernorm_grad_workspace_size(n, d, code(tg, dt))
    ws = workspace(size)
    first = None
    for with_bias in (True, True, False):
        full, dx = padded(n, d, pad, dt)
        dw, db = torch.empty(d, dtype=dt, device="cuda"), torch.empty(d, dtype=dt, device="cuda")
        tg.layernorm_grad(n, d, dy, dy.stride(0), x, x.stride(0), w, mean, rstd, dx, dx.stride(0), dw,
                          db if with_bias else None, code(tg, dt), ws, size)
        ok(tg)
        u = ref.HALF_ULP[dt] * 1.01
        xh = ((x.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs()
        gg = (dy.double() * w.double()).abs()
        adds = d / 32 + 48
        # xh is off by 3 roundings; g by one; the two means by their sums' additions
        c1 = adds * ref.EPS32 * gg.mean(1, keepdim=True)
        c2 = (adds + 8) * ref.EPS32 * (gg * xh).mean(1, keepdim=True)
        m2 = (dy.double() * w.double() * (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
              ).mean(1, keepdim=True).abs()
        bx = rstd.double()[:, None] * (c1 + xh * c2 + 8 * ref.EPS32 * (gg + gg.mean(1, keepdim=True) + xh * m2))
        ref.assert_within(dx, wx, bx + u * wx.abs() + ref.TINY[dt], "dx")
        adds = n + 64
        ref.assert_within(dw, ww, (adds + 4) * ref.EPS32 * (dy.double().abs() * xh).sum(0) + u * ww.abs()
                          + ref.TINY[dt], "dweight")
        if with_bias:
            ref.assert_within(db, wb, adds * ref.EPS32 * dy.double().abs().sum(0) + u * wb.abs()
                              + ref.TINY[dt], "dbias")
        assert (full[:, d:] == 77).all()
        if first is not None:  # the same bits each time
            assert torch.equal(first[0], dx) and torch.equal(first[1], dw)
        first = (dx.clone(), dw.clone())


def test_layernorm_grad_against_differences(tg):
    """<dx, u>, <dw, u>, <db, u> against central differences of <y, dy> in 64 bits."""
    n, d, dt = 6, 136, torch.float16
    g = gen(5)
    x, dy = ref.rows(g, n, d, 0, dt), ref.rows(g, n, d, 0, dt)
    w, b = ref.rows(g, 1, d, 0, dt)[0], ref.rows(g, 1, d, 0, dt)[0]
    _, mean, rstd = (t.float() for t in ref.layernorm(x, w, None, 1e-5))
    size = tg.tg_layernorm_grad_workspace_size(n, d, tg.TG_F16)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    tg.layernorm_grad(n, d, dy, d, x, d, w, mean, rstd, dx, d, dw, db, tg.TG_F16, workspace(size), size)
    ok(tg)
    h = 1e-4
    f = lambda x, w, b: float((ref.layernorm(x, w, b, 1e-5)[0] * dy.double()).sum())  # noqa: E731
    for what, grad, at in (("dx", dx, 0), ("dw", dw, 1), ("db", db, 2)):
        u = torch.randn(grad.shape, generator=g, device="cuda", dtype=torch.float64)
        lo, hi = ([t.double() for t in (x, w, b)] for _ in range(2))
        lo[at], hi[at] = lo[at] - h * u, hi[at] + h * u
        diff = (f(*hi) - f(*lo)) / (2 * h)
        # the gradient's own rounding, and the third derivative times h^2 / 6
        # (y has scale 1, so each derivative of it along u is of the size of |u|^k |dy|)
        room = ref.HALF_ULP[dt] * 1.1 * float((grad.double() * u).abs().sum())
        room += h * h * 100 * float(u.norm()) ** 3 * float(dy.double().norm())
        assert abs(float((grad.double() * u).sum()) - diff) <= room, what


# --------------------------------------------------- linear cross entropy

CE = [  # T, V, D, pad of the rows
    (1, 1, 1, 0), (1, 1000, 64, 0), (2, 33, 8, 0), (7, 129, 40, 8), (31, 500, 100, 0), (128, 512, 128, 0),
    (129, 513, 192, 0), (100, 2000, 333, 0), (256, 1024, 256, 0), (300, 3001, 520, 16), (257, 777, 72, 5),
    (513, 5003, 264, 0), (90, 70001, 64, 0), (1100, 256, 1032, 0)]


def ce_problem(t, v, d, pad, dt, seed, ignored=0.2):
    g = gen(seed)
    h, w = ref.rows(g, t, d, pad, dt), ref.rows(g, v, d, pad, dt, 2 / math.sqrt(d))
    target = torch.randint(0, v, (t,), device="cuda", generator=g)
    drop = torch.rand(t, device="cuda", generator=g) < ignored
    outside = torch.where(torch.arange(t, device="cuda") % 2 == 0, -100, v)
    return h, w, torch.where(drop, outside, target), g


def forward(tg, h, w, target, dt, stream=None):
    t, v, d = h.shape[0], w.shape[0], h.shape[1]
    size = tg.tg_linear_ce_workspace_size(t, v, d, h, h.stride(0), w, w.stride(0), code(tg, dt))
    out = torch.full((2, t + 1), 77.0, device="cuda")
    tg.linear_ce(t, v, d, h, h.stride(0), w, w.stride(0), target, out[0], out[1], code(tg, dt),
                 workspace(size), size, stream)
    ok(tg)
    assert (out[:, t] == 77).all()
    return out[0, :t], out[1, :t]


def backward(tg, h, w, target, lse, dloss, dt, want=(True, True), pads=(0, 0)):
    t, v, d = h.shape[0], w.shape[0], h.shape[1]
    fh, dh = padded(t, d, pads[0], dt)
    fw, dw = padded(v, d, pads[1], dt)
    a = dh if want[0] else None
    b = dw if want[1] else None
    size = tg.tg_linear_ce_grad_workspace_size(t, v, d, h, h.stride(0), w, w.stride(0), a, dh.stride(0), b,
                                               dw.stride(0), code(tg, dt))
    tg.linear_ce_grad(t, v, d, h, h.stride(0), w, w.stride(0), target, lse, dloss, a, dh.stride(0), b,
                      dw.stride(0), code(tg, dt), workspace(size), size)
    ok(tg)
    assert (fh[:, d:] == 77).all() and (fw[:, d:] == 77).all()
    return dh, dw


@pytest.mark.parametrize("dt", BOTH, ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d,pad", CE)
def test_linear_ce(tg, t, v, d, pad, dt):
    h, w, target, _ = ce_problem(t, v, d, pad, dt, t + v + d)
    loss, lse = forward(tg, h, w, target, dt)
    want_loss, want = ref.linear_ce(h, w, target)
    bound = ref.lse_bound(h, w, want)
    ref.assert_within(lse, want, bound, "lse")
    ref.assert_within(loss, want_loss, 2 * bound, "loss")
    assert (loss[(target < 0) | (target >= v)] == 0).all()


@pytest.mark.parametrize("dt", BOTH, ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d,pad", CE)
def test_linear_ce_grad(tg, t, v, d, pad, dt):
    h, w, target, g = ce_problem(t, v, d, pad, dt, t + v + d + 1)
    _, lse = ref.linear_ce(h, w, target)
    lse = lse.float()
    for dloss in (torch.full((t,), 64.0 / t, device="cuda"), torch.randn(t, device="cuda", generator=g)):
        dh, dw = backward(tg, h, w, target, lse, dloss, dt, pads=(pad, pad))
        wh, ww, bh, bw = ref.linear_ce_grad(h, w, target, lse, dloss)
        ref.assert_within(dh, wh, bh, "dh")
        ref.assert_within(dw, ww, bw, "dw")
    only_h, _ = backward(tg, h, w, target, lse, dloss, dt, (True, False))
    _, only_w = backward(tg, h, w, target, lse, dloss, dt, (False, True))
    assert torch.equal(only_h, dh) and torch.equal(only_w, dw)  # and the same bits each time


def test_linear_ce_grad_in_several_pieces(tg):
    """T large enough that G's pieces do not hold the vocabulary."""
    t, v, d, dt = 16000, 24001, 64, torch.bfloat16
    h, w, target, _ = ce_problem(t, v, d, 0, dt, 3)
    _, lse = forward(tg, h, w, target, dt)
    dloss = torch.full((t,), 1.0 / t, device="cuda")
    dh, dw = backward(tg, h, w, target, lse, dloss, dt)
    wh, ww, bh, bw = ref.linear_ce_grad(h, w, target, lse, dloss)
    ref.assert_within(dh, wh, bh, "dh")
    ref.assert_within(dw, ww, bw, "dw")


@pytest.mark.parametrize("t", [40, 300])
def test_ignored_tokens_may_hold_anything(tg, t):
    v, d, dt = 700, 96, torch.float16
    h, w, target, _ = ce_problem(t, v, d, 0, dt, 9, ignored=0.5)
    out = (target < 0) | (target >= v)
    _, lse = ref.linear_ce(h, w, target)
    lse, dloss = lse.float(), torch.full((t,), 0.5, device="cuda")
    want = backward(tg, h, w, target, lse, dloss, dt)
    dirty = h.clone()
    dirty[out] = torch.tensor([float("nan"), float("inf"), -65504.0], dtype=dt, device="cuda").repeat(d // 3)
    dirty_lse = torch.where(out, torch.full_like(lse, float("nan")), lse)
    dirty_up = torch.where(out, torch.full_like(lse, float("inf")), dloss)
    got = backward(tg, dirty, w, target, dirty_lse, dirty_up, dt)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0][out] == 0).all()
    loss, lse2 = forward(tg, dirty, w, target, dt)
    ref.assert_within(lse2[~out], lse[~out], 1e-4, "lse beside dirty rows")
    assert (loss[out] == 0).all()


@pytest.mark.parametrize("t", [5, 200])
def test_no_token_counts(tg, t):
    v, d, dt = 600, 80, torch.bfloat16
    h, w, target, _ = ce_problem(t, v, d, 0, dt, 11)
    target = torch.full_like(target, -1)
    loss, lse = forward(tg, h, w, target, dt)
    assert (loss == 0).all()
    dh, dw = backward(tg, h, w, target, lse, torch.ones(t, device="cuda"), dt)
    assert (dh == 0).all() and (dw == 0).all()


def test_large_logits(tg):
    """Logits of several hundred, the target's far below the largest; and one
    token whose softmax is a single one."""
    t, v, d, dt = 64, 900, 128, torch.bfloat16
    h, w, target, _ = ce_problem(t, v, d, 0, dt, 13, ignored=0.0)
    h = (h * 60).to(dt)
    loss, lse = forward(tg, h, w, target, dt)
    want_loss, want = ref.linear_ce(h, w, target)
    bound = ref.lse_bound(h, w, want)
    assert float(want.max()) > 200
    ref.assert_within(lse, want, bound, "lse")
    ref.assert_within(loss, want_loss, 2 * bound, "loss")
    dloss = torch.ones(t, device="cuda")
    dh, dw = backward(tg, h, w, target, lse, dloss, dt)
    wh, ww, bh, bw = ref.linear_ce_grad(h, w, target, lse, dloss)
    ref.assert_within(dh, wh, bh, "dh")
    ref.assert_within(dw, ww, bw, "dw")


def test_targets_that_do_not_fit_32_bits(tg):
    t, v, d, dt = 8, 500, 64, torch.float16
    h, w, target, _ = ce_problem(t, v, d, 0, dt, 15, ignored=0.0)
    wild = target.clone()
    wild[0], wild[1], wild[2], wild[3] = 2**32, -2**63, 2**63 - 1, 2**32 + int(target[3])
    plain = target.clone()
    plain[:4] = -1
    assert torch.equal(forward(tg, h, w, wild, dt)[0], forward(tg, h, w, plain, dt)[0])
    lse, up = forward(tg, h, w, plain, dt)[1], torch.ones(t, device="cuda")
    a, b = backward(tg, h, w, wild, lse, up, dt), backward(tg, h, w, plain, lse, up, dt)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_linear_ce_grad_against_differences(tg):
    """<dH, U> against central differences of the library's own loss.  H and U
    are multiples of 2^-6, so that H +- hU are fp16 values."""
    t, v, d, dt, h_ = 40, 300, 64, torch.float16, 2.0**-4
    g = gen(17)
    h = (torch.randint(-64, 65, (t, d), generator=g, device="cuda") / 64).to(dt)
    u = (torch.randint(-4, 5, (t, d), generator=g, device="cuda") / 4).to(dt)
    w = ref.rows(g, v, d, 0, dt, 0.1)
    target = torch.randint(0, v, (t,), device="cuda", generator=g)
    dloss = torch.rand(t, device="cuda", generator=g)
    loss = lambda x: forward(tg, x, w, target, dt)[0].double()  # noqa: E731
    lse = forward(tg, h, w, target, dt)[1]
    dh, _ = backward(tg, h, w, target, lse, dloss, dt)
    up, down = (h + h_ * u).to(dt), (h - h_ * u).to(dt)
    assert torch.equal(up.double() - h.double(), h_ * u.double())
    diff = float(((loss(up) - loss(down)) * dloss.double()).sum()) / (2 * h_)
    # each token's third derivative along u is a third central moment of the
    # logits' changes, at most the cube of their range; times h^2 / 6
    change = u.double() @ w.double().T
    spread = (change.amax(1) - change.amin(1)) ** 3
    room = h_**2 / 6 * float((spread * dloss.double()).sum())
    room += float((2 * ref.lse_bound(up, w, lse.double()) * dloss.double()).sum()) / h_
    room += float((ref.linear_ce_grad(h, w, target, lse, dloss)[2] * u.double().abs()).sum())
    assert abs(float((dh.double() * u.double()).sum()) - diff) <= room


def test_linear_ce_on_another_stream_and_in_a_graph(tg):
    t, v, d, dt = 130, 1500, 128, torch.bfloat16
    h, w, target, _ = ce_problem(t, v, d, 0, dt, 19)
    loss, lse = forward(tg, h, w, target, dt)
    dloss = torch.full((t,), 1.0 / t, device="cuda")
    want = backward(tg, h, w, target, lse, dloss, dt)
    c = code(tg, dt)
    size = max(tg.tg_linear_ce_workspace_size(t, v, d, h, d, w, d, c),
               tg.tg_linear_ce_grad_workspace_size(t, v, d, h, d, w, d, h, d, w, d, c))
    ws, out = workspace(size), torch.zeros(2, t, device="cuda")
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    stream = torch.cuda.Stream()

    def both():
        s = torch.cuda.current_stream()
        tg.linear_ce(t, v, d, h, d, w, d, target, out[0], out[1], c, ws, size, s)
        tg.linear_ce_grad(t, v, d, h, d, w, d, target, out[1], dloss, dh, d, dw, d, c, ws, size, s)

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both()
    ok(tg)
    assert torch.equal(out[0], loss) and torch.equal(dh, want[0]) and torch.equal(dw, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        both()
    for x in (out, dh, dw):
        x.zero_()
    graph.replay()
    ok(tg)
    assert torch.equal(out[0], loss) and torch.equal(dh, want[0]) and torch.equal(dw, want[1])


# ------------------------------------------------------------------ AdamW

HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.1, step=3)
SIZES = [1, 7, 255, 256, 257, 0, 2047, 2048, 2049, 100003]


def adam_state(sizes, pt, gt, seed, offset=0):
    g = gen(seed)
    draw = lambda n, s, dt: (torch.randn(n + offset, generator=g, device="cuda") * s).to(dt)[offset:]  # noqa: E731
    return dict(p=[draw(n, 0.05, pt) for n in sizes], g=[draw(n, 0.01, gt) for n in sizes],
                m=[draw(n, 0.003, torch.float32) for n in sizes],
                v=[draw(n, 0.01, torch.float32).square() for n in sizes],
                master=[draw(n, 0.05, torch.float32) if pt != torch.float32 else None for n in sizes])


def adam_bounds(w, m, v, move, g, m0, v0, b1, b2):
    """Of the fp32 roundings: two products and a sum for m and v; m, root,
    product, sum, quotient, product for the step; product and difference."""
    bm = 3 * ref.EPS32 * (b1 * m0.double().abs() + (1 - b1) * g.double().abs()) * 1.01
    bv = 4 * ref.EPS32 * v * 1.01
    bw = 3 * ref.EPS32 * (w.abs() + move.abs()) + move.abs() * 10 * ref.EPS32
    rel = torch.where(m != 0, bm / m.abs().clamp(min=1e-300), torch.zeros_like(m))
    return bw + move.abs() * rel, bm, bv


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("pt,gt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                   (torch.float16, torch.float16), (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.float32)])
def test_adamw_32(tg, pt, gt, offset):
    s = adam_state(SIZES, pt, gt, 21, offset)
    before = {k: [x.clone() if x is not None else None for x in v] for k, v in s.items()}
    scale = torch.tensor(0.25, device="cuda")
    tensors = tg.make_adamw_tensors(s["p"], s["g"], s["m"], s["v"], master=s["master"])
    tg.adamw(tensors, tg.make_adamw_options(**HYPER, dtype=code(tg, pt), grad_dtype=code(tg, gt),
                                            grad_scale=scale))
    torch.cuda.synchronize()
    for i in range(len(SIZES)):
        w0 = before["master"][i] if pt != torch.float32 else before["p"][i]
        g = before["g"][i].float() * 0.25
        w, m, v, move = ref.adamw(w0, g, before["m"][i], before["v"][i], HYPER["lr"], 0.9, 0.999, 1e-8, 0.1, 3)
        bw, bm, bv = adam_bounds(w, m, v, move, g, before["m"][i], before["v"][i], 0.9, 0.999)
        ref.assert_within(s["m"][i], m, bm, "m")
        ref.assert_within(s["v"][i], v, bv + 2.0**-149, "v")
        if pt == torch.float32:
            ref.assert_within(s["p"][i], w, bw, "p")
        else:
            ref.assert_within(s["master"][i], w, bw, "master")
            assert torch.equal(s["p"][i], s["master"][i].to(pt))


def test_adamw_without_a_master_copy(tg):
    s = adam_state([1000], torch.bfloat16, torch.bfloat16, 23)
    p0 = s["p"][0].clone()
    m0, v0 = s["m"][0].clone(), s["v"][0].clone()
    tg.adamw(tg.make_adamw_tensors(s["p"], s["g"], s["m"], s["v"]),
             tg.make_adamw_options(**HYPER, dtype=tg.TG_BF16))
    torch.cuda.synchronize()
    w, m, v, move = ref.adamw(p0, s["g"][0], m0, v0, HYPER["lr"], 0.9, 0.999, 1e-8, 0.1, 3)
    bw = adam_bounds(w, m, v, move, s["g"][0], m0, v0, 0.9, 0.999)[0]
    ref.assert_within(s["p"][0], w, bw + ref.HALF_ULP[torch.bfloat16] * 1.01 * w.abs(), "p")


def blocks(x):
    return torch.nn.functional.pad(x.double(), (0, -x.numel() % 256)).view(-1, 256)


def decode(c, scale):
    return (blocks(c.view(torch.float8_e4m3fn).float()) * scale.double()[:, None]).view(-1)[:c.numel()]


def spacing(q):
    """e4m3's step at magnitude q."""
    e = torch.floor(torch.log2(q.clamp(min=2.0**-6)))
    return 2.0 ** (e - 3)


@pytest.mark.parametrize("offset", [0, 3])
@pytest.mark.parametrize("pt", [torch.float16, torch.bfloat16, torch.float32])
def test_adamw_8(tg, pt, offset):
    g = gen(25)
    s = adam_state(SIZES, pt, pt, 25)
    codes = lambda n, lo, hi: torch.randint(lo, hi, (n + offset,), generator=g, device="cuda",  # noqa: E731
                                            dtype=torch.uint8)[offset:]
    s["m"] = [codes(n, 0, 0x7F) | (codes(n, 0, 2) << 7) for n in SIZES]  # every code but NaN
    s["v"] = [codes(n, 0, 0x7F) for n in SIZES]
    nb = [(n + 255) // 256 for n in SIZES]
    s["ms"] = [torch.rand(b, generator=g, device="cuda") * 1e-4 for b in nb]
    s["vs"] = [torch.rand(b, generator=g, device="cuda") * 1e-4 for b in nb]
    before = {k: [x.clone() if x is not None else None for x in v] for k, v in s.items()}
    tensors = tg.make_adamw_tensors(s["p"], s["g"], s["m"], s["v"], master=s["master"], m_scale=s["ms"],
                                    v_scale=s["vs"])
    tg.adamw(tensors, tg.make_adamw_options(**HYPER, dtype=code(tg, pt), state_bits=8, seed=99))
    torch.cuda.synchronize()
    for i, n in enumerate(SIZES):
        if n == 0:
            continue
        w0 = before["master"][i] if pt != torch.float32 else before["p"][i]
        m0, r0 = decode(before["m"][i], before["ms"][i]), decode(before["v"][i], before["vs"][i])
        v0 = r0.float().square()
        gr = before["g"][i].float()
        w, m, v, move = ref.adamw(w0, gr, m0, v0, HYPER["lr"], 0.9, 0.999, 1e-8, 0.1, 3)
        bw, bm, bv = adam_bounds(w, m, v, move, gr, m0, v0, 0.9, 0.999)
        ref.assert_within(s["p"][i] if pt == torch.float32 else s["master"][i], w, bw * 2, "p")
        r = v.sqrt()
        for got, want, scale, half in ((s["m"][i], m, s["ms"][i], 0.5), (s["v"][i], r, s["vs"][i], 1.0)):
            top = blocks(want.abs()).amax(1)
            ref.assert_within(scale, top / 448, top / 448 * 8 * ref.EPS32, "scale")
            of = (torch.arange(n, device="cuda") // 256)
            q = want.abs() / (top[of] / 448)
            room = spacing(q * (1 + 1e-6)) * (half + 1e-4) + q * 1e-5
            ref.assert_within(decode(got, scale), want, room * scale.double()[of], "state")
        kept = decode(s["v"][i], s["vs"][i])
        assert (kept[r > 0] > 0).all()


def test_adamw_8_rounds_the_root_without_bias(tg):
    """65536 equal roots halfway up and an eighth up an e4m3 step, beside the
    block's largest: their mean is theirs, within five standard errors."""
    n = 65536
    for at in (1.0 + 1 / 16, 1.0 + 1 / 64, 2.0**-8 * 1.25):
        r = torch.full((n,), at, device="cuda")
        r[::256] = 448.0
        v = r.square()
        st = dict(p=torch.zeros(n, device="cuda"), g=torch.zeros(n, device="cuda"),
                  m=torch.zeros(n, dtype=torch.uint8, device="cuda"))
        # beta2 = 0 and g = r make v = r^2
        st["g"].copy_(r)
        c = torch.zeros(n, dtype=torch.uint8, device="cuda")
        ms, vs = torch.ones(n // 256, device="cuda"), torch.ones(n // 256, device="cuda")
        tg.adamw(tg.make_adamw_tensors([st["p"]], [st["g"]], [st["m"]], [c], m_scale=[ms], v_scale=[vs]),
                 tg.make_adamw_options(1e-3, 0.9, 0.0, 1e-8, 0.0, 1, dtype=tg.TG_F32, state_bits=8, seed=4))
        torch.cuda.synchronize()
        got = decode(c, vs)[r != 448]
        step = float(spacing(torch.tensor(at)))
        frac = (at / step) % 1
        sigma = step * math.sqrt(frac * (1 - frac) / got.numel())
        assert abs(float(got.mean()) - at) <= 5 * sigma + at * 1e-6
        assert set(torch.unique((got / step).round()).tolist()) <= {math.floor(at / step), math.floor(at / step) + 1}
    assert float(v.max()) > 0


def test_adamw_8_lets_v_decay(tg):
    """200 steps without a gradient: sqrt(v) falls by 0.999^100."""
    n = 1 << 16
    c = torch.full((n,), 0x60, dtype=torch.uint8, device="cuda")  # 32
    c[::256] = 0x7E                                              # 448
    m = torch.zeros(n, dtype=torch.uint8, device="cuda")
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    ms, vs = torch.zeros(n // 256, device="cuda"), torch.ones(n // 256, device="cuda")
    t = tg.make_adamw_tensors([p], [g], [m], [c], m_scale=[ms], v_scale=[vs])
    g[::256] = 0.0
    for step in range(200):
        tg.adamw(t, tg.make_adamw_options(1e-3, 0.9, 0.999, 1e-8, 0.0, step + 1, dtype=tg.TG_F32, state_bits=8,
                                          seed=step))
    torch.cuda.synchronize()
    r = decode(c, vs)[(torch.arange(n, device="cuda") % 256) != 0]
    want = 32 * 0.999 ** 100
    # a step's rounding has a standard deviation of at most half an e4m3 step
    # (2 to 4 here, of 32): 200 of them, over 65280 elements, five times
    assert abs(float(r.mean()) - want) <= 5 * 2 * math.sqrt(200 / r.numel()) + 0.01 * want
    assert (p == 0).all() and (decode(m, ms) == 0).all()


def test_adamw_many_tensors(tg):
    """More tensors than one launch takes."""
    sizes = [1 + 37 * (k % 11) for k in range(600)]
    s = adam_state(sizes, torch.float32, torch.float32, 29)
    p0 = [x.clone() for x in s["p"]]
    m0, v0 = [x.clone() for x in s["m"]], [x.clone() for x in s["v"]]
    tg.adamw(tg.make_adamw_tensors(s["p"], s["g"], s["m"], s["v"]),
             tg.make_adamw_options(**HYPER, dtype=tg.TG_F32))
    torch.cuda.synchronize()
    cat = torch.cat
    w, m, v, move = ref.adamw(cat(p0), cat(s["g"]), cat(m0), cat(v0), HYPER["lr"], 0.9, 0.999, 1e-8, 0.1, 3)
    bw, bm, bv = adam_bounds(w, m, v, move, cat(s["g"]), cat(m0), cat(v0), 0.9, 0.999)
    ref.assert_within(cat(s["p"]), w, bw, "p")
    ref.assert_within(cat(s["m"]), m, bm, "m")


def test_adamw_non_finite_gradients_stay_where_they_are(tg):
    n = 1024
    for bits in (32, 8):
        p = torch.ones(n, device="cuda")
        g = torch.ones(n, device="cuda") * 0.1
        g[300] = float("nan")
        g[700] = float("inf")
        dt = torch.float32 if bits == 32 else torch.uint8
        m, v = torch.zeros(n, dtype=dt, device="cuda"), torch.zeros(n, dtype=dt, device="cuda")
        ms, vs = torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda")
        tg.adamw(tg.make_adamw_tensors([p], [g], [m], [v], m_scale=[ms], v_scale=[vs]),
                 tg.make_adamw_options(**HYPER, dtype=tg.TG_F32, state_bits=bits))
        torch.cuda.synchronize()
        bad = p.isnan().nonzero()[:, 0].tolist()
        assert bad == [300, 700]  # inf / inf is not a number either
        if bits == 8:
            assert ms[0].isfinite() and ms[3].isfinite() and not ms[1].isfinite()
