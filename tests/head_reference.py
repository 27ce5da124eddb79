"""Plain 64-bit forms of the output head's operators and the error bounds that
follow from what the library rounds (test infrastructure, torch float64)."""
import torch

EPS32 = 2.0**-24                                   # half an ulp of 1 in fp32
# largest relative error of rounding to nearest: half the distance of 1 to the next value
HALF_ULP = {torch.float16: 2.0**-11, torch.bfloat16: 2.0**-8}
TINY = {torch.float16: 2.0**-25, torch.bfloat16: 2.0**-134}  # half the smallest subnormal


def assert_within(got, want, bound, what):
    """|got - want| <= bound everywhere, NaN where NaN is wanted."""
    got, want = got.double(), want.double()
    bad = ~((got - want).abs() <= bound) & ~(got.isnan() & want.isnan()) & ~(got == want)
    if bad.any():
        i = tuple(int(k) for k in bad.nonzero()[0])
        b = torch.as_tensor(bound, device=got.device).expand_as(got)[i]
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: got "
                             f"{float(got[i])!r}, want {float(want[i])!r} +- {float(b):.3g}")


def rows(gen, n, d, pad, dtype, scale=1.0):
    """n x d view of a buffer with rows of d + pad elements (padding is NaN)."""
    full = torch.full((n, d + pad), float("nan"), dtype=dtype, device="cuda")
    full[:, :d] = (torch.randn(n, d, generator=gen, device="cuda") * scale).to(dtype)
    return full[:, :d]


# ------------------------------------------------------------- layer norm

def layernorm(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (x - mean) * rstd * w.double() + (b.double() if b is not None else 0.0)
    return y, mean[:, 0], rstd[:, 0]


def layernorm_grad(dy, x, w, mean, rstd):
    dy, x, w = dy.double(), x.double(), w.double()
    rstd = rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * rstd
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


# --------------------------------------------------- linear cross entropy

def linear_ce(h, w, target):
    logits = h.double() @ w.double().T
    lse = torch.logsumexp(logits, 1)
    v = w.shape[0]
    ok = (target >= 0) & (target < v)
    hit = logits.gather(1, target.clamp(0, v - 1)[:, None])[:, 0]
    return torch.where(ok, lse - hit, torch.zeros_like(lse)), lse


def logit_bound(h, w):
    """Products of 16-bit values are exact in fp32; the tensor core adds them
    16 at a time, each addition off by at most 2^-23 of the largest partial
    sum, which sum |h||w| bounds."""
    d = h.shape[1]
    largest = (h.double().abs() @ w.double().abs().T).amax(1)
    return (d / 16 + 2) * 2 * EPS32 * largest


def lse_bound(h, w, lse):
    """Of the logits, of 2^x (2^-22 relative, and the argument's rounding), of
    the sums (64 additions per tile, one per tile and the joins) and of the
    result's own roundings."""
    tiles = w.shape[0] / 128 + 1
    return logit_bound(h, w) + 2.0**-21 + (96 + tiles) * EPS32 + 8 * EPS32 * (1 + lse.abs())


def linear_ce_grad(h, w, target, lse, dloss):
    """dH, dW and their elementwise bounds for the library's rounding of G."""
    dt = h.dtype
    u, v, t = HALF_ULP[dt], w.shape[0], h.shape[0]
    ok = (target >= 0) & (target < v)
    hh = torch.where(ok[:, None], h.double(), torch.zeros((), device=h.device, dtype=torch.float64))
    ww = w.double()
    up = torch.where(ok, dloss.double(), torch.zeros_like(dloss, dtype=torch.float64))
    p = torch.exp(hh @ ww.T - torch.where(ok, lse.double(), torch.zeros_like(lse, dtype=torch.float64))[:, None])
    g = p * up[:, None]
    # of exp's argument and of its result, relative to p
    slack = logit_bound(hh, ww)[:, None] + 16 * EPS32 * (1 + lse.nan_to_num().abs().max().double()) + 2.0**-20
    off = g.abs() * slack
    rows_ = torch.arange(t, device=h.device)
    g[rows_, target.clamp(0, v - 1)] -= up
    # G rounded to 16 bits: scaled so that its largest possible entry is 1 or 1024
    floor = float(up.abs().max()) * (2.0**-25 / 1024 if dt == torch.float16 else 2.0**-134)
    off = off + u * g.abs() * 1.01 + floor
    dh, dw = g @ ww, g.T @ hh
    acc = 2 * EPS32
    bh = off @ ww.abs() + (v / 16 + 8) * acc * (g.abs() @ ww.abs()) + 1.01 * u * dh.abs() + TINY[dt]
    bw = off.T @ hh.abs() + (t / 16 + 8) * acc * (g.abs().T @ hh.abs()) + 1.01 * u * dw.abs() + TINY[dt]
    return dh, dw, bh, bw


# ------------------------------------------------------------------ AdamW

def adamw(p, g, m, v, lr, b1, b2, eps, wd, step, scale=1.0):
    g = g.double() * scale
    m = b1 * m.double() + (1 - b1) * g
    v = b2 * v.double() + (1 - b2) * g * g
    move = lr / (1 - b1**step) * m / ((v / (1 - b2**step)).sqrt() + eps)
    return p.double() * (1 - lr * wd) - move, m, v, move
