"""Refusals of the output head's calls without a GPU: every argument check
fires before any device work (fake, never-dereferenced pointers)."""
import pytest

G = 1 << 30
FAKE = 1 << 44
F16, BF16, F32 = 0, 1, 2


def at(k):
    return FAKE + k * 64 * G


def no_device():
    import torch
    return not torch.cuda.is_available()


def status(tg, rc):
    return tg.tg_status_string(rc)


def ln(tg, rows=8, cols=64, X=at(0), ldx=None, weight=at(1), bias=at(2), eps=1e-5, Y=at(3), ldy=None,
       mean=at(4), rstd=at(5), dtype=F16):
    return tg.tg_layernorm(rows, cols, X, cols if ldx is None else ldx, weight, bias, eps, Y,
                           cols if ldy is None else ldy, mean, rstd, dtype)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), "TG_ERR_INVALID_ARG"), (dict(cols=-1), "TG_ERR_INVALID_ARG"),
    (dict(rows=1 << 31), "TG_ERR_INVALID_ARG"), (dict(X=None), "TG_ERR_INVALID_ARG"),
    (dict(weight=None), "TG_ERR_INVALID_ARG"), (dict(Y=None), "TG_ERR_INVALID_ARG"),
    (dict(mean=None), "TG_ERR_INVALID_ARG"), (dict(rstd=None), "TG_ERR_INVALID_ARG"),
    (dict(eps=-1.0), "TG_ERR_INVALID_ARG"), (dict(eps=float("nan")), "TG_ERR_INVALID_ARG"),
    (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(dtype=7), "TG_ERR_DTYPE"),
    (dict(ldx=63), "TG_ERR_STRIDE"), (dict(ldy=0), "TG_ERR_STRIDE"), (dict(ldx=1 << 40), "TG_ERR_STRIDE"),
    (dict(X=at(0) + 1), "TG_ERR_ALIGN"), (dict(mean=at(4) + 2), "TG_ERR_ALIGN"),
    (dict(Y=at(0) + 8 * 64 * 2 - 2), "TG_ERR_OVERLAP"), (dict(rstd=at(4) + 28), "TG_ERR_OVERLAP"),
    (dict(Y=at(2) - 8 * 64 * 2 + 2), "TG_ERR_OVERLAP"),
])
def test_layernorm_refusals(tg, kw, code):
    assert status(tg, ln(tg, **kw)) == code


def ln_grad(tg, rows=8, cols=64, dY=at(0), lddy=64, X=at(1), ldx=64, weight=at(2), mean=at(3), rstd=at(4),
            dX=at(5), lddx=64, dweight=at(6), dbias=at(7), dtype=BF16, ws=at(8), size=1 << 30):
    return tg.tg_layernorm_grad(rows, cols, dY, lddy, X, ldx, weight, mean, rstd, dX, lddx, dweight, dbias,
                                dtype, ws, size)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "TG_ERR_INVALID_ARG"), (dict(cols=0), "TG_ERR_INVALID_ARG"),
    (dict(dY=None), "TG_ERR_INVALID_ARG"), (dict(dX=None), "TG_ERR_INVALID_ARG"),
    (dict(dweight=None), "TG_ERR_INVALID_ARG"), (dict(ws=None), "TG_ERR_INVALID_ARG"),
    (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(lddx=60), "TG_ERR_STRIDE"), (dict(lddy=63), "TG_ERR_STRIDE"),
    (dict(dX=at(5) + 1), "TG_ERR_ALIGN"), (dict(ws=at(8) + 128), "TG_ERR_ALIGN"),
    (dict(dX=at(0)), "TG_ERR_OVERLAP"), (dict(dweight=at(2)), "TG_ERR_OVERLAP"),
    (dict(dbias=at(6) + 100), "TG_ERR_OVERLAP"),
])
def test_layernorm_grad_refusals(tg, kw, code):
    assert status(tg, ln_grad(tg, **kw)) == code


def ce(tg, T=8, V=100, D=64, H=at(0), ldh=64, W=at(1), ldw=64, target=at(2), loss=at(3), lse=at(4), dtype=F16,
       ws=at(5), size=1 << 30):
    return tg.tg_linear_ce(T, V, D, H, ldh, W, ldw, target, loss, lse, dtype, ws, size)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), "TG_ERR_INVALID_ARG"), (dict(V=0), "TG_ERR_INVALID_ARG"), (dict(D=1 << 31), "TG_ERR_INVALID_ARG"),
    (dict(T=(1 << 31) - 1, V=(1 << 31) - 1, D=1, ldh=1, ldw=1), "TG_ERR_INVALID_ARG"),  # more tiles than 32 bits
    (dict(H=None), "TG_ERR_INVALID_ARG"), (dict(target=None), "TG_ERR_INVALID_ARG"),
    (dict(lse=None), "TG_ERR_INVALID_ARG"), (dict(ws=None), "TG_ERR_INVALID_ARG"),
    (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(ldh=63), "TG_ERR_STRIDE"), (dict(ldw=-1), "TG_ERR_STRIDE"),
    (dict(H=at(0) + 1), "TG_ERR_ALIGN"), (dict(target=at(2) + 4), "TG_ERR_ALIGN"),
    (dict(loss=at(3) + 2), "TG_ERR_ALIGN"), (dict(ws=at(5) + 16), "TG_ERR_ALIGN"),
    (dict(size=16), "TG_ERR_BUFFER"), (dict(loss=at(4) + 16), "TG_ERR_OVERLAP"),
    (dict(lse=at(2) + 32), "TG_ERR_OVERLAP"), (dict(ws=at(1)), "TG_ERR_OVERLAP"),
])
def test_linear_ce_refusals(tg, kw, code):
    assert status(tg, ce(tg, **kw)) == code


def ce_grad(tg, T=8, V=100, D=64, H=at(0), ldh=64, W=at(1), ldw=64, target=at(2), lse=at(3), dloss=at(4),
            dH=at(5), lddh=64, dW=at(6), lddw=64, dtype=F16, ws=at(7), size=1 << 30):
    return tg.tg_linear_ce_grad(T, V, D, H, ldh, W, ldw, target, lse, dloss, dH, lddh, dW, lddw, dtype, ws, size)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-5), "TG_ERR_INVALID_ARG"), (dict(dH=None, dW=None), "TG_ERR_INVALID_ARG"),
    (dict(lse=None), "TG_ERR_INVALID_ARG"), (dict(dloss=None), "TG_ERR_INVALID_ARG"),
    (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(lddh=63), "TG_ERR_STRIDE"), (dict(lddw=8), "TG_ERR_STRIDE"),
    (dict(dW=at(6) + 1), "TG_ERR_ALIGN"), (dict(dloss=at(4) + 1), "TG_ERR_ALIGN"),
    (dict(dH=at(0)), "TG_ERR_OVERLAP"), (dict(dW=at(1) + 128), "TG_ERR_OVERLAP"),
    (dict(dH=at(6)), "TG_ERR_OVERLAP"),
])
def test_linear_ce_grad_refusals(tg, kw, code):
    assert status(tg, ce_grad(tg, **kw)) == code


def adam(tg, n=1000, p=at(0), g=at(1), m=at(2), v=at(3), master=at(4), ms=at(5), vs=at(6), dtype=BF16,
         grad_dtype=None, bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, more=(), grad_scale=None):
    rows = [(p, g, m, v, master, ms, vs, n)] + list(more)
    cols = list(zip(*rows))
    t = tg.make_adamw_tensors(cols[0], cols[1], cols[2], cols[3], master=cols[4], m_scale=cols[5],
                              v_scale=cols[6], numel=cols[7])
    return tg.tg_adamw(t, tg.make_adamw_options(lr, b1, b2, eps, wd, step, dtype, grad_dtype, bits, 0, grad_scale))


@pytest.mark.parametrize("kw,code", [
    (dict(p=None), "TG_ERR_INVALID_ARG"), (dict(g=None), "TG_ERR_INVALID_ARG"),
    (dict(v=None), "TG_ERR_INVALID_ARG"), (dict(bits=8, ms=None), "TG_ERR_INVALID_ARG"),
    (dict(n=-1), "TG_ERR_INVALID_ARG"), (dict(step=0), "TG_ERR_INVALID_ARG"), (dict(b1=1.0), "TG_ERR_INVALID_ARG"),
    (dict(b2=-0.1), "TG_ERR_INVALID_ARG"), (dict(eps=-1.0), "TG_ERR_INVALID_ARG"),
    (dict(lr=float("inf")), "TG_ERR_INVALID_ARG"), (dict(bits=16), "TG_ERR_INVALID_ARG"),
    (dict(dtype=F32), "TG_ERR_INVALID_ARG"),           # a master copy of an fp32 parameter
    (dict(dtype=3), "TG_ERR_DTYPE"), (dict(dtype=BF16, grad_dtype=F16), "TG_ERR_DTYPE"),
    (dict(dtype=F32, grad_dtype=BF16, master=None), "TG_ERR_DTYPE"),
    (dict(p=at(0) + 1), "TG_ERR_ALIGN"), (dict(m=at(2) + 2), "TG_ERR_ALIGN"), (dict(master=at(4) + 2), "TG_ERR_ALIGN"),
    (dict(grad_scale=at(7) + 2), "TG_ERR_ALIGN"),
    (dict(g=at(0)), "TG_ERR_OVERLAP"), (dict(v=at(2) + 3996), "TG_ERR_OVERLAP"),
    (dict(bits=8, vs=at(5) + 12), "TG_ERR_OVERLAP"),
    # one tensor's state is another's parameter
    (dict(more=[(at(10), at(11), at(12), at(0) + 1000, at(14), None, None, 50)]), "TG_ERR_OVERLAP"),
    # one tensor's gradient is written as another's state
    (dict(more=[(at(10), at(3), at(12), at(13), at(14), None, None, 50)]), "TG_ERR_OVERLAP"),
])
def test_adamw_refusals(tg, kw, code):
    assert status(tg, adam(tg, **kw)) == code


def test_valid_arguments_reach_the_device_check(tg):
    if not no_device():
        pytest.skip("device present: covered by the GPU tests")
    want = tg.TG_ERR_UNSUPPORTED_DEVICE
    assert ln(tg) == want and ln(tg, bias=None) == want and ln(tg, X=at(0) + 2, ldx=65) == want
    assert ln_grad(tg) == want and ln_grad(tg, dbias=None) == want
    assert ce(tg) == want and ce_grad(tg) == want
    assert ce_grad(tg, dH=None) == want and ce_grad(tg, dW=None) == want
    assert adam(tg) == want and adam(tg, bits=8) == want and adam(tg, grad_dtype=F32) == want
    # two tensors may share a gradient, and adjacent operands do not overlap
    assert adam(tg, more=[(at(10), at(1), at(12), at(13), at(14), None, None, 50)]) == want
    assert adam(tg, v=at(2) + 4000) == want
    # nothing to do needs no device
    assert adam(tg, n=0, p=None, g=None, m=None, v=None, master=None) == tg.TG_OK


def test_workspace_sizes(tg):
    c = [tg.tg_linear_ce_workspace_size(8, 1000, 64, at(0), 64, at(1), 64, F16)]
    c.append(tg.tg_linear_ce_workspace_size(8, 1000, 64, at(0) + 2, 64, at(1), 64, F16))
    c.append(tg.tg_linear_ce_workspace_size(8, 1000, 64, at(0) + 2, 64, at(1), 65, F16))
    assert c[0] < c[1] < c[2] and c[2] >= 1000 * 64 * 2
    with pytest.raises(tg.TileGemmError) as e:
        tg.tg_linear_ce_workspace_size(8, 0, 64, at(0), 64, at(1), 64, F16)
    assert e.value.status == tg.TG_ERR_INVALID_ARG
    with pytest.raises(tg.TileGemmError) as e:
        tg.tg_layernorm_grad_workspace_size(8, 64, F32)
    assert e.value.status == tg.TG_ERR_DTYPE
    with pytest.raises(tg.TileGemmError) as e:
        tg.make_adamw_tensors([1, 2], [1], [1], [1], numel=[3, 4])
    assert e.value.status == tg.TG_ERR_INVALID_ARG
