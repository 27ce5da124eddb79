"""Refusals of routing, grouping, grouped products, combining and adapters without
a GPU: every argument check fires before any device work (fake, never-
dereferenced pointers)."""
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


def options(tg, k=2, score=0, groups=1, kept=1, top=1, renorm=0, scale=1.0):
    o = tg.make_route_options(k, score, groups, kept, top, False, scale)
    o.renormalise = renorm
    return o


BAD_OPTIONS = [dict(k=0), dict(k=33), dict(k=5, groups=4, kept=2), dict(score=2), dict(score=-1), dict(groups=0),
               dict(groups=33), dict(groups=3), dict(groups=4, kept=5), dict(kept=0), dict(top=0), dict(top=3),
               dict(renorm=2), dict(scale=float("inf")), dict(scale=float("nan"))]


def route(tg, T=4, E=8, logits=at(0), ld=None, bias=at(1), index=at(2), weight=at(3), dtype=BF16, opts=None, **kw):
    o = None if opts == "none" else options(tg, **kw)
    return tg.tg_route(T, E, logits, E if ld is None else ld, bias, index, weight, dtype, o)


@pytest.mark.parametrize("kw,code", [(k, "TG_ERR_INVALID_ARG") for k in BAD_OPTIONS] + [
    (dict(opts="none"), "TG_ERR_INVALID_ARG"), (dict(T=0), "TG_ERR_INVALID_ARG"), (dict(E=1025), "TG_ERR_INVALID_ARG"),
    (dict(E=0), "TG_ERR_INVALID_ARG"), (dict(k=9), "TG_ERR_INVALID_ARG"), (dict(T=1 << 31), "TG_ERR_INVALID_ARG"),
    (dict(logits=None), "TG_ERR_INVALID_ARG"), (dict(index=None), "TG_ERR_INVALID_ARG"),
    (dict(weight=None), "TG_ERR_INVALID_ARG"), (dict(dtype=3), "TG_ERR_DTYPE"), (dict(ld=7), "TG_ERR_STRIDE"),
    (dict(ld=1 << 41), "TG_ERR_STRIDE"), (dict(logits=at(0) + 1), "TG_ERR_ALIGN"),
    (dict(logits=at(0) + 2, dtype=F32), "TG_ERR_ALIGN"), (dict(bias=at(1) + 2), "TG_ERR_ALIGN"),
    (dict(index=at(2) + 2), "TG_ERR_ALIGN"), (dict(weight=at(3) + 1), "TG_ERR_ALIGN"),
    (dict(weight=at(2) + 28), "TG_ERR_OVERLAP"), (dict(index=at(0) + 60), "TG_ERR_OVERLAP"),
    (dict(weight=at(1) + 28), "TG_ERR_OVERLAP"),
])
def test_route_refusals(tg, kw, code):
    assert status(tg, route(tg, **kw)) == code


def route_grad(tg, T=4, E=8, logits=at(0), ld=8, index=at(1), dweight=at(2), dlogits=at(3), lddl=8, dtype=BF16,
               opts=None, **kw):
    o = None if opts == "none" else options(tg, **kw)
    return tg.tg_route_grad(T, E, logits, ld, index, dweight, dlogits, lddl, dtype, o)


@pytest.mark.parametrize("kw,code", [(k, "TG_ERR_INVALID_ARG") for k in BAD_OPTIONS] + [
    (dict(opts="none"), "TG_ERR_INVALID_ARG"), (dict(T=-1), "TG_ERR_INVALID_ARG"),
    (dict(index=None), "TG_ERR_INVALID_ARG"), (dict(dweight=None), "TG_ERR_INVALID_ARG"),
    (dict(dlogits=None), "TG_ERR_INVALID_ARG"), (dict(dtype=-1), "TG_ERR_DTYPE"), (dict(lddl=7), "TG_ERR_STRIDE"),
    (dict(ld=0), "TG_ERR_STRIDE"), (dict(dlogits=at(3) + 1), "TG_ERR_ALIGN"), (dict(dweight=at(2) + 2), "TG_ERR_ALIGN"),
    (dict(dlogits=at(0)), "TG_ERR_OVERLAP"), (dict(dlogits=at(2) + 16), "TG_ERR_OVERLAP"),
])
def test_route_grad_refusals(tg, kw, code):
    assert status(tg, route_grad(tg, **kw)) == code


def group_rows(tg, R=10, g=4, index=at(0), offset=at(1), row=at(2), place=at(3), ws=at(4), size=1 << 30):
    return tg.tg_group_rows(R, g, index, offset, row, place, ws, size)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), "TG_ERR_INVALID_ARG"), (dict(g=0), "TG_ERR_INVALID_ARG"), (dict(g=4097), "TG_ERR_INVALID_ARG"),
    (dict(R=(1 << 30) + 1), "TG_ERR_INVALID_ARG"), (dict(index=None), "TG_ERR_INVALID_ARG"),
    (dict(offset=None), "TG_ERR_INVALID_ARG"), (dict(row=None), "TG_ERR_INVALID_ARG"),
    (dict(R=5000, ws=None), "TG_ERR_INVALID_ARG"), (dict(R=5000, ws=at(4) + 64), "TG_ERR_ALIGN"),
    (dict(R=5000, size=47), "TG_ERR_BUFFER"), (dict(row=at(2) + 2), "TG_ERR_ALIGN"),
    (dict(place=at(2) + 36), "TG_ERR_OVERLAP"), (dict(offset=at(0) + 36), "TG_ERR_OVERLAP"),
    (dict(row=at(1) + 16), "TG_ERR_OVERLAP"), (dict(R=5000, ws=at(0)), "TG_ERR_OVERLAP"),
])
def test_group_rows_refusals(tg, kw, code):
    assert status(tg, group_rows(tg, **kw)) == code


def grouped(tg, R=100, N=64, K=32, g=4, X=at(0), x_rows=100, ldx=None, row=at(1), per_row=1, B=at(2), ldb=None, stride=None,
            perm=1, offset=at(3), Y=at(4), ldy=None, dtype=F16, bias=None, ld_bias=64, relu=0, relu_of=None, ld_relu=64):
    ldb = (K if perm == 1 else N) if ldb is None else ldb
    stride = N * K if stride is None else stride
    epi = tg.make_group_epilogue(bias, ld_bias, False, relu_of, ld_relu)
    epi.relu = relu
    return tg.tg_grouped_gemm(R, N, K, g, X, x_rows, K if ldx is None else ldx, row, per_row, B, ldb, stride, perm, offset, Y,
                              N if ldy is None else ldy, dtype, epi)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), "TG_ERR_INVALID_ARG"), (dict(N=-1), "TG_ERR_INVALID_ARG"), (dict(K=0), "TG_ERR_INVALID_ARG"),
    (dict(g=0), "TG_ERR_INVALID_ARG"), (dict(g=4097), "TG_ERR_INVALID_ARG"), (dict(x_rows=0), "TG_ERR_INVALID_ARG"),
    (dict(per_row=0), "TG_ERR_INVALID_ARG"), (dict(row=None, x_rows=99), "TG_ERR_INVALID_ARG"),
    (dict(perm=2), "TG_ERR_INVALID_ARG"), (dict(X=None), "TG_ERR_INVALID_ARG"), (dict(B=None), "TG_ERR_INVALID_ARG"),
    (dict(offset=None), "TG_ERR_INVALID_ARG"), (dict(Y=None), "TG_ERR_INVALID_ARG"), (dict(relu=2), "TG_ERR_INVALID_ARG"),
    (dict(R=1 << 30, x_rows=1 << 30, N=1 << 20, K=8), "TG_ERR_INVALID_ARG"),  # more tiles than 32 bits
    (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(ldx=24), "TG_ERR_STRIDE"), (dict(ldb=24), "TG_ERR_STRIDE"),
    (dict(perm=0, ldb=56), "TG_ERR_STRIDE"), (dict(ldy=56), "TG_ERR_STRIDE"), (dict(stride=64 * 32 - 8), "TG_ERR_STRIDE"),
    (dict(stride=-64 * 32), "TG_ERR_STRIDE"), (dict(bias=at(5), ld_bias=63), "TG_ERR_STRIDE"),
    (dict(relu_of=at(5), ld_relu=56), "TG_ERR_STRIDE"),
    (dict(X=at(0) + 8), "TG_ERR_ALIGN"), (dict(B=at(2) + 2), "TG_ERR_ALIGN"), (dict(Y=at(4) + 8), "TG_ERR_ALIGN"),
    (dict(ldx=33), "TG_ERR_ALIGN"), (dict(ldb=36, stride=64 * 36), "TG_ERR_ALIGN"), (dict(ldy=65), "TG_ERR_ALIGN"),
    (dict(stride=64 * 32 + 4), "TG_ERR_ALIGN"), (dict(row=at(1) + 2), "TG_ERR_ALIGN"), (dict(offset=at(3) + 1), "TG_ERR_ALIGN"),
    (dict(bias=at(5) + 1), "TG_ERR_ALIGN"), (dict(relu_of=at(5) + 2), "TG_ERR_ALIGN"),
    (dict(relu_of=at(5), ld_relu=68), "TG_ERR_ALIGN"),
    (dict(Y=at(0)), "TG_ERR_OVERLAP"), (dict(Y=at(2) + 16), "TG_ERR_OVERLAP"), (dict(relu_of=at(4)), "TG_ERR_OVERLAP"),
    (dict(bias=at(4) + 2), "TG_ERR_OVERLAP"), (dict(row=at(4) + 4), "TG_ERR_OVERLAP"),
])
def test_grouped_gemm_refusals(tg, kw, code):
    assert status(tg, grouped(tg, **kw)) == code


def grouped_grad(tg, R=100, N=64, K=32, g=4, dY=at(0), lddy=64, X=at(1), x_rows=100, ldx=32, row=at(2), per_row=1, offset=at(3),
                 dB=at(4), lddb=32, stride=64 * 32, perm=1, dtype=F16):
    return tg.tg_grouped_gemm_grad(R, N, K, g, dY, lddy, X, x_rows, ldx, row, per_row, offset, dB, lddb, stride, perm, dtype)


@pytest.mark.parametrize("kw,code", [
    (dict(R=0), "TG_ERR_INVALID_ARG"), (dict(g=5000), "TG_ERR_INVALID_ARG"), (dict(row=None, x_rows=10), "TG_ERR_INVALID_ARG"),
    (dict(dY=None), "TG_ERR_INVALID_ARG"), (dict(dB=None), "TG_ERR_INVALID_ARG"), (dict(dtype=7), "TG_ERR_DTYPE"),
    (dict(lddb=24), "TG_ERR_STRIDE"), (dict(perm=0), "TG_ERR_STRIDE"), (dict(stride=8), "TG_ERR_STRIDE"),
    (dict(lddy=68), "TG_ERR_ALIGN"), (dict(dB=at(4) + 4), "TG_ERR_ALIGN"), (dict(dB=at(0) + 64), "TG_ERR_OVERLAP"),
    (dict(dB=at(1)), "TG_ERR_OVERLAP"), (dict(offset=at(4) + 64), "TG_ERR_OVERLAP"),
])
def test_grouped_gemm_grad_refusals(tg, kw, code):
    assert status(tg, grouped_grad(tg, **kw)) == code


def combine(tg, T=4, k=2, D=64, Y=at(0), y_rows=8, ldy=64, place=at(1), weight=at(2), out=at(3), ldo=64, dtype=F16):
    return tg.tg_combine(T, k, D, Y, y_rows, ldy, place, weight, out, ldo, dtype)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), "TG_ERR_INVALID_ARG"), (dict(k=0), "TG_ERR_INVALID_ARG"), (dict(k=1025), "TG_ERR_INVALID_ARG"),
    (dict(T=1 << 30, k=2), "TG_ERR_INVALID_ARG"), (dict(D=0), "TG_ERR_INVALID_ARG"), (dict(y_rows=0), "TG_ERR_INVALID_ARG"),
    (dict(Y=None), "TG_ERR_INVALID_ARG"), (dict(place=None), "TG_ERR_INVALID_ARG"), (dict(out=None), "TG_ERR_INVALID_ARG"),
    (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(ldy=63), "TG_ERR_STRIDE"), (dict(ldo=1), "TG_ERR_STRIDE"),
    (dict(Y=at(0) + 1), "TG_ERR_ALIGN"), (dict(place=at(1) + 2), "TG_ERR_ALIGN"), (dict(weight=at(2) + 2), "TG_ERR_ALIGN"),
    (dict(out=at(0) + 512), "TG_ERR_OVERLAP"), (dict(out=at(1)), "TG_ERR_OVERLAP"), (dict(weight=at(3) + 4), "TG_ERR_OVERLAP"),
])
def test_combine_refusals(tg, kw, code):
    assert status(tg, combine(tg, **kw)) == code


def combine_grad(tg, T=4, k=2, D=64, dout=at(0), lddo=64, Y=at(1), y_rows=8, ldy=64, place=at(2), weight=at(3), dY=at(4),
                 lddy=64, dweight=at(5), dtype=F16):
    return tg.tg_combine_grad(T, k, D, dout, lddo, Y, y_rows, ldy, place, weight, dY, lddy, dweight, dtype)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), "TG_ERR_INVALID_ARG"), (dict(dout=None), "TG_ERR_INVALID_ARG"), (dict(Y=None), "TG_ERR_INVALID_ARG"),
    (dict(dY=None, dweight=None), "TG_ERR_INVALID_ARG"), (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(lddy=63), "TG_ERR_STRIDE"),
    (dict(lddo=8), "TG_ERR_STRIDE"), (dict(dY=at(4) + 1), "TG_ERR_ALIGN"), (dict(dweight=at(5) + 1), "TG_ERR_ALIGN"),
    (dict(dY=at(1)), "TG_ERR_OVERLAP"), (dict(dY=at(0) + 256), "TG_ERR_OVERLAP"), (dict(dweight=at(3)), "TG_ERR_OVERLAP"),
    (dict(dweight=at(4) + 128), "TG_ERR_OVERLAP"),
])
def test_combine_grad_refusals(tg, kw, code):
    assert status(tg, combine_grad(tg, **kw)) == code


def adapters(tg, T=4, N=64, K=32, rank=8, g=3, X=at(0), ldx=32, row=at(1), offset=at(2), A=at(3), lda=32, B=at(4), ldb=8,
             scale=at(5), Y=at(6), ldy=64, dtype=F16, ws=at(7), size=1 << 30):
    return tg.tg_adapters(T, N, K, rank, g, X, ldx, row, offset, A, lda, B, ldb, scale, Y, ldy, dtype, ws, size)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), "TG_ERR_INVALID_ARG"), (dict(rank=0), "TG_ERR_INVALID_ARG"), (dict(rank=129, ldb=136), "TG_ERR_INVALID_ARG"),
    (dict(g=4097), "TG_ERR_INVALID_ARG"), (dict(X=None), "TG_ERR_INVALID_ARG"), (dict(row=None), "TG_ERR_INVALID_ARG"),
    (dict(A=None), "TG_ERR_INVALID_ARG"), (dict(B=None), "TG_ERR_INVALID_ARG"), (dict(Y=None), "TG_ERR_INVALID_ARG"),
    (dict(ws=None), "TG_ERR_INVALID_ARG"), (dict(dtype=F32), "TG_ERR_DTYPE"), (dict(lda=24), "TG_ERR_STRIDE"),
    (dict(ldb=4), "TG_ERR_STRIDE"), (dict(ldy=32), "TG_ERR_STRIDE"), (dict(ldx=0), "TG_ERR_STRIDE"),
    (dict(ldb=12), "TG_ERR_ALIGN"), (dict(ldx=36), "TG_ERR_ALIGN"), (dict(Y=at(6) + 8), "TG_ERR_ALIGN"),
    (dict(A=at(3) + 2), "TG_ERR_ALIGN"), (dict(ws=at(7) + 16), "TG_ERR_ALIGN"), (dict(scale=at(5) + 1), "TG_ERR_ALIGN"),
    (dict(size=8), "TG_ERR_BUFFER"), (dict(Y=at(0)), "TG_ERR_OVERLAP"), (dict(ws=at(6)), "TG_ERR_OVERLAP"),
    (dict(scale=at(6) + 64), "TG_ERR_OVERLAP"),
])
def test_adapters_refusals(tg, kw, code):
    assert status(tg, adapters(tg, **kw)) == code


def test_valid_arguments_reach_the_device_check(tg):
    if not no_device():
        pytest.skip("device present: covered by the GPU tests")
    want = tg.TG_ERR_UNSUPPORTED_DEVICE
    assert route(tg) == want and route(tg, bias=None) == want and route(tg, dtype=F32) == want
    assert route(tg, E=60, ld=63, logits=at(0) + 2, groups=4, kept=2, top=2, k=30, score=1, renorm=1) == want
    assert route_grad(tg) == want
    assert group_rows(tg) == want and group_rows(tg, place=None) == want and group_rows(tg, R=2048, ws=None, size=0) == want
    assert grouped(tg) == want and grouped(tg, row=None) == want and grouped(tg, perm=0) == want
    assert grouped(tg, g=1, stride=0) == want and grouped(tg, bias=at(5), relu=1, relu_of=at(6)) == want
    assert grouped(tg, K=31, ldx=32, ldb=32, N=63, ldy=64, stride=64 * 32) == want
    assert grouped_grad(tg) == want and grouped_grad(tg, row=None) == want and grouped_grad(tg, perm=0, lddb=64) == want
    assert combine(tg) == want and combine(tg, weight=None) == want and combine(tg, Y=at(0) + 2, ldy=65) == want
    assert combine_grad(tg) == want and combine_grad(tg, dY=None) == want
    assert combine_grad(tg, dweight=None, Y=None) == want
    assert adapters(tg) == want and adapters(tg, scale=None) == want


def test_workspace_sizes(tg):
    assert tg.tg_group_rows_workspace_size(2048, 100) == 0
    assert tg.tg_group_rows_workspace_size(2049, 100) == 2 * 100 * 4
    for call in (lambda: tg.tg_group_rows_workspace_size(0, 1), lambda: tg.tg_adapters_workspace_size(1, 1, 1, 129, 1, F16)):
        with pytest.raises(tg.TileGemmError) as e:
            call()
        assert e.value.status == tg.TG_ERR_INVALID_ARG
    with pytest.raises(tg.TileGemmError) as e:
        tg.tg_adapters_workspace_size(1, 1, 1, 1, 1, F32)
    assert e.value.status == tg.TG_ERR_DTYPE
    assert tg.tg_adapters_workspace_size(64, 4096, 4096, 16, 64, BF16) > 0
    assert tg.tg_adapters_workspace_size(1000, 4096, 4096, 17, 64, BF16) >= 1000 * 32 * 4
