"""Refusals of tg_adamw without a GPU that concern operands of the whole call
(fake, never-dereferenced pointers)."""
import pytest

G = 1 << 30
FAKE = 1 << 44
BF16 = 1


def at(k):
    return FAKE + k * 64 * G


def step(tg, grad_scale, bits=8, n=1000, master=at(4)):
    scales = (at(5), at(6)) if bits == 8 else (None, None)
    t = tg.make_adamw_tensors([at(0), at(10)], [at(1), at(11)], [at(2), at(12)], [at(3), at(13)],
                              master=[master, None], m_scale=[scales[0], scales[0] and at(15)],
                              v_scale=[scales[1], scales[1] and at(16)], numel=[n, 50])
    return tg.tg_adamw(t, tg.make_adamw_options(1e-3, 0.9, 0.99, 1e-8, 0.1, 1, BF16, None, bits, 0, grad_scale))


# the first and the last bytes of what one of the two tensors writes
@pytest.mark.parametrize("where", [at(0), at(0) + 1996, at(2), at(2) + 996, at(3) + 500, at(4) + 3996, at(5) + 12, at(6),
                                   at(10) + 96, at(13) + 48, at(15)])
def test_a_gradient_scale_inside_what_the_step_writes(tg, where):
    assert tg.tg_status_string(step(tg, where)) == "TG_ERR_OVERLAP"


def test_a_gradient_scale_inside_32_bit_states(tg):
    for where in (at(2) + 3996, at(3), at(13) + 196):
        assert tg.tg_status_string(step(tg, where, bits=32)) == "TG_ERR_OVERLAP"


def test_a_gradient_scale_beside_them_passes_the_overlap_check(tg):
    import torch
    if torch.cuda.is_available():
        pytest.skip("device present: the pointers are then looked up")
    # beside an operand, inside a gradient (both are read only), inside scales
    # that 32-bit states do not have
    for where in (at(0) + 2000, at(5) + 16, at(1), at(11) + 96, at(9)):
        assert step(tg, where) == tg.TG_ERR_UNSUPPORTED_DEVICE
    assert step(tg, at(5), bits=32) == tg.TG_ERR_UNSUPPORTED_DEVICE
    assert step(tg, at(4), master=None) == tg.TG_ERR_UNSUPPORTED_DEVICE


def lists(shape=(6, 100), **other):
    """Tensors of one parameter (on the CPU: only their shapes and strides are looked at)."""
    import torch
    n, blocks = shape[0] * shape[1], (shape[0] * shape[1] + 255) // 256
    t = dict(p=torch.zeros(shape), g=torch.zeros(shape), m=torch.zeros(n), v=torch.zeros(shape),
             master=torch.zeros(shape), ms=torch.zeros(blocks), vs=torch.zeros(blocks))
    t.update(other)
    return ([t["p"]], [t["g"]], [t["m"]], [t["v"]]), dict(master=[t["master"]], m_scale=[t["ms"]], v_scale=[t["vs"]])


def test_tensors_whose_elements_do_not_lie_one_after_another(tg):
    import torch
    wide = torch.zeros(6, 108)[:, :100]
    for kw in (dict(g=torch.zeros(1).expand(6, 100)),          # the gradient of a sum
               dict(g=torch.zeros(100).expand(6, 100)),        # of a broadcast
               dict(p=wide), dict(master=wide), dict(v=wide),  # rows of a wider buffer
               dict(g=torch.zeros(100, 6).t()),                # another order than the parameter's
               dict(m=torch.zeros(1200)[::2]), dict(ms=torch.zeros(6)[::2])):
        at, rest = lists(**kw)
        with pytest.raises(tg.TileGemmError) as e:
            tg.make_adamw_tensors(*at, **rest)
        assert e.value.status == tg.TG_ERR_STRIDE, kw


def test_tensors_that_are_too_small(tg):
    import torch
    for kw, code in ((dict(g=torch.zeros(6, 99)), tg.TG_ERR_INVALID_ARG), (dict(m=torch.zeros(599)), tg.TG_ERR_INVALID_ARG),
                     (dict(v=torch.zeros(6, 99)), tg.TG_ERR_INVALID_ARG), (dict(master=torch.zeros(1)), tg.TG_ERR_INVALID_ARG),
                     (dict(ms=torch.zeros(2)), tg.TG_ERR_BUFFER), (dict(vs=torch.zeros(0)), tg.TG_ERR_BUFFER)):
        at, rest = lists(**kw)
        with pytest.raises(tg.TileGemmError) as e:
            tg.make_adamw_tensors(*at, **rest)
        assert e.value.status == code, kw


def test_tensors_that_may_be_given(tg):
    import torch
    at, rest = lists()
    t = tg.make_adamw_tensors(*at, **rest)
    assert t[0].numel == 600 and t[0].grad == at[1][0].data_ptr() and t[0].v_scale == rest["v_scale"][0].data_ptr()
    # one dense order for all of them, whichever it is; flat states beside contiguous parameters
    turned = {k: torch.zeros(100, 6).t() for k in ("p", "g", "m", "v", "master")}
    at, rest = lists(**turned)
    assert tg.make_adamw_tensors(*at, **rest)[0].param == turned["p"].data_ptr()
    cubes = {k: torch.zeros(2, 3, 4, 5).contiguous(memory_format=torch.channels_last) for k in ("p", "g", "m", "v", "master")}
    at, rest = lists(**cubes)
    assert tg.make_adamw_tensors(*at, **rest)[0].numel == 120
    empty = {k: torch.zeros(0, 5) for k in ("p", "g", "m", "v", "master")}
    assert tg.make_adamw_tensors(*lists(**empty)[0])[0].numel == 0
    # states that were rounded up to whole blocks; fewer elements than the tensors hold, on request
    at, rest = lists(m=torch.zeros(768), v=torch.zeros(768), ms=torch.zeros(4))
    assert tg.make_adamw_tensors(*at, **rest)[0].numel == 600
    at, rest = lists()
    assert tg.make_adamw_tensors(*at, **rest, numel=[512])[0].numel == 512
