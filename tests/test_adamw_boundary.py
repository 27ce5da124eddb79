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
