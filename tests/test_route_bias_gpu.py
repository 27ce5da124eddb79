"""Balance biases near the ends of fp32: experts and groups that are all but shut out or forced."""
import pytest
import torch

from rows_reference import assert_within, code, route

pytestmark = pytest.mark.gpu

LOWEST = torch.finfo(torch.float32).min


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("t,size", [(5, 4), (5, 24), (3000, 8)])
@pytest.mark.parametrize("of_group", [
    [-3.0e38, -2.5e38, -2.0e38, 0.0],          # sums of two are below fp32's range
    [2.0e38, 2.5e38, 3.0e38, 2.2e38],          # and above it
    [LOWEST, LOWEST, LOWEST, LOWEST],
    [LOWEST, 0.0, LOWEST, -0.5],
    [-3.0e38, 3.0e38, 2.9e38, -2.9e38]])
def test_groups_of_large_biases(tg, of_group, t, size, top, sigmoid, dtype):
    gen = torch.Generator(device="cuda").manual_seed(size)
    e, k = 4 * size, 6
    logits = torch.randn(t, e, generator=gen, device="cuda").to(dtype)
    bias = torch.tensor(of_group, device="cuda").repeat_interleave(size)
    index, weight = torch.empty(t, k, dtype=torch.int32, device="cuda"), torch.empty(t, k, device="cuda")
    tg.route(t, e, logits, e, bias, index, weight, code(tg, dtype),
             tg.make_route_options(k, tg.TG_ROUTE_SIGMOID if sigmoid else tg.TG_ROUTE_SOFTMAX, 4, 2, top, True))
    some = slice(0, t, max(1, t // 40))
    want_index, want = route(logits[some], bias, k, sigmoid, 4, 2, top, True, 1.0)
    assert torch.equal(index[some], want_index)
    # an exponential, a quotient and a sum of six, each within 2^-22
    assert_within(weight[some], want, 2.0**-19 * want, "weight")


def test_an_infinite_logit_is_above_the_largest_finite_one(tg):
    """Groups ranked by their largest logits, which are keys themselves."""
    logits = torch.zeros(3, 8, device="cuda")
    logits[:, 1], logits[0, 6], logits[1, 6] = torch.finfo(torch.float32).max, float("inf"), 1.0
    index, weight = torch.empty(3, 2, dtype=torch.int32, device="cuda"), torch.empty(3, 2, device="cuda")
    tg.route(3, 8, logits, 8, None, index, weight, tg.TG_F32, tg.make_route_options(2, tg.TG_ROUTE_SIGMOID, 2, 1, 1))
    assert index.tolist() == [[6, 4], [1, 0], [1, 0]]
    assert weight.tolist() == [[1.0, 0.5], [1.0, 0.5], [1.0, 0.5]]
