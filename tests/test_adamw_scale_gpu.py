"""AdamW's gradient factor with 8-bit states."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16, torch.float32], ids=["f16", "bf16", "f32"])
def test_a_power_of_two_equals_scaled_gradients(tg, dt):
    """Gradients times 2^-3 by the factor, and beforehand: the same bits."""
    sizes = [1, 300, 2049, 70001]
    g = torch.Generator(device="cuda").manual_seed(31)
    code = {torch.float16: tg.TG_F16, torch.bfloat16: tg.TG_BF16, torch.float32: tg.TG_F32}[dt]
    grads = [torch.randn(n, device="cuda", generator=g).to(dt) for n in sizes]
    start = dict(p=[torch.randn(n, device="cuda", generator=g).to(dt) for n in sizes],
                 m=[torch.randint(0, 0x7F, (n,), device="cuda", generator=g, dtype=torch.uint8) for n in sizes],
                 v=[torch.randint(0, 0x7F, (n,), device="cuda", generator=g, dtype=torch.uint8) for n in sizes],
                 ms=[torch.rand((n + 255) // 256, device="cuda", generator=g) * 1e-3 for n in sizes],
                 vs=[torch.rand((n + 255) // 256, device="cuda", generator=g) * 1e-3 for n in sizes])
    ends = []
    for factor in (torch.tensor(0.125, device="cuda"), None):
        s = {k: [x.clone() for x in v] for k, v in start.items()}
        used = grads if factor is not None else [x * 0.125 for x in grads]
        # (fp16: a product below 2^-14 would be rounded beforehand, and not by the factor)
        if dt == torch.float16:
            used = [torch.where(x.abs() < 2.0**-10, torch.zeros_like(x), x if factor is not None else x * 0.125) for x in grads]
        tg.adamw(tg.make_adamw_tensors(s["p"], used, s["m"], s["v"], m_scale=s["ms"], v_scale=s["vs"]),
                 tg.make_adamw_options(1e-2, 0.9, 0.99, 1e-8, 0.1, 4, dtype=code, state_bits=8, seed=5, grad_scale=factor))
        torch.cuda.synchronize()
        ends.append(s)
    for k in start:
        for a, b, before in zip(ends[0][k], ends[1][k], start[k]):
            assert torch.equal(a, b) and not torch.equal(a, before), k
