"""The operators of an output head's training step, as cases that can be timed.

Layer norm, linear cross entropy (a projection onto a vocabulary and the
softmax cross entropy of its logits, which are never kept), their gradients,
and the AdamW step.  Each case is one call of one of them:

    ln_fwd   y, mean, rstd            of x[T, D], weight[D], bias[D]
    ln_bwd   dx, dweight, dbias       of dy[T, D] and what ln_fwd read and kept
    ce_fwd   loss[T], lse[T]          of h[T, D], w[V, D], target[T]
    ce_bwd   dh[T, D], dw[V, D]       of those, lse[T] and the upstream dloss[T]
    adamw    parameters, fp32 master copies and both states, updated in place

`own` chooses who computes: elementary torch operations in 32 bits, rounded
once at the end, or the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5              # layer norm
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP, SEED = 1e-3, 0.9, 0.999, 1e-8, 0.1, 7, 12345
BLOCK = 256             # elements that share a scale of an 8-bit state
IGNORED = -100          # a target outside the vocabulary: no loss, no gradient


def listed():
    return [
        # the norm before the projection, of the one token a decoder is at: launch latency
        {"name": "ln_fwd_one_token", "op": "ln_fwd", "T": 1, "D": 4096, "dtype": "bf16", "pad": 0},
        # a training batch of long sequences through a wide model
        {"name": "ln_fwd_batch", "op": "ln_fwd", "T": 16384, "D": 4096, "dtype": "bf16", "pad": 0},
        # a small fp16 model's ragged batch; x and dy are column slices of wider buffers
        {"name": "ln_bwd_ragged_f16", "op": "ln_bwd", "T": 1501, "D": 1000, "dtype": "f16", "pad": 24},
        # the gradient of the batch above
        {"name": "ln_bwd_batch", "op": "ln_bwd", "T": 16384, "D": 4096, "dtype": "bf16", "pad": 0},
        # the log-likelihood of one token under a large vocabulary: reading w is all the time
        {"name": "ce_fwd_one_token", "op": "ce_fwd", "T": 1, "D": 4096, "V": 131072, "dtype": "bf16", "pad": 0},
        # scoring a few ragged texts with an fp16 model, an odd vocabulary
        {"name": "ce_fwd_scoring_f16", "op": "ce_fwd", "T": 777, "D": 1000, "V": 50021, "dtype": "f16", "pad": 8},
        # the loss of a training batch
        {"name": "ce_fwd_batch", "op": "ce_fwd", "T": 8192, "D": 4096, "V": 131072, "dtype": "bf16", "pad": 0},
        # one short text of a small model
        {"name": "ce_bwd_small", "op": "ce_bwd", "T": 128, "D": 512, "V": 4096, "dtype": "bf16", "pad": 0},
        # ragged everything, fp16
        {"name": "ce_bwd_ragged_f16", "op": "ce_bwd", "T": 1111, "D": 2056, "V": 20011, "dtype": "f16", "pad": 8},
        # the gradients of a training batch
        {"name": "ce_bwd_batch", "op": "ce_bwd", "T": 4096, "D": 4096, "V": 65536, "dtype": "bf16", "pad": 0},
        # the norms' weights and biases of a model: many small tensors, 32-bit states
        {"name": "adamw_small_tensors", "op": "adamw", "tensors": 12, "total": 60000, "dtype": "bf16", "bits": 32},
        # a projection and its neighbours, 8-bit states
        {"name": "adamw_head_8bit", "op": "adamw", "tensors": 4, "total": 200000003, "dtype": "bf16", "bits": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ce_fwd", "ce_bwd", "adamw"])
    dtype = rng.choice(["f16", "bf16"])
    pad = rng.choice([0, 0, 8, 24, 3])
    if op in ("ln_fwd", "ln_bwd"):
        d = _log(rng, 64, 16384)
        t = _log(rng, 1, min(16384, (16384 * 4096) // d))
        return {"op": op, "T": t, "D": d, "dtype": dtype, "pad": pad}
    if op in ("ce_fwd", "ce_bwd"):
        d = _log(rng, 64, 4096)
        v = _log(rng, 1000, 131072 if op == "ce_fwd" else 65536)
        if rng.random() < 0.6:  # whole rows of 16 bytes, as models have them
            d = (d + 7) // 8 * 8
        t = _log(rng, 1, 8192 if op == "ce_fwd" else 4096)
        return {"op": op, "T": t, "D": d, "V": v, "dtype": dtype, "pad": pad if d % 8 == 0 else 0}
    n = rng.randint(1, 12)
    return {"op": op, "tensors": n, "total": max(n, _log(rng, 1000, 200000003)),
            "dtype": rng.choice(["f16", "bf16", "f32"]), "bits": rng.choice([8, 32])}


def _sizes(case):
    """Uneven parts of case["total"]: each next tensor is about half of what is left."""
    left, sizes = case["total"], []
    for k in range(case["tensors"] - 1):
        keep = case["tensors"] - 1 - k
        sizes.append(max(1, min(left - keep, left // 2 if case["total"] > 1 << 20 else left // (keep + 1))))
        left -= sizes[-1]
    return sizes + [left]


def _rows(gen, rows, cols, pad, dtype, scale=1.0, shift=0.0):
    """A rows x cols view of a buffer whose rows are `pad` elements longer."""
    full = torch.empty(rows, cols + pad, device="cuda", dtype=dtype)
    step = max(1, (1 << 28) // (cols + pad))
    for r in range(0, rows, step):
        part = torch.randn(min(step, rows - r), cols + pad, device="cuda", generator=gen)
        full[r:r + step] = part * scale + shift
    return full[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        t, d = case["T"], case["D"]
        s["x"] = _rows(gen, t, d, case["pad"], dt, 1.5, 0.25)
        s["weight"] = (1 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(dt)
        s["bias"] = (0.1 * torch.randn(d, device="cuda", generator=gen)).to(dt)
        if case["op"] == "ln_fwd":
            s["y"] = torch.empty(t, d, device="cuda", dtype=dt)
            s["mean"], s["rstd"] = torch.empty(2, t, device="cuda").unbind(0)
            return s
        s["dy"] = _rows(gen, t, d, case["pad"], dt, 0.5)
        s["mean"], s["rstd"] = _ln_statistics(s["x"])
        s["dx"] = torch.empty(t, d, device="cuda", dtype=dt)
        s["dweight"], s["dbias"] = torch.empty(d, device="cuda", dtype=dt), torch.empty(d, device="cuda", dtype=dt)
        return s
    if case["op"] in ("ce_fwd", "ce_bwd"):
        t, d, v = case["T"], case["D"], case["V"]
        s["h"] = _rows(gen, t, d, case["pad"], dt)  # a norm's output
        s["w"] = _rows(gen, v, d, case["pad"], dt, 2 / math.sqrt(d))
        s["target"] = torch.randint(0, v, (t,), device="cuda", generator=gen)
        if t > 1:  # the prompt's and the padding's tokens
            s["target"][torch.rand(t, device="cuda", generator=gen) < 0.1] = IGNORED
        if case["op"] == "ce_fwd":
            s["loss"], s["lse"] = torch.empty(2, t, device="cuda").unbind(0)
            return s
        s["lse"] = torch.logsumexp(s["h"].float() @ s["w"].float().T, 1)  # as the forward call left it
        valid = s["target"] >= 0
        # the mean over the tokens that count, times a loss scale as fp16 training needs it
        up = (1024.0 if case["dtype"] == "f16" else 1.0) / valid.sum().clamp(min=1)
        s["dloss"] = up.float().expand(t).contiguous()
        s["dh"] = torch.empty(t, d, device="cuda", dtype=dt)
        s["dw"] = torch.empty(v, d, device="cuda", dtype=dt)
        return s
    flat = lambda scale: [torch.randn(n, device="cuda", generator=gen) * scale for n in _sizes(case)]  # noqa: E731
    master = flat(0.02)
    s["p"] = [x.to(dt) for x in master]
    s["master"] = master if dt != torch.float32 else None
    s["g"] = [x.to(dt) for x in flat(1e-2)]
    m, v = flat(3e-3), [x.square() for x in flat(1e-2)]
    if case["bits"] == 8:
        s["m"], s["m_scale"] = map(list, zip(*[_encode_signed(x) for x in m]))
        s["v"], s["v_scale"] = map(list, zip(*[_encode_root(x) for x in v]))
    else:
        s["m"], s["v"] = m, v
    return s


# ------------------------------------------------------------ plain forms

def _ln_statistics(x):
    x = x.float()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return mean, 1 / torch.sqrt(var + EPS)


def _plain_ln_fwd(s):
    x = s["x"].float()
    mean, rstd = _ln_statistics(x)
    y = (x - mean[:, None]) * rstd[:, None] * s["weight"].float() + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(s):
    dy, dt = s["dy"].float(), s["x"].dtype
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return {"dx": dx.to(dt), "dweight": (dy * xhat).sum(0).to(dt), "dbias": dy.sum(0).to(dt)}


def _plain_ce_fwd(s):
    logits = s["h"].float() @ s["w"].float().T
    top = logits.amax(1)
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    counts = (s["target"] >= 0) & (s["target"] < s["V"])
    picked = logits.gather(1, s["target"].clamp(0, s["V"] - 1)[:, None])[:, 0]
    return {"loss": torch.where(counts, lse - picked, 0.0), "lse": lse}


def _plain_ce_bwd(s):
    h, w, dt = s["h"].float(), s["w"].float(), s["h"].dtype
    counts = (s["target"] >= 0) & (s["target"] < s["V"])
    g = torch.exp(h @ w.T - s["lse"][:, None])
    rows = torch.arange(s["T"], device="cuda")
    g[rows, s["target"].clamp(0, s["V"] - 1)] -= 1.0
    g *= torch.where(counts, s["dloss"], 0.0)[:, None]
    return {"dh": (g @ w).to(dt), "dw": (g.T @ h).to(dt)}


def _blocks(x):
    """x as rows of BLOCK elements, the last one filled up with zeros."""
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def _scaled(x):
    """Each element over its block's scale, and the scales: a 448th of the block's largest magnitude."""
    rows = _blocks(x)
    scale = rows.abs().amax(1) * (1.0 / 448.0)
    q = torch.where(scale[:, None] == 0, rows, rows / scale[:, None])
    return q.clamp(-448.0, 448.0).view(-1)[:x.numel()], scale


def _encode_signed(x):
    q, scale = _scaled(x)
    return q.to(torch.float8_e4m3fn), scale


def _mixed(n, seed):
    """20 bits for each of n elements, from its index and the seed (32-bit arithmetic)."""
    x = (torch.arange(n, device="cuda") + seed * 0x9E3779B9) & 0xFFFFFFFF
    x = ((x ^ (x >> 16)) * 0x21F0AAAD) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x735A2D97) & 0xFFFFFFFF
    return (x ^ (x >> 15)) & 0xFFFFF


def _encode_root(v):
    """sqrt(v) in e4m3, rounded up with the probability of what is cut off; above zero it stays so."""
    q, scale = _scaled(torch.sqrt(v))
    bits = _mixed(q.numel(), SEED)
    normal = ((q.view(torch.int32) + bits.to(torch.int32)) & ~0xFFFFF).view(torch.float32)
    tiny = torch.floor(q * 512.0 + bits.float() * 2.0**-20).clamp(min=1.0) * 2.0**-9
    code = torch.where(q >= 2.0**-6, normal, torch.where(q > 0, tiny, q))
    return code.to(torch.float8_e4m3fn), scale


def _decode(code, scale):
    return (_blocks(code.float()) * scale[:, None]).view(-1)[:code.numel()]


def _plain_adamw(s):
    step_size = LR / (1 - BETA1**STEP)
    root = 1 / math.sqrt(1 - BETA2**STEP)
    for i, p in enumerate(s["p"]):
        g = s["g"][i].float()
        w = s["master"][i] if s["master"] else p
        eight = s["bits"] == 8
        m = _decode(s["m"][i], s["m_scale"][i]) if eight else s["m"][i]
        v = _decode(s["v"][i], s["v_scale"][i]).square() if eight else s["v"][i]
        m = m * BETA1 + g * (1 - BETA1)
        v = v * BETA2 + g * g * (1 - BETA2)
        w.copy_(w * (1 - LR * DECAY) - m / (torch.sqrt(v) * root + ADAM_EPS) * step_size)
        if s["master"]:
            p.copy_(w)
        if eight:
            for name, (code, scale) in (("m", _encode_signed(m)), ("v", _encode_root(v))):
                s[name][i].copy_(code)
                s[name + "_scale"][i].copy_(scale)
        else:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)


# ---------------------------------------------------- the library's calls

def _workspace(s, bytes_needed):
    """A program's workspace, made on the first call and kept."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(max(1, bytes_needed()), device="cuda", dtype=torch.uint8)
    return s["workspace"], s["workspace"].numel()


def _own(s):
    import tiled_gemm_layouts_gb300 as tg
    op = s["op"]
    dt = {"f16": tg.TG_F16, "bf16": tg.TG_BF16, "f32": tg.TG_F32}[s["dtype"]]
    if op == "ln_fwd":
        tg.layernorm(s["T"], s["D"], s["x"], s["x"].stride(0), s["weight"], s["bias"], EPS, s["y"], s["D"], s["mean"],
                     s["rstd"], dt)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_bwd":
        ws, size = _workspace(s, lambda: tg.tg_layernorm_grad_workspace_size(s["T"], s["D"], dt))
        tg.layernorm_grad(s["T"], s["D"], s["dy"], s["dy"].stride(0), s["x"], s["x"].stride(0), s["weight"], s["mean"],
                          s["rstd"], s["dx"], s["D"], s["dweight"], s["dbias"], dt, ws, size)
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if op == "ce_fwd":
        ws, size = _workspace(s, lambda: tg.tg_linear_ce_workspace_size(
            s["T"], s["V"], s["D"], s["h"], s["h"].stride(0), s["w"], s["w"].stride(0), dt))
        tg.linear_ce(s["T"], s["V"], s["D"], s["h"], s["h"].stride(0), s["w"], s["w"].stride(0), s["target"], s["loss"],
                     s["lse"], dt, ws, size)
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "ce_bwd":
        ws, size = _workspace(s, lambda: tg.tg_linear_ce_grad_workspace_size(
            s["T"], s["V"], s["D"], s["h"], s["h"].stride(0), s["w"], s["w"].stride(0), s["dh"], s["D"], s["dw"], s["D"], dt))
        tg.linear_ce_grad(s["T"], s["V"], s["D"], s["h"], s["h"].stride(0), s["w"], s["w"].stride(0), s["target"], s["lse"],
                          s["dloss"], s["dh"], s["D"], s["dw"], s["D"], dt, ws, size)
        return {"dh": s["dh"], "dw": s["dw"]}
    if "plan" not in s:  # the parameters' descriptors, made once
        n = len(s["p"])
        s["plan"] = tg.make_adamw_tensors(s["p"], s["g"], s["m"], s["v"], master=s["master"] or [None] * n,
                                          m_scale=s.get("m_scale"), v_scale=s.get("v_scale"))
    tg.adamw(s["plan"], tg.make_adamw_options(LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP, dtype=dt, grad_dtype=dt,
                                              state_bits=s["bits"], seed=SEED))


def run(state):
    if state["op"] == "adamw":  # in place
        _own(state) if own else _plain_adamw(state)
        return {k: state[k] for k in ("p", "master", "m", "v", "m_scale", "v_scale") if state.get(k) is not None}
    if own:
        return _own(state)
    return {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "ce_fwd": _plain_ce_fwd, "ce_bwd": _plain_ce_bwd}[state["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        t, d = case["T"], case["D"]
        if op == "ln_fwd":
            return {"bytes": 4 * t * d + 4 * d + 8 * t, "flops": 8 * t * d}
        return {"bytes": 6 * t * d + 6 * d + 8 * t, "flops": 14 * t * d}
    if op in ("ce_fwd", "ce_bwd"):
        t, d, v = case["T"], case["D"], case["V"]
        if op == "ce_fwd":
            return {"bytes": 2 * (t + v) * d + 16 * t, "flops": 2 * t * v * d}
        return {"bytes": 4 * (t + v) * d + 16 * t, "flops": 6 * t * v * d}  # the logits once more, and two products
    n, e = case["total"], 4 if case["dtype"] == "f32" else 2
    weights = 8 if e == 4 else 8 + 2  # read and written; with a 16-bit copy written beside the fp32 one
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (weights + e + states), "flops": 14 * n}


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    wide = lambda k: s[k].double()  # noqa: E731
    if op in ("ln_fwd", "ln_bwd"):
        x, w, b = (wide(k).requires_grad_() for k in ("x", "weight", "bias"))
        if op == "ln_bwd":  # the statistics are inputs here: their own gradient is part of the formula
            var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
            y = (x - mean) / torch.sqrt(var + EPS) * w + b
            dx, dw, db = torch.autograd.grad(y, (x, w, b), wide("dy"))
            return {"dx": dx, "dweight": dw, "dbias": db}
        with torch.no_grad():
            mean = x.sum(1) / case["D"]
            rstd = (x.square().sum(1) / case["D"] - mean.square() + EPS) ** -0.5
            return {"y": w * (x * rstd[:, None] - (mean * rstd)[:, None]) + b, "mean": mean, "rstd": rstd}
    if op in ("ce_fwd", "ce_bwd"):
        if 2e-12 * case["T"] * case["D"] * case["V"] * (1 if op == "ce_fwd" else 3) > 15:
            return None
        t, v = case["T"], case["V"]
        h, w = wide("h").requires_grad_(op == "ce_bwd"), wide("w").requires_grad_(op == "ce_bwd")
        valid = s["target"] >= 0
        logits = torch.mm(h, w.t())
        if op == "ce_fwd":
            lse = torch.logsumexp(logits, 1)
            loss = torch.nn.functional.nll_loss(logits - lse[:, None], s["target"], ignore_index=IGNORED, reduction="none")
            return {"loss": loss, "lse": lse}
        # a function of h and w whose derivative by the logits is exp(l - lse) less one at the target
        mass = torch.exp(logits - wide("lse")[:, None]).sum(1)
        hit = (h * w[s["target"].clamp(min=0)]).sum(1)
        dh, dw = torch.autograd.grad(((mass - hit) * wide("dloss"))[valid].sum(), (h, w))
        return {"dh": dh, "dw": dw}
    out = {"p": [], "master": [], "m": [], "v": []}
    for i, g in enumerate(s["g"]):
        g = g.double()
        w = (s["master"] or s["p"])[i].double()
        m, v = s["m"][i].double(), s["v"][i].double()
        if case["bits"] == 8:
            of = torch.arange(g.numel(), device="cuda") // BLOCK
            m, v = m * s["m_scale"][i].double()[of], (v * s["v_scale"][i].double()[of]) ** 2
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g**2 - v)
        w = w - LR * (DECAY * w + (m / (1 - BETA1**STEP)) / ((v / (1 - BETA2**STEP)) ** 0.5 + ADAM_EPS))
        # an 8-bit state's rounding has no 64-bit value of its own
        for k, x in (("p", w), ("master", w if s["master"] else None)) + ((("m", m), ("v", v)) if case["bits"] == 32 else (("m", None), ("v", None))):
            out[k].append(x)
    if not s["master"]:
        del out["master"]
    return out
