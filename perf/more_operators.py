"""The operators of rows that choose their weights, as cases that can be timed.

Routing of tokens to experts, the experts' products, the sum of their
outputs, and low-rank adapters of many requests.  Each case is one pass:

    route         index, weight [T, k] of logits[T, E], and the rows grouped by expert:
                  offset[E + 1], row[T k], place[T k]
    route_grad    dlogits[T, E] of dweight[T, k]
    experts       y[i] = relu(x[row[i] / k] w[e]^T + bias[e]) for the grouped rows i of each expert e
    experts_grad  dx[i] = (dy[i] w[e]) where h[i] > 0, and dw[e], the sum of dy[i]^T x[row[i] / k]
    combine       out[t] = sum over j of weight[t, j] y[place[t, j]], and its gradients dy, dweight
    adapters      y[t] += scale[a] (x[t] a[a]^T) b[a]^T, in place, a the adapter of the token's request

`own` chooses who computes: elementary torch operations in 32 bits, rounded
once at the end (64 bits where experts are ranked), or the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the token a decoder is at: sigmoid scores, a bias for balance, half of the groups kept
        {"name": "route_one_token", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5, "dtype": "bf16", "pad": 0},
        # a training batch through the same router
        {"name": "route_batch", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "kept": 4, "top": 2, "renorm": True, "scale": 2.5, "dtype": "bf16", "pad": 0},
        # a small model's ragged batch, its router in 32 bits, weights renormalised over the chosen experts
        {"name": "route_grad_ragged_f32", "op": "route_grad", "T": 1501, "E": 60, "k": 4, "score": "softmax", "bias": False,
         "groups": 1, "kept": 1, "top": 1, "renorm": True, "scale": 1.0, "dtype": "f32", "pad": 4},
        # the gradient of a training batch, softmax over all experts
        {"name": "route_grad_batch", "op": "route_grad", "T": 16384, "E": 256, "k": 8, "score": "softmax", "bias": False,
         "groups": 1, "kept": 1, "top": 1, "renorm": False, "scale": 1.0, "dtype": "bf16", "pad": 0},
        # one token through its eight experts: reading their weights is all the time
        {"name": "experts_one_token", "op": "experts", "T": 1, "k": 8, "E": 64, "N": 2048, "K": 4096, "relu": True,
         "bias": False, "dtype": "bf16", "pad": 0},
        # a training batch, skewed as routers are before they balance
        {"name": "experts_batch", "op": "experts", "T": 8192, "k": 8, "E": 64, "N": 1024, "K": 4096, "relu": True,
         "bias": False, "dtype": "bf16", "pad": 0},
        # a few ragged texts of a small fp16 model with few, large experts
        {"name": "experts_grad_ragged_f16", "op": "experts_grad", "T": 1111, "k": 2, "E": 8, "N": 1000, "K": 2056,
         "relu": False, "bias": False, "dtype": "f16", "pad": 8},
        # the gradients of a training batch
        {"name": "experts_grad_batch", "op": "experts_grad", "T": 8192, "k": 8, "E": 64, "N": 2048, "K": 1024,
         "relu": True, "bias": False, "dtype": "bf16", "pad": 0},
        # a decoder's batch of sixteen requests
        {"name": "combine_decode", "op": "combine", "T": 16, "k": 8, "D": 4096, "grad": False, "dropped": 0.0,
         "dtype": "bf16", "pad": 0},
        # a training batch, padding tokens among it, with the gradients
        {"name": "combine_batch", "op": "combine", "T": 8192, "k": 8, "D": 4096, "grad": True, "dropped": 0.05,
         "dtype": "bf16", "pad": 0},
        # a decoder's batch: each request brings an adapter of its own
        {"name": "adapters_decode", "op": "adapters", "T": 64, "G": 64, "runs": 64, "rank": 16, "N": 4096, "K": 4096,
         "dtype": "bf16", "pad": 0},
        # ragged prompts of twelve requests, some without an adapter
        {"name": "adapters_prompts_f16", "op": "adapters", "T": 7777, "G": 8, "runs": 12, "rank": 32, "N": 4096, "K": 4096,
         "dtype": "f16", "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "experts", "experts_grad", "combine", "adapters"])
    dtype = rng.choice(["f16", "bf16"])
    pad = rng.choice([0, 0, 8, 24])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8])
        size = _log(rng, 4, 512 // groups)
        kept = rng.randint(1, groups)
        e = groups * size
        t = _log(rng, 1, min(16384, 16384 * 256 // e))
        return {"op": op, "T": t, "E": e, "k": rng.randint(1, min(8, kept * size)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups, "kept": kept,
                "top": rng.choice([1, 2]), "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]),
                "dtype": rng.choice(["f16", "bf16", "f32"]), "pad": rng.choice([0, 0, 4, 3])}
    if op in ("experts", "experts_grad"):
        e = _log(rng, 2, 64)
        k = rng.randint(1, min(8, e))
        n, d = _log(rng, 64, 4096), _log(rng, 64, 4096)
        if rng.random() < 0.7:  # whole rows of 16 bytes, as models have them
            n, d = (n + 7) // 8 * 8, (d + 7) // 8 * 8
        most = 8192 * 8 * 1024 * (4096 if op == "experts" else 2048)
        t = _log(rng, 1, max(1, min(8192, most // (k * n * d))))
        return {"op": op, "T": t, "k": k, "E": e, "N": n, "K": d, "relu": rng.random() < 0.5,
                "bias": op == "experts" and rng.random() < 0.5, "dtype": dtype, "pad": pad}
    if op == "combine":
        d, k = _log(rng, 64, 8192), rng.randint(1, 8)
        t = _log(rng, 1, min(8192, 8192 * 8 * 4096 // (k * d)))
        return {"op": op, "T": t, "k": k, "D": d, "grad": rng.random() < 0.5, "dropped": rng.choice([0.0, 0.1]),
                "dtype": dtype, "pad": pad}
    g = _log(rng, 1, 128)
    t = _log(rng, 1, 7777)
    return {"op": op, "T": t, "G": g, "runs": min(t, _log(rng, 1, 128)), "rank": rng.choice([4, 8, 16, 24, 32, 64]),
            "N": _log(rng, 64, 4096), "K": _log(rng, 64, 4096), "dtype": dtype, "pad": pad}


# ----------------------------------------------------------------- inputs

def _rows(gen, rows, cols, pad, dtype, scale=1.0):
    """A rows x cols view of a buffer whose rows are whole 16-byte units and `pad` elements longer."""
    ld = (cols + 7) // 8 * 8 + pad
    full = torch.empty(rows, ld, device="cuda", dtype=dtype)
    step = max(1, (1 << 28) // ld)
    for r in range(0, rows, step):
        full[r:r + step] = torch.randn(min(step, rows - r), ld, device="cuda", generator=gen) * scale
    return full[:, :cols]


def _stack(gen, count, rows, cols, pad, dtype, scale):
    """count matrices of rows x cols, the rows as in _rows."""
    flat = _rows(gen, count * rows, cols, pad, dtype, scale)
    return flat.as_strided((count, rows, cols), (rows * flat.stride(0), flat.stride(0), 1))


def _grouped(index, groups):
    """offset, row and place of a stable sort of index; indexes outside 0 .. groups - 1 are in no group."""
    flat = index.reshape(-1).long()
    inside = (flat >= 0) & (flat < groups)
    order = torch.sort(torch.where(inside, flat, groups), stable=True).indices
    count = torch.bincount(flat[inside], minlength=groups)
    offset = torch.cat([count.new_zeros(1), count.cumsum(0)])
    ranked = torch.arange(flat.numel(), device=flat.device)
    place = torch.empty_like(flat).scatter_(0, order, ranked)
    row = torch.where(ranked < offset[-1], order, -1)
    return offset.int(), row.int(), torch.where(inside, place, -1).int()


def _chosen(gen, tokens, experts, k):
    """k different experts for each token, some of them more popular."""
    popular = torch.randn(experts, device="cuda", generator=gen) * 0.5
    return torch.topk(torch.randn(tokens, experts, device="cuda", generator=gen) + popular, k, dim=1).indices.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    op = case["op"]
    empty = lambda *n, dtype=dt: torch.empty(*n, device="cuda", dtype=dtype)  # noqa: E731
    if op in ("route", "route_grad"):
        t, e, k = case["T"], case["E"], case["k"]
        full = (torch.randn(t, e + case["pad"], device="cuda", generator=gen) * 1.5).to(dt)
        s["logits"] = full[:, :e]
        s["balance"] = torch.randn(e, device="cuda", generator=gen) * 0.05 if case["bias"] else None
        if op == "route":
            s["index"], s["weight"] = empty(t, k, dtype=torch.int32), empty(t, k, dtype=torch.float32)
            s["offset"] = empty(e + 1, dtype=torch.int32)
            s["row"], s["place"] = empty(t * k, dtype=torch.int32), empty(t * k, dtype=torch.int32)
            return s
        s["index"], _ = _route(s)
        s["dweight"] = torch.randn(t, k, device="cuda", generator=gen)
        s["dlogits"] = empty(t, e)
        return s
    if op in ("experts", "experts_grad"):
        t, k, e, n, d = (case[x] for x in ("T", "k", "E", "N", "K"))
        s["x"] = _rows(gen, t, d, case["pad"], dt)
        s["w"] = _stack(gen, e, n, d, case["pad"], dt, 1 / math.sqrt(d))
        s["offset"], s["row"], _ = _grouped(_chosen(gen, t, e, k), e)
        s["bounds"] = s["offset"].tolist()
        r = t * k
        if op == "experts":
            s["b"] = (torch.randn(e, n, device="cuda", generator=gen) * 0.1).to(dt) if case["bias"] else None
            s["y"] = _rows(gen, r, n, 0, dt)
            return s
        s["dy"] = _rows(gen, r, n, case["pad"], dt, 0.5)
        s["h"] = _rows(gen, r, d, 0, dt).relu_() if case["relu"] else None  # what the products' input was
        s["dx"] = _rows(gen, r, d, 0, dt)
        s["dw"] = _stack(gen, e, n, d, 0, dt, 1.0)
        return s
    if op == "combine":
        t, k, d = case["T"], case["k"], case["D"]
        r = t * k
        choice = torch.argsort(torch.rand(t, 4 * k, device="cuda", generator=gen), dim=1)[:, :k]
        if case["dropped"]:  # the padding's tokens have no experts
            choice[torch.rand(t, device="cuda", generator=gen) < case["dropped"]] = -1
        s["offset"], s["row"], place = _grouped(choice, 4 * k)
        s["place"] = place.view(t, k)
        s["weight"] = torch.rand(t, k, device="cuda", generator=gen)
        s["y"] = _rows(gen, r, d, case["pad"], dt)
        s["out"] = _rows(gen, t, d, 0, dt)
        if case["grad"]:
            s["dout"] = _rows(gen, t, d, case["pad"], dt, 0.5)
            s["dy"] = _rows(gen, r, d, 0, dt)
            s["dy"][:] = 0  # rows of no token stay as they are
            s["dweight"] = empty(t, k, dtype=torch.float32)
        return s
    t, g, n, d, rank = (case[x] for x in ("T", "G", "N", "K", "rank"))
    # each request's tokens stand together; an adapter of -1 is none
    ends = torch.sort(torch.randperm(t - 1, device="cuda", generator=gen)[:case["runs"] - 1] + 1).values if case["runs"] > 1 \
        else torch.zeros(0, dtype=torch.long, device="cuda")
    request = torch.searchsorted(ends, torch.arange(t, device="cuda"), right=True)
    if case["runs"] == g:
        adapter = torch.randperm(g, device="cuda", generator=gen)
    else:
        adapter = torch.randint(-1, g, (case["runs"],), device="cuda", generator=gen)
    s["offset"], s["row"], _ = _grouped(adapter[request], g)
    s["bounds"] = s["offset"].tolist()
    s["x"] = _rows(gen, t, d, case["pad"], dt)
    s["a"] = _stack(gen, g, rank, d, 0, dt, 1 / math.sqrt(d))
    s["b"] = _stack(gen, g, n, rank, 0, dt, 1 / math.sqrt(rank))
    s["factor"] = torch.rand(g, device="cuda", generator=gen) + 0.5
    s["y"] = _rows(gen, t, n, case["pad"], dt)  # the shared projection's output
    return s


# ------------------------------------------------------------ plain forms

def _route(s):
    """index and weight of the k experts with the largest score + bias, in 64 bits."""
    logits = s["logits"].double()
    t, e, k = s["T"], s["E"], s["k"]
    if s["score"] == "softmax":
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    key = score + s["balance"].double() if s["balance"] is not None else logits
    if s["groups"] > 1:
        size = e // s["groups"]
        by_group = (key if s["balance"] is not None or s["top"] == 1 else score).view(t, s["groups"], size)
        best = torch.sort(by_group, dim=2, descending=True).values[:, :, :s["top"]].sum(2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["kept"]]
        keep = torch.zeros_like(best).scatter_(1, order, 1.0) > 0
        key = key.masked_fill(~keep.repeat_interleave(size, 1), -math.inf)
    index = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    weight = score.gather(1, index)
    if s["renorm"]:
        weight = weight / weight.sum(1, keepdim=True)
    return index.int(), (weight * s["scale"]).float()


def _plain_route(s):
    index, weight = _route(s)
    offset, row, place = _grouped(index, s["E"])
    return {"index": index, "weight": weight, "offset": offset, "row": row, "place": place}


def _plain_route_grad(s):
    logits, c = s["logits"].float(), s["scale"]
    index, g = s["index"].long(), s["dweight"] * c
    if s["score"] == "softmax":
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-logits))
    picked = score.gather(1, index)
    if s["renorm"]:
        share = picked / picked.sum(1, keepdim=True)
        slope = 1 - picked if s["score"] == "sigmoid" else 1.0
        part = share * slope * (g - (g * share).sum(1, keepdim=True))
        out = torch.zeros_like(logits).scatter_(1, index, part)
    elif s["score"] == "sigmoid":
        out = torch.zeros_like(logits).scatter_(1, index, g * picked * (1 - picked))
    else:
        full = torch.zeros_like(logits).scatter_(1, index, g)
        out = score * (full - (g * picked).sum(1, keepdim=True))
    return {"dlogits": out.to(s["logits"].dtype)}


def _each_group(s):
    for e in range(len(s["bounds"]) - 1):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo < hi:
            yield e, lo, hi


def _plain_experts(s):
    y = torch.empty(s["y"].shape, device="cuda", dtype=s["y"].dtype)
    for e, lo, hi in _each_group(s):
        part = s["x"][s["row"][lo:hi].long() // s["k"]].float() @ s["w"][e].float().T
        if s["b"] is not None:
            part = part + s["b"][e].float()
        y[lo:hi] = part.clamp(min=0.0) if s["relu"] else part
    return {"y": y}


def _plain_experts_grad(s):
    dt = s["x"].dtype
    dx = torch.empty(s["dx"].shape, device="cuda", dtype=dt)
    dw = torch.zeros(s["dw"].shape, device="cuda", dtype=dt)
    for e, lo, hi in _each_group(s):
        dy = s["dy"][lo:hi].float()
        part = dy @ s["w"][e].float()
        dx[lo:hi] = torch.where(s["h"][lo:hi] > 0, part, 0.0) if s["h"] is not None else part
        dw[e] = dy.T @ s["x"][s["row"][lo:hi].long() // s["k"]].float()
    return {"dx": dx, "dw": dw}


def _plain_combine(s):
    dt, place = s["y"].dtype, s["place"].long()
    there = place >= 0
    weight = torch.where(there, s["weight"], 0.0)
    out = torch.zeros(s["out"].shape, device="cuda")
    for j in range(s["k"]):
        out += weight[:, j, None] * s["y"][place[:, j].clamp(min=0)].float()
    result = {"out": out.to(dt)}
    if s["grad"]:
        dout = s["dout"].float()
        r = len(s["dy"])
        dy, dweight = torch.zeros(r + 1, s["D"], device="cuda", dtype=dt), torch.zeros_like(weight)
        for j in range(s["k"]):
            at = torch.where(there[:, j], place[:, j], r)  # the last row takes what no row of y is to have
            dy[at] = (weight[:, j, None] * dout).to(dt)
            dweight[:, j] = torch.where(there[:, j], (dout * s["y"][at.clamp(max=r - 1)].float()).sum(1), 0.0)
        result.update(dy=dy[:r], dweight=dweight)
    return result


def _plain_adapters(s):
    for g, lo, hi in _each_group(s):
        t = s["row"][lo:hi].long()
        low = s["x"][t].float() @ s["a"][g].float().T
        s["y"][t] = (s["y"][t].float() + s["factor"][g] * (low @ s["b"][g].float().T)).to(s["y"].dtype)
    return {"y": s["y"]}


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
    if op in ("route", "route_grad"):
        t, e, k = s["T"], s["E"], s["k"]
        opts = tg.make_route_options(k, tg.TG_ROUTE_SIGMOID if s["score"] == "sigmoid" else tg.TG_ROUTE_SOFTMAX,
                                     s["groups"], s["kept"], s["top"], s["renorm"], s["scale"])
        if op == "route_grad":
            tg.route_grad(t, e, s["logits"], s["logits"].stride(0), s["index"], s["dweight"], s["dlogits"], e, dt, opts)
            return {"dlogits": s["dlogits"]}
        tg.route(t, e, s["logits"], s["logits"].stride(0), s["balance"], s["index"], s["weight"], dt, opts)
        ws, size = _workspace(s, lambda: tg.tg_group_rows_workspace_size(t * k, e))
        tg.group_rows(t * k, e, s["index"], s["offset"], s["row"], s["place"], ws, size)
        return {x: s[x] for x in ("index", "weight", "offset", "row", "place")}
    if op in ("experts", "experts_grad"):
        t, k, e, n, d = (s[x] for x in ("T", "k", "E", "N", "K"))
        r = t * k
        if op == "experts":
            epi = tg.make_group_epilogue(bias=s["b"], ld_bias=n, relu=s["relu"])
            tg.grouped_gemm(r, n, d, e, s["x"], t, s["x"].stride(0), s["row"], k, s["w"], s["w"].stride(1),
                            s["w"].stride(0), tg.TG_OP_T, s["offset"], s["y"], s["y"].stride(0), dt, epi)
            return {"y": s["y"]}
        epi = tg.make_group_epilogue(relu_of=s["h"], ld_relu=s["h"].stride(0) if s["h"] is not None else 0)
        tg.grouped_gemm(r, d, n, e, s["dy"], r, s["dy"].stride(0), None, 1, s["w"], s["w"].stride(1), s["w"].stride(0),
                        tg.TG_OP_N, s["offset"], s["dx"], s["dx"].stride(0), dt, epi)
        tg.grouped_gemm_grad(r, n, d, e, s["dy"], s["dy"].stride(0), s["x"], t, s["x"].stride(0), s["row"], k, s["offset"],
                             s["dw"], s["dw"].stride(1), s["dw"].stride(0), tg.TG_OP_T, dt)
        return {"dx": s["dx"], "dw": s["dw"]}
    if op == "combine":
        t, k, d = s["T"], s["k"], s["D"]
        tg.combine(t, k, d, s["y"], t * k, s["y"].stride(0), s["place"], s["weight"], s["out"], s["out"].stride(0), dt)
        if not s["grad"]:
            return {"out": s["out"]}
        tg.combine_grad(t, k, d, s["dout"], s["dout"].stride(0), s["y"], t * k, s["y"].stride(0), s["place"], s["weight"],
                        s["dy"], s["dy"].stride(0), s["dweight"], dt)
        return {"out": s["out"], "dy": s["dy"], "dweight": s["dweight"]}
    t, g, n, d, rank = (s[x] for x in ("T", "G", "N", "K", "rank"))
    ws, size = _workspace(s, lambda: tg.tg_adapters_workspace_size(t, n, d, rank, g, dt))
    tg.adapters(t, n, d, rank, g, s["x"], s["x"].stride(0), s["row"], s["offset"], s["a"], s["a"].stride(1), s["b"],
                s["b"].stride(1), s["factor"], s["y"], s["y"].stride(0), dt, ws, size)
    return {"y": s["y"]}


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "experts": _plain_experts,
            "experts_grad": _plain_experts_grad, "combine": _plain_combine, "adapters": _plain_adapters}[state["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "f32" else 2
    if op == "route":
        t, e, k = case["T"], case["E"], case["k"]
        return {"bytes": size * t * e + 4 * e + 16 * t * k, "flops": 8 * t * e}
    if op == "route_grad":
        t, e, k = case["T"], case["E"], case["k"]
        return {"bytes": size * t * e * (1 if case["renorm"] or case["score"] == "sigmoid" else 2)
                + (0 if not (case["renorm"] or case["score"] == "sigmoid") else size * t * k) + 8 * t * k,
                "flops": 8 * t * e}
    if op in ("experts", "experts_grad"):
        t, k, e, n, d = (case[x] for x in ("T", "k", "E", "N", "K"))
        r = t * k
        used = min(e, r)  # at most
        if op == "experts":
            return {"bytes": 2 * (t * d + used * n * d + r * n) + 4 * r, "flops": 2 * r * n * d}
        return {"bytes": 2 * (t * d + used * n * d + e * n * d + r * n + r * d + (r * d if case["relu"] else 0)) + 4 * r,
                "flops": 4 * r * n * d}
    if op == "combine":
        t, k, d = case["T"], case["k"], case["D"]
        r = int(t * k * (1 - case["dropped"]))
        moved = r * d + t * d + ((r * d + t * d) if case["grad"] else 0)
        return {"bytes": 2 * moved + 8 * t * k + (4 * t * k if case["grad"] else 0), "flops": (5 if case["grad"] else 2) * r * d}
    t, n, d, rank = (case[x] for x in ("T", "N", "K", "rank"))
    used = min(case["G"], case["runs"])  # at most
    return {"bytes": 2 * (t * d + 2 * t * n + used * rank * (n + d)) + 4 * t, "flops": 2 * t * rank * (n + d)}


# ------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("route", "route_grad"):
        logits = s["logits"].double().requires_grad_(op == "route_grad")
        scores = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
        if op == "route":
            return _exact_route(case, s, logits, scores)
        weight = torch.take_along_dim(scores, s["index"].long(), 1) * case["scale"]
        if case["renorm"]:
            weight = case["scale"] * weight / weight.sum(1, keepdim=True)
        return {"dlogits": torch.autograd.grad((weight * s["dweight"].double()).sum(), logits)[0]}
    if op in ("experts", "experts_grad"):
        if 2e-12 * case["T"] * case["k"] * case["N"] * case["K"] * (1 if op == "experts" else 2) > 15:
            return None
        token = torch.div(s["row"].long(), case["k"], rounding_mode="floor")
        count = s["offset"].diff().long()
        owner = torch.repeat_interleave(torch.arange(case["E"], device="cuda"), count)
        out = {"y": torch.zeros(s["y"].shape, device="cuda", dtype=torch.float64)} if op == "experts" else \
              {"dx": torch.zeros(s["dx"].shape, device="cuda", dtype=torch.float64),
               "dw": torch.zeros(s["dw"].shape, device="cuda", dtype=torch.float64)}
        wide = s["x"].double()
        for e in range(case["E"]):
            at = (owner == e).nonzero()[:, 0]
            w, x = s["w"][e].double(), wide.index_select(0, token[at])
            if op == "experts":
                y = torch.einsum("id,nd->in", x, w)
                y = y + s["b"][e].double() if s["b"] is not None else y
                out["y"][at] = torch.relu(y) if case["relu"] else y
                continue
            dy = s["dy"].double()[at]
            dx = torch.einsum("in,nd->id", dy, w)
            out["dx"][at] = dx * (s["h"][at] > 0) if case["relu"] else dx
            out["dw"][e] = torch.einsum("in,id->nd", dy, x)
        return out
    if op == "combine":
        place = s["place"].long()
        there = (place >= 0).double()[..., None]
        y, w = s["y"].double().requires_grad_(case["grad"]), s["weight"].double().requires_grad_(case["grad"])
        total = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
        for j in range(case["k"]):
            total = total + (w[:, j, None] * there[:, j]) * torch.nn.functional.embedding(place[:, j].clamp(min=0), y)
        if not case["grad"]:
            return {"out": total}
        dy, dw = torch.autograd.grad(total, (y, w), s["dout"].double())
        return {"out": total.detach(), "dy": dy, "dweight": dw}
    y = s["y"].double()
    for g in range(case["G"]):
        t = s["row"][s["bounds"][g]:s["bounds"][g + 1]].long()
        delta = torch.linalg.multi_dot([s["x"][t].double(), s["a"][g].double().T, s["b"][g].double().T]) if len(t) else None
        if delta is not None:
            y.index_add_(0, t, s["factor"][g].double() * delta)
    return {"y": y}


def _exact_route(case, s, logits, scores):
    t, e, k = case["T"], case["E"], case["k"]
    biased = case["bias"]
    key = scores + s["balance"].double()[None] if biased else logits
    if case["groups"] > 1:
        grouped = (key if biased or case["top"] == 1 else scores).unflatten(1, (case["groups"], -1))
        value = grouped.topk(min(case["top"], grouped.shape[2]), dim=2).values.sum(2)
        # a group is kept if fewer than `kept` come before it
        ahead = (value[:, None, :] > value[:, :, None]) | \
                ((value[:, None, :] == value[:, :, None]) & torch.ones(case["groups"], case["groups"], device="cuda").tril(-1).bool())
        kept = ahead.sum(2) < case["kept"]
        key = torch.where(kept[:, :, None].expand_as(grouped).flatten(1), key, -math.inf)
    index = torch.empty(t, k, device="cuda", dtype=torch.long)
    left = key.clone()
    number = torch.arange(e, device="cuda")
    for j in range(k):  # the first of the largest that are left
        top = left.amax(1, keepdim=True)
        index[:, j] = torch.where(left == top, number, e).amin(1)
        left.scatter_(1, index[:, j:j + 1], -math.inf)
    weight = torch.take_along_dim(scores, index, 1)
    weight = case["scale"] * (weight / weight.sum(1, keepdim=True) if case["renorm"] else weight)
    flat = index.flatten()
    before = torch.zeros(e + 1, device="cuda", dtype=torch.long)
    before[1:] = torch.bincount(flat, minlength=e).cumsum(0)
    row = torch.argsort(flat * flat.numel() + torch.arange(flat.numel(), device="cuda"))
    return {"index": index.int(), "weight": weight, "offset": before.int(), "row": row.int(), "place": torch.argsort(row).int()}
