"""Plain 64-bit forms of routing, grouped products, combining and adapters, and
the error bounds that follow from what the library rounds (test
infrastructure, torch float64)."""
import math

import torch

from head_reference import EPS32, HALF_ULP, TINY, assert_within, rows  # noqa: F401  (used by the tests)

DTYPES = [torch.float16, torch.bfloat16]


def code(tg, dtype):
    return {torch.float16: tg.TG_F16, torch.bfloat16: tg.TG_BF16, torch.float32: tg.TG_F32}[dtype]


def padded(gen, n, d, pad, dtype, scale=1.0):
    """n x d view of rows of whole 16-byte units plus `pad` elements; what is not of the view is NaN."""
    return rows(gen, n, d, (-d) % 8 + pad, dtype, scale)


def stacked(gen, g, n, d, pad, gap, dtype, scale=1.0):
    """g matrices of n x d, `gap` elements between them; what is not of the matrices is NaN."""
    ld = (d + 7) // 8 * 8 + pad
    stride = n * ld + gap
    flat = torch.full((g * stride,), float("nan"), dtype=dtype, device="cuda")
    view = flat.as_strided((g, n, d), (stride, ld, 1))
    view.copy_((torch.randn(g, n, d, generator=gen, device="cuda") * scale).to(dtype))
    return view


def offsets(counts):
    total, out = 0, [0]
    for c in counts:
        total += c
        out.append(total)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- routing

def route(logits, bias, k, sigmoid, groups, kept, top, renorm, scale):
    """index and weight as the documentation has them, expert by expert on the host in 64 bits."""
    t, e = logits.shape
    index = torch.full((t, k), -1, dtype=torch.int32)
    weight = torch.zeros(t, k, dtype=torch.float64)
    size = e // groups
    for r, row in enumerate(logits.double().cpu().tolist()):
        may = [x > -math.inf for x in row]
        finite = torch.tensor(row, dtype=torch.float64)
        if sigmoid:
            score = (1 / (1 + torch.exp(-finite))).tolist()
        else:
            big = max([x for x in row if x == x], default=-math.inf)
            p = torch.where(finite == big, 1.0, torch.exp(finite - big)).nan_to_num(nan=0.0)
            score = (p / p.sum()).tolist()
        b = bias.double().cpu().tolist() if bias is not None else [0.0] * e
        key = [score[i] + b[i] for i in range(e)] if bias is not None else row
        group_key = key if bias is not None or top == 1 else score
        ranks = []
        for g in range(groups):
            best = sorted([group_key[i] for i in range(g * size, (g + 1) * size) if may[i]], reverse=True)[:top]
            ranks.append((-sum(best) if best else math.inf, g))
        keep = {g for _, g in sorted(ranks)[:kept]}
        order = sorted([i for i in range(e) if may[i] and (groups == 1 or i // size in keep)], key=lambda i: (-key[i], i))[:k]
        if not order:
            continue
        chosen = torch.tensor([row[i] for i in order], dtype=torch.float64)
        if not sigmoid and any(x != x or x == math.inf for x in row):
            w = torch.full((len(order),), math.nan, dtype=torch.float64)
        elif renorm and sigmoid:  # without underflow
            logs = torch.nn.functional.logsigmoid(chosen)
            w = torch.softmax(logs, 0)
        elif renorm:
            w = torch.softmax(chosen, 0)
        else:
            w = torch.tensor([score[i] for i in order], dtype=torch.float64)
        index[r, :len(order)] = torch.tensor(order, dtype=torch.int32)
        weight[r, :len(order)] = w * scale
    return index.cuda(), weight.cuda()


def route_weights(logits, index, sigmoid, renorm, scale):
    """The weights of given experts, for differentiation."""
    score = torch.sigmoid(logits) if sigmoid else torch.softmax(logits, 1)
    there = index >= 0
    w = torch.where(there, score.gather(1, index.long().clamp(min=0)), torch.zeros((), dtype=torch.float64, device="cuda"))
    return scale * (w / w.sum(1, keepdim=True) if renorm else w)


def group_rows(index, g):
    flat = index.flatten().tolist()
    members = [[i for i, x in enumerate(flat) if x == q] for q in range(g)]
    row = [i for m in members for i in m]
    offset = [0]
    for m in members:
        offset.append(offset[-1] + len(m))
    place = [-1] * len(flat)
    for at, i in enumerate(row):
        place[i] = at
    row += [-1] * (len(flat) - len(row))
    return offset, row, place


# ------------------------------------------------------- grouped products

def source(x, row, per_row, lo, hi):
    """Rows lo .. hi-1 of a grouped product's operand, zeros for sources outside it."""
    if row is None:
        return x[lo:hi].double()
    r = row[lo:hi].long()
    at = torch.where(r < 0, -1, torch.div(r, per_row, rounding_mode="floor"))
    ok = (at >= 0) & (at < len(x))
    return torch.where(ok[:, None], x[at.clamp(0, len(x) - 1)].double(), torch.zeros((), dtype=torch.float64, device=x.device))


def product(a, b, dtype):
    """a @ b and its bound: products of 16-bit values are exact in fp32, the tensor
    core adds them 16 at a time, each time off by at most 2^-23 of the largest
    partial sum, which |a| @ |b| bounds; then one rounding."""
    y, mass = a @ b, a.abs() @ b.abs()
    return y, (a.shape[1] / 16 + 2) * 2 * EPS32 * mass, HALF_ULP[dtype]


def rounded(y, slack, dtype):
    """The bound of y rounded once, when it was off by slack before."""
    return slack + 1.01 * HALF_ULP[dtype] * (y.abs() + slack) + TINY[dtype]
