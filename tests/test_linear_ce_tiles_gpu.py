"""Linear cross entropy in the tiles, parts, pieces and splits that batches run,
against 64 bits.  Each case names the kernels it is there for, as the launches
of a captured call show them, so that another rule of dispatch cannot empty it."""
import ctypes
import math
import re

import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu

BOTH = [torch.float16, torch.bfloat16]
LSE, GRAD, PRODUCTS = 0, 1, 2


def problem(t, v, d, pad, dt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h, w = ref.rows(g, t, d, pad, dt), ref.rows(g, v, d, pad, dt, 2 / math.sqrt(d))
    target = torch.randint(0, v, (t,), device="cuda", generator=g)
    target[torch.rand(t, device="cuda", generator=g) < 0.2] = -100
    target[0], target[t - 1] = v - 1, 0
    return h, w, target, g


class Calls:
    def __init__(self, tg, h, w, target, dloss):
        self.tg, self.h, self.w, self.target, self.dloss = tg, h, w, target, dloss
        self.t, self.d, self.v = h.shape[0], h.shape[1], w.shape[0]
        self.code = tg.TG_BF16 if h.dtype == torch.bfloat16 else tg.TG_F16
        self.loss, self.lse = torch.empty(2, self.t, device="cuda").unbind(0)
        self.dh, self.dw = (torch.full(x.shape, 7.0, device="cuda", dtype=h.dtype) for x in (h, w))
        at = self.t, self.v, self.d, h, h.stride(0), w, w.stride(0)
        self.size = max(tg.tg_linear_ce_workspace_size(*at, self.code),
                        tg.tg_linear_ce_grad_workspace_size(*at, self.dh, self.d, self.dw, self.d, self.code))
        self.ws = torch.full((self.size,), 0xFF, dtype=torch.uint8, device="cuda")

    def forward(self):
        self.tg.linear_ce(self.t, self.v, self.d, self.h, self.h.stride(0), self.w, self.w.stride(0), self.target,
                          self.loss, self.lse, self.code, self.ws, self.size, torch.cuda.current_stream())

    def backward(self):
        self.tg.linear_ce_grad(self.t, self.v, self.d, self.h, self.h.stride(0), self.w, self.w.stride(0), self.target,
                               self.lse, self.dloss, self.dh, self.d, self.dw, self.d, self.code, self.ws, self.size,
                               torch.cuda.current_stream())

    def launched(self, tmp_path):
        """(mode, columns of a tile, pair, deep) of every product kernel."""
        graph = torch.cuda.CUDAGraph(keep_graph=True)
        with torch.cuda.graph(graph):
            self.forward()
            self.backward()
        path = str(tmp_path / "graph.dot")
        printed = ctypes.CDLL("libcuda.so.1").cuGraphDebugDotPrint
        printed.argtypes = ctypes.c_void_p, ctypes.c_char_p, ctypes.c_uint
        assert printed(graph.raw_cuda_graph(), path.encode(), 1) == 0
        with open(path) as f:
            names = re.findall(r"_ZN2tg9ce_kernelILi(\d)ELi(\d+)ELb([01])ELb([01])E", f.read())
        return [(int(m), int(bn), pair == "1", deep == "1") for m, bn, pair, deep in names]

    def checked(self, tmp_path, kernels, pieces=1):
        found = self.launched(tmp_path)
        assert set(found) == set(kernels)
        assert len({x[0] for x in found}) == 3
        self.ws.fill_(0xFF)
        self.forward()
        self.backward()
        torch.cuda.synchronize()
        st, detail = self.tg.tg_debug_status()
        assert st == self.tg.TG_OK, hex(detail)
        want_loss, want = ref.linear_ce(self.h, self.w, self.target)
        bound = ref.lse_bound(self.h, self.w, want)
        ref.assert_within(self.lse, want, bound, "lse")
        ref.assert_within(self.loss, want_loss, 2 * bound, "loss")
        del want_loss, bound
        # against the gradient at the exact lse: the one handed on is off by lse_bound,
        # which its slack has beside the logits'
        wh, ww, bh, bw = ref.linear_ce_grad(self.h, self.w, self.target, self.lse, self.dloss)
        ref.assert_within(self.dh, wh, bh, "dh")
        ref.assert_within(self.dw, ww, bw, "dw")
        return found


@pytest.mark.parametrize("dt", BOTH, ids=["f16", "bf16"])
@pytest.mark.parametrize("t,v,d,pad,kernels", [
    # pairs in every product: 9 K-blocks, ragged everything; a last part of one K-block; 33 K-blocks
    (300, 10001, 520, 8, [(LSE, 256, True, False), (GRAD, 256, True, False), (PRODUCTS, 256, True, False)]),
    (1100, 5003, 1032, 0, [(LSE, 256, True, True), (GRAD, 256, True, True), (PRODUCTS, 256, True, False)]),
    (520, 9800, 2112, 16, [(LSE, 256, True, True), (GRAD, 256, True, True), (PRODUCTS, 256, True, False)]),
    # rows that no tensor map describes
    (300, 10001, 1101, 0, [(LSE, 256, True, True), (GRAD, 256, True, True), (PRODUCTS, 256, True, False)]),
    # a narrow D: 128 columns on a pair
    (1500, 24000, 96, 0, [(LSE, 256, True, False), (GRAD, 256, True, False), (PRODUCTS, 128, True, False)]),
    # single CTAs, contractions in several parts
    (100, 1500, 4104, 0, [(LSE, 128, False, True), (GRAD, 128, False, True), (PRODUCTS, 128, False, False)]),
    (1, 3000, 8192, 0, [(LSE, 128, False, True), (GRAD, 128, False, True), (PRODUCTS, 128, False, False)]),
])
def test_against_64_bits(tg, tmp_path, t, v, d, pad, kernels, dt):
    h, w, target, g = problem(t, v, d, pad, dt, t + d)
    Calls(tg, h, w, target, torch.randn(t, device="cuda", generator=g)).checked(tmp_path, kernels)


@pytest.mark.parametrize("dt,pad", [(torch.float16, 0), (torch.bfloat16, 0), (torch.float16, 1)],
                         ids=["f16", "bf16", "f16-unaligned"])
def test_pieces_and_splits_together(tg, tmp_path, dt, pad):
    """G in two pieces of 65536 columns; 16 tiles of dH on 76 pairs, each
    piece's contraction in several splits that add to what the piece before left."""
    t, v, d = 4096, 131072, 256
    h, w, target, _ = problem(t, v, d, pad, dt, 5)
    c = Calls(tg, h, w, target, torch.full((t,), 64.0 / t, device="cuda"))
    found = c.checked(tmp_path, [(LSE, 256, True, False), (GRAD, 256, True, False), (PRODUCTS, 256, True, False)])
    assert [x[0] for x in found].count(GRAD) == 2
    # the planes of dH that the splits leave: more than one of T x D x 4 bytes
    one_piece_of_g, gathered = 4096 * 65536 * 2, t * d * 2
    copy_of_w = v * d * 2 if pad else 0
    planes = (c.size - one_piece_of_g - gathered * (2 if dt == torch.float16 else 1) - copy_of_w) / (t * d * 4)
    assert planes > 1.9, planes
