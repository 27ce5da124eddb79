"""A host thread whose first use of CUDA is a call of the library: the call is accepted,
and a refused call leaves the thread's current context as it was."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def in_a_new_thread(f):
    out = []
    t = threading.Thread(target=lambda: out.append(f()))
    t.start()
    t.join()
    assert len(out) == 1
    return out[0]


def calls(tg):
    """name: (call, output, what it is to be).  Small whole numbers, exact in 16 bits."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    whole = lambda *n: torch.randint(-2, 3, n, generator=gen, device="cuda").half()  # noqa: E731
    a, b = whole(64, 32), whole(32, 72)
    c, p = (torch.zeros(64, n, device="cuda", dtype=torch.float16) for n in (72, 32))
    y, place = whole(64, 32), torch.arange(64, device="cuda", dtype=torch.int32)
    s = torch.zeros(32, 32, device="cuda", dtype=torch.float16)
    return {
        "gemm": (lambda: tg.tg_gemm(64, 72, 32, a, 32, tg.TG_OP_N, b, 72, tg.TG_OP_N, c, 72, tg.TG_F16), c, a.float() @ b.float()),
        "pointwise": (lambda: tg.tg_pointwise(64, 32, a, 32, tg.TG_OP_N, p, 32, tg.TG_F16, tg.make_epilogue(relu=True)), p,
                      a.float().clamp(min=0.0)),
        "combine": (lambda: tg.tg_combine(32, 2, 32, y, 64, 32, place, None, s, 32, tg.TG_F16), s, y.float().view(32, 2, 32).sum(1)),
    }


@pytest.mark.parametrize("name", ["gemm", "pointwise", "combine"])
def test_first_call_of_a_thread(tg, name):
    call, out, want = calls(tg)[name]
    assert call() == tg.TG_OK  # what the library does once per process is done
    out.zero_()
    torch.cuda.synchronize()
    rc = in_a_new_thread(call)
    torch.cuda.synchronize()
    assert rc == tg.TG_OK, tg.tg_status_string(rc)
    assert torch.equal(out.float(), want)


def test_refused_call_keeps_the_threads_context(tg):
    """A thread that works in a context of its own still does after a host pointer was refused."""
    _, s, _ = calls(tg)["combine"]
    y, place = torch.zeros(64, 32, dtype=torch.float16), torch.arange(64, device="cuda", dtype=torch.int32)
    lib = ctypes.CDLL("libcuda.so.1")

    def work():
        mine, now = ctypes.c_void_p(), ctypes.c_void_p()
        assert lib.cuCtxCreate_v2(ctypes.byref(mine), ctypes.c_uint(0), ctypes.c_int(0)) == 0
        try:
            rc = tg.tg_combine(32, 2, 32, y, 64, 32, place, None, s, 32, tg.TG_F16)
            assert lib.cuCtxGetCurrent(ctypes.byref(now)) == 0
            return rc, now.value == mine.value
        finally:
            lib.cuCtxDestroy_v2(mine)

    rc, kept = in_a_new_thread(work)
    assert rc == tg.TG_ERR_POINTER and kept
