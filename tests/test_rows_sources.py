"""Source guards of routing, grouping, grouped products and adapters (CPU only):
rules that a run need not show to be broken."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_gemm_layouts_gb300", "csrc")
FILES = ["route.cu", "group_rows.cu", "combine.cu", "adapters.cu", "direct.cuh", "grouped_kernel.cuh", "grouped_few.cu"]
COLLECTIVE = r"(?:__shfl\w*_sync|__ballot_sync|__any_sync|__all_sync|__reduce_\w+_sync|warp_sum|warp_max|warp_min|warp_fmax|token_max|token_sum)"


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_collective_behind_a_condition_of_one_lane():
    """A warp's collective right of && or ||, or in a branch of ?:, is not reached by
    lanes whose left side decides: the others wait for them."""
    for name in FILES:
        code = text(name)
        found = [m.group(0) for m in re.finditer(r"(?:&&|\|\||\?|(?<!:):(?!:))\s*\(*!?" + COLLECTIVE + r"\s*(?:<[^>]*>)?\(", code)]
        # (the left side of these is the same for the whole warp)
        found = [f for f in found if f not in ("&& __any_sync(", "&& !__all_sync(")]
        assert not found, (name, found)
    uniform = re.findall(r"if \((\w+) && __any_sync", text("route.cu"))
    assert uniform == ["by_two_scores"]


def test_every_thread_that_initialises_barriers_fences():
    code = text("grouped_kernel.cuh")
    at = code.index("fence_barrier_init();")
    block = code[code.rindex("if (threadIdx.x == 0) {", 0, at):at]
    assert block.count("mbar_init(") == code.count("mbar_init(") > 0


def test_kernels_wait_before_they_read_what_the_kernel_before_wrote():
    """counts and totals (grouping) and the low-rank rows (adapters) are read behind the wait."""
    for name, kernel, words in (("group_rows.cu", "place_kernel(", ("counts[", "totals[")), ("group_rows.cu", "scan_kernel(", ("counts[",)),
                                ("adapters.cu", "add_kernel(", ("p.low",))):
        code = text(name)
        body = code[code.index(kernel):]
        wait = body.index("wait_for_previous_kernel();")
        for w in words:
            assert body.index(w, body.index("{")) > wait, (name, kernel, w)
        assert "__ldg(" not in code
