"""Source guards of the output head's kernels (CPU only): rules of the memory
model that no run on one compiler can show to be broken."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tiled_gemm_layouts_gb300", "csrc")
FILES = ["ce.cu", "ce_kernel.cuh", "layernorm.cu"]


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# what one kernel of a call writes and a later one reads
HANDED_ON = ["live", "alpha", "token", "place", "row_scale", "row_target", "part", "hit", "planes"]


def test_no_read_only_load_of_what_the_kernel_before_writes():
    """A chained kernel is resident before its predecessor has written these:
    a load through the read-only path is defined only for memory that nobody
    writes during the kernel's life, and need not stay behind the wait."""
    names = "|".join(HANDED_ON)
    found = []
    for name in FILES:
        code = text(name)
        found += [f"{name}: {m}" for m in re.findall(rf"__ldg\(\s*&?(?:\w+(?:\.|->))?(?:{names})\b[^;]*", code)]
        found += [f"{name}: {m}" for m in re.findall(rf"const\s+\w+\s*\*\s*__restrict__\s+(?:{names})\b", code)]
    assert not found, found


def test_the_guard_above_sees_the_kernels():
    code = "".join(text(name) for name in FILES)
    for name in ("live", "alpha", "row_scale", "row_target", "part", "hit", "planes"):
        assert re.search(rf"\b{name}\b", code), name
    assert code.count("wait_for_previous_kernel();") >= 5
