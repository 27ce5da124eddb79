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


def test_every_thread_that_initialises_barriers_fences():
    """fence.mbarrier_init covers its own thread's initialisations only: it stands
    in the block of all the initialisations of its kernel."""
    for name in FILES:
        code = text(name)
        for m in re.finditer(r"fence_barrier_init\(\);", code):
            before = code[:m.start()]
            assert before.rstrip()[-1] in "{};", (name, "a condition of the fence's own", before[-80:])
            # the innermost block around the fence holds every mbar_init of its kernel
            depth, at = 0, len(before)
            while depth < 1:
                at -= 1
                depth += {"{": 1, "}": -1}.get(code[at], 0)
            kernel = code[before.rfind("__global__"):m.start()]
            assert kernel.count("mbar_init(") == code[at:m.start()].count("mbar_init(") > 0, (name, kernel[:80])


def test_tensor_maps_are_prefetched_only_where_a_side_has_work():
    """A side without work (dH or dW not asked for) has no encoded maps, and
    prefetch.tensormap is defined on tensor maps only."""
    code = text("ce_kernel.cuh")
    calls = list(re.finditer(r"prefetch_tensormap\(&(.*?)\);", code))
    assert calls
    for m in calls:
        side = re.match(r"(p\.side\[\w+\]|\w+)\.", m.group(1)).group(1)
        assert re.search(re.escape(side) + r"\.tiles_m\b", code[m.start() - 200:m.start()]), m.group(0)
    # and every side of a launch is looked at
    assert not any("side[0]" in m.group(1) for m in calls)


def test_producers_fence_before_they_copy_what_stores_wrote():
    """The gathered H and the copies of W are written with ordinary stores and read
    by tensor copies in the kernel after, which belong to another proxy."""
    code = text("ce_kernel.cuh")
    producer = code[code.index("auto run_producer"):code.index("if (warp == 0 && lane == 0)")]
    assert "fence_proxy_async_global();" in producer[:producer.index("items.next(it)")]
    assert code.index("wait_for_previous_kernel();") < code.index("auto run_producer")
