"""How the tensor-core kernels over an 8-bit cache end, read from their source: a wait that runs out there cannot be
caused without breaking them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_context_parallelism_gb300", "csrc")


def source(file):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())


def body(file, kernel):
    """The kernel's text without comments, from its name to the brace that closes it."""
    text = source(file)
    at = text.index("{", text.index(")", text.index(f" {kernel}(const __grid_constant__")))
    depth = 0
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[at:end + 1]


KERNELS = [("cache_q8_tc.cu", "q8_tc_kernel"), ("cache_q8_wide.cu", "q8_wide_kernel")]


@pytest.mark.parametrize("file,kernel", KERNELS)
def test_copies_land_after_every_role_is_done(file, kernel):
    """A role can give up on a copy whose producer has finished: only after the last barrier is it known whether one did,
    and only there does waiting for the copies keep the CTA's shared memory until they have landed."""
    text = body(file, kernel)
    assert text.count("mma_commit") > 3 and "tmem_dealloc" in text   # the whole kernel
    before, after = text[:text.rindex("__syncthreads();")], text[text.rindex("__syncthreads();"):]
    assert "if (*abort_flag" in after
    assert not re.search(r"if \([^)]*\*abort_flag", before), "tested before the other roles are done"
    assert "mbar_wait_landing(&bar.full[" in after
    assert "mbar_wait_landing(&bar.full[" not in before


@pytest.mark.parametrize("file,kernel", KERNELS)
def test_tensor_memory_is_written_before_it_is_freed(file, kernel):
    """The softmax role leaves its loop in the middle of a tile when it gives up: its stores end before the last barrier."""
    text = body(file, kernel)
    before = text[:text.rindex("__syncthreads();")]
    assert "tmem_wait_st();" in before[before.rindex("tc_fence_before();", 0, before.rindex("tc_fence_before();")):]


def test_softmax_warps_meet_the_same_number_of_times():
    """The few-rows kernel's softmax warps meet at a named barrier.  One that gave up a wait still comes there, so no path
    between two meetings leaves the loops but through one: the only exits are after a meeting that told all four."""
    text = body("cache_q8_tc.cu", "q8_tc_kernel")
    role = text[text.index("auto wait = [&](uint64_t* b"):text.rindex("__syncthreads();")]
    for m in re.finditer(r"\b(break|return|goto)\b", role):
        line_start = role.rindex("\n", 0, m.start())
        context = role[max(0, line_start - 160):m.end()]
        assert ("group_any(dead)" in context or "if (out) break" in context or "if (dead) return" in context), context[-200:]
    # a thread that is dead waits for nothing, and reads and writes no tensor memory
    assert "if (!dead && !warp_wait(b, parity, abort_flag, status, where)) dead = true;" in role
    assert role.count("warp_wait(") == 1


def test_kernels_that_start_early_promise_nothing_about_their_inputs():
    """They may run while the kernel before them still writes their inputs."""
    for file in ("cache_q8.cuh", "cache_q8_mma.cuh", "cache_q8_ops.cu", "cache_q8_simt.cu", "cache_q8_tc.cu",
                 "cache_q8_wide.cu", "cache_simt.cuh", "qk_norm_rope.cu"):
        text = source(file)
        assert "__restrict__" not in text and "__ldg" not in text and ".nc." not in text, file


def test_every_kernel_waits_for_the_one_before():
    """grid_dependency_wait() comes before the first access to global memory in every kernel of these files."""
    for file in ("cache_q8_ops.cu", "cache_q8_simt.cu", "cache_q8_tc.cu", "cache_q8_wide.cu", "qk_norm_rope.cu"):
        text = source(file)
        for m in re.finditer(r"__global__ void[^;{]*\{", text):
            part = text[m.end():m.end() + 6000]
            at = part.index("grid_dependency_wait();")
            head = part[:at]
            assert "find_range" not in head and "load(0)" not in head and "p.pages[" not in head, file
