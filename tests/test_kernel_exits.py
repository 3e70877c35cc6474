"""How the tensor-core kernels over paged sequences end, read from their source: a wait that runs out there cannot be
caused without breaking them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ring_context_parallelism_gb300", "csrc")


def body(file, kernel):
    """The kernel's text without comments, from its name to the brace that closes it."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
    at = text.index("{", text.index(")", text.index(f" {kernel}(const __grid_constant__")))
    depth = 0
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return text[at:end + 1]


KERNELS = [("cache_attn_tc.cu", "tree_tc_kernel", ("full[ring]", "q_full")),
           ("key_mass_tc.cu", "mass_tc_kernel", ("k_full", "q_full"))]


@pytest.mark.parametrize("file,kernel,copies", KERNELS)
def test_copies_land_after_every_role_is_done(file, kernel, copies):
    """A role can give up on a copy whose producer has finished: only after the last barrier is it known whether one
    did, and only there does waiting for the copies keep the CTA's shared memory until they have landed."""
    text = body(file, kernel)
    assert text.count("griddepcontrol") == 0 and text.count("mma_commit") > 3   # the whole kernel
    before, after = text[:text.rindex("__syncthreads();")], text[text.rindex("__syncthreads();"):]
    assert "if (*abort_flag" in after
    assert not re.search(r"if \([^)]*\*abort_flag", before), "tested before the other roles are done"
    for bar in copies:
        assert f"mbar_wait_landing(&bar.{bar}" in after, bar
        assert f"mbar_wait_landing(&bar.{bar}" not in before, bar


def test_tensor_memory_is_written_before_it_is_freed():
    """The softmax role leaves its loop in the middle of a tile when it gives up: its stores end before the last barrier."""
    text = body("cache_attn_tc.cu", "tree_tc_kernel")
    before = text[:text.rindex("__syncthreads();")]
    loop_end = before.rindex("if (mine) tiles += T;")
    assert "tmem_wait_st();" in before[loop_end:]


def test_kernels_that_start_early_promise_nothing_about_their_inputs():
    """They may run while the kernel before them still writes their inputs: `__restrict__` on these, or a load that
    needs memory nobody writes, would allow reads that a wait for that kernel does not order."""
    for file in ("cache_attn_simt.cu", "cache_attn_tc.cu", "cache_batch.cuh", "cache_ops.cu", "key_mass_tc.cu", "mass_walk.h"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, file)).read())
        assert "__restrict__" not in text and "__ldg" not in text and ".nc." not in text, file
