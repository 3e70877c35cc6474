"""Every kernel that may be scheduled while the one before it drains waits for that one before it touches global memory:
read from each kernel's own body (CPU), and run behind a producer that lets its dependents start at once and writes their
inputs late (GPU)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300.build import ARCH, build, nvcc
from cache_cases import make_batch
from cache_q8_cases import Batch8
from head_norm_cases import make_case

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "ring_context_parallelism_gb300", "csrc")
FILES = ("cache_attn_simt.cu", "cache_attn_tc.cu", "cache_ops.cu", "cache_q8_ops.cu", "cache_q8_simt.cu", "cache_q8_tc.cu",
         "cache_q8_wide.cu", "key_mass_tc.cu", "qk_norm_rope.cu")
WAIT = "grid_dependency_wait();"
# how these kernels come to global memory: the batch's range and sequences, loads by name or through a cast pointer,
# copies, atomics, and the arguments' arrays by index
ACCESS = re.compile(r"find_range|load_seq|\bload\w*\(|\bload = |turns\.|reinterpret_cast<const (?!CUtensorMap)|tma_load|copy16|cp\.async|"
                    r"atomic\w*\(|\b(?:jobs|parts|stats|positions|inv_freq|kv_lens|row_offsets|pages|counts|mass|dst_start)\[")


def closing(text, at, pair):
    depth = 0
    for end in range(at, len(text)):
        depth += (text[end] == pair[0]) - (text[end] == pair[1])
        if depth == 0:
            return end
    raise AssertionError("unbalanced")


def kernels(text):
    """(name, body) of every kernel of a source text without comments."""
    text = re.sub(r"//[^\n]*", "", text)
    found = []
    for m in re.finditer(r"__global__ void\s+(?:__launch_bounds__\()?", text):
        at = m.end()
        if text[at - 1] == "(":
            at = closing(text, at - 1, "()") + 1
        name = re.match(r"\s*(\w+)\s*", text[at:])
        start = text.index("{", closing(text, at + name.end(), "()"))
        found.append((name.group(1), text[start:closing(text, start, "{}") + 1]))
    return found


def fault(body):
    """What is wrong with a kernel's waits, or None."""
    if body.count(WAIT) != 1:
        return f"{body.count(WAIT)} waits"
    first = ACCESS.search(body)
    if not first:
        return "no access found"
    if first.start() < body.index(WAIT):
        return f"{first.group(0)} ahead of the wait"
    return None


def source(file):
    return open(os.path.join(CSRC, file)).read()


@pytest.mark.parametrize("file", FILES)
def test_kernels_wait_before_their_first_access(file):
    text = source(file)
    found = kernels(text)
    assert len(found) == len(re.findall(r"__global__", re.sub(r"//[^\n]*", "", text)))
    for name, body in found:
        assert fault(body) is None, (file, name, fault(body))


@pytest.mark.parametrize("file", FILES)
def test_a_wait_that_is_missing_or_late_is_seen(file):
    """The check itself, on altered text: without the wait, and with it behind the statement of the first access."""
    for name, body in kernels(source(file)):
        without = body.replace(WAIT, "")
        assert fault(without) == "0 waits", name
        end = without.index(";", ACCESS.search(without).end()) + 1
        assert "ahead of the wait" in fault(without[:end] + WAIT + without[end:]), name


# ---------------------------------------------------------------------------
# on a GPU
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def late(tmp_path_factory):
    """late(pairs): on the current stream, a kernel that lets its dependents start at once, and some 100 us later copies
    every source to its destination."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    ra.load()
    out = str(tmp_path_factory.mktemp("late") / "late_writer.so")
    subprocess.run([nvcc(), *ARCH, "-O2", "-shared", "-Xcompiler", "-fPIC", "-o", out, os.path.join(HERE, "late_writer.cu")],
                   check=True, capture_output=True)
    fn = ctypes.CDLL(out).late_writes
    fn.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_size_t),
                   ctypes.c_uint, ctypes.c_void_p]

    def run(pairs):
        n = len(pairs)
        dst, src = ((ctypes.c_void_p * n)(*(p[i].data_ptr() for p in pairs)) for i in (0, 1))
        size = (ctypes.c_size_t * n)(*(p[0].numel() * p[0].element_size() for p in pairs))
        assert all(p[0].is_contiguous() and p[1].is_contiguous() and p[0].shape == p[1].shape for p in pairs)
        assert fn(n, dst, src, size, 100000, torch.cuda.current_stream().cuda_stream) == 0
    return run


def behind(late, call, old, new):
    """call on tensors that hold `old`, valid as they are, when it is launched, and `new` once the kernel before it is done:
    what it gives for `new`."""
    want = [t.clone() for t in call(*[t.clone() for t in new])]
    for _ in range(3):
        live = [t.clone() for t in old]
        torch.cuda.synchronize()
        late(list(zip(live, new)))
        got = call(*live)
        torch.cuda.synchronize()
        ra.device_status()
        for g, w in zip(got, want):
            g, w = (x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in (g, w))
            assert torch.equal(g, w)


BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_head_norm_and_gradient_behind_a_late_producer(late, dtype):
    old, new = (make_case((300,), 8, 2, 128, dtype, seed=s).cuda() for s in (1, 2))
    tensors = lambda c: [c.q, c.k, c.wq, c.wk, c.positions, c.inv_freq]  # noqa: E731
    behind(late, lambda *a: ra.qk_norm_rope(*a), tensors(old), tensors(new))
    behind(late, lambda *a: ra.qk_norm_rope_bwd(*a), [*tensors(old), old.gq, old.gk], [*tensors(new), new.gq, new.gk])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 4, 8, 40])
def test_attention_over_the_8_bit_cache_behind_a_late_producer(late, tokens, dtype):
    # the same sizes: offsets, pages and lengths are valid in both
    old, new = (Batch8([(900, tokens), (300, tokens)], 8, 2, 128, 16, dtype, seed=s).args() for s in (3, 4))
    behind(late, lambda *a: ra.tree_attn_q8(*a), list(old), list(new))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_8_bit_writes_and_reads_behind_a_late_producer(late, dtype):
    b = [Batch8([(200, 33), (90, 90)], 4, 4, 64, 8, dtype, seed=s) for s in (5, 6)]
    rows = [[torch.randn(123, 4, 64, generator=torch.Generator().manual_seed(10 * s + i)).to(dtype).cuda() for i in (0, 1)] for s in (5, 6)]

    def write(kr, vr, offs, k, v, ks, vs, pages, lens):
        ra.cache_append_q8(kr, vr, offs, k, v, ks, vs, pages, lens)
        return k, v, ks, vs
    args = [[*r, *x.args()[1:]] for r, x in zip(rows, b)]
    behind(late, write, *args)
    behind(late, lambda offs, *rest: ra.cache_read_q8(offs, 123, *rest, dtype=dtype), *[list(x.args()[1:]) for x in b])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("tokens", [1, 40])
def test_paged_batches_behind_a_late_producer(late, tokens, dtype):
    old, new = (make_batch([(900, tokens), (300, tokens)], 8, 2, 128, 16, dtype, seed=s).cuda() for s in (7, 8))
    both = [[c.q, c.offs, c.k_pages, c.v_pages, c.pages, c.lens] for c in (old, new)]
    behind(late, lambda *a: ra.tree_attn(*a), *both)
    lses = [ra.tree_attn(*x)[1] for x in both]

    def weights(q, lse, offs, k, pages, lens):
        out = torch.zeros(2, 2, 900, device="cuda")
        ra.key_mass(q, lse, offs, k, pages, lens, out)
        return (out,)
    mass = [[c.q, s, c.offs, c.k_pages, c.pages, c.lens] for c, s in zip((old, new), lses)]
    behind(late, weights, *mass)
    behind(late, lambda m, lens: ra.evict_select(m, lens, 128, 4, 8), *[[*weights(*m), m[-1]] for m in mass])

    def append(kr, vr, offs, k, v, pages, lens):
        ra.cache_append(kr, vr, offs, k, v, pages, lens)
        return k.nan_to_num(7.0), v.nan_to_num(7.0)
    R = 2 * tokens
    rows = [[torch.randn(R, 2, 128, generator=torch.Generator().manual_seed(20 * s + i)).to(dtype).cuda() for i in (0, 1)] for s in (7, 8)]
    behind(late, append, *[[*r, c.offs, c.k_pages, c.v_pages, c.pages, c.lens] for r, c in zip(rows, (old, new))])
