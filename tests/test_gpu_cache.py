"""GPU parity of the paged-cache operators against their 64-bit definitions, element by element, with
bounds that count roundings (cache_cases.py)."""
import math
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300 import ra as rab
from ring_context_parallelism_gb300.build import build
from cache_cases import attention, make_batch, mass, select

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    ra.load()


def within(got, want, bound, what):
    got, want = got.double().cpu(), want.cpu()
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {off[bad].max().item():.3e} "
                           f"where {bound[bad][off[bad].argmax()].item():.3e} is allowed; first at {bad.nonzero()[0].tolist()}")


def attend(b, **kw):
    c = b.cuda()
    out, lse = ra.tree_attn(c.q, c.offs, c.k_pages, c.v_pages, c.pages, c.lens, tree_mask=c.mask, **kw)
    ra.device_status()
    return out, lse


def check_attention(b):
    out, lse = attend(b)
    ref, ref_lse, e_out, e_lse = attention(b)
    within(out, ref, e_out, "out")
    within(lse, ref_lse, e_lse, "lse")


SEQS = {
    "one key": [(1, 1)],
    "no key": [(0, 1)],
    "no key at all": [(0, 0), (0, 2), (7, 0)],
    "one token": [(1000, 1)],
    "fewer keys than tokens": [(3, 5), (70, 71)],
    "only new tokens": [(64, 64), (1, 1), (129, 129)],
    "tile ends": [(63, 1), (64, 2), (65, 3), (127, 1), (128, 4), (129, 1), (191, 2), (192, 1), (193, 5)],
    "ragged": [(257, 33), (5, 1), (0, 0), (128, 1), (700, 17), (1, 1), (31, 8)],
    "long": [(20000, 1), (3, 1)],
}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", SEQS)
@pytest.mark.parametrize("mask", ["chain", "tree"])
def test_tree_attn_lengths(name, mask, dtype):
    check_attention(make_batch(SEQS[name], 8, 2, 128, 16, dtype, mask, seed=1))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 8, 64, 8), (32, 4, 128, 64), (14, 2, 64, 32), (5, 1, 128, 128),
                                           (128, 1, 64, 16), (12, 4, 128, 256), (66, 2, 128, 1024)])
@pytest.mark.parametrize("mask", ["chain", "random"])
def test_tree_attn_heads_and_pages(Hq, Hkv, D, page, mask, dtype):
    check_attention(make_batch([(300, 9), (40, 40), (130, 1)], Hq, Hkv, D, page, dtype, mask, seed=2))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mask", ["empty", "narrow", "random"])
def test_tree_attn_masks(mask, dtype):
    """Rows without a key (no earlier key, no bit set) give O = 0 and lse = -inf; columns the mask lacks are not seen."""
    check_attention(make_batch([(6, 6), (90, 20), (33, 33), (1, 1)], 8, 2, 64, 8, dtype, mask, seed=4))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_tree_attn_many_sequences(dtype):
    """More sequences than CTAs, most of them short; and page lists longer than needed."""
    g = torch.Generator().manual_seed(5)
    seqs = [(int(torch.randint(0, 90, (1,), generator=g)), int(torch.randint(0, 3, (1,), generator=g))) for _ in range(700)]
    check_attention(make_batch(seqs, 4, 2, 64, 16, dtype, "chain", seed=5, max_pages=40))


@pytest.mark.parametrize("keys", [64, 65, 128, 192, 256, 384])
def test_tree_attn_many_equal_sequences(keys):
    """Several units per CTA with whole tiles only: nothing but the pipeline's own waits orders them."""
    one = make_batch([(keys, 1)], 4, 2, 64, 64, BF16, seed=keys)
    ref, _, e_out, _ = attention(one)
    c = one.cuda()
    n = 1400
    out, _ = ra.tree_attn(c.q.expand(n, 4, 64).contiguous(), torch.arange(n + 1, dtype=torch.int32, device="cuda"), c.k_pages,
                          c.v_pages, c.pages.expand(n, -1).contiguous(), c.lens.expand(n).contiguous())
    ra.device_status()
    within(out, ref.expand(n, 4, 64), e_out.expand(n, 4, 64), "out")   # cut units round in another order


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_tree_attn_long_chain(dtype):
    """A chunk of a prompt: many row tiles, each with its own last visible key."""
    check_attention(make_batch([(500, 300), (90, 70)], 8, 2, 128, 16, dtype, "chain", seed=6))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_tree_attn_sharp_scores(dtype):
    """Scores of tens: the running maximum moves from tile to tile and across cut units."""
    check_attention(make_batch([(3000, 2), (900, 4)], 8, 2, 64, 16, dtype, "tree", seed=7, scale=8.0))


def test_tree_attn_repeats_and_options():
    """The same call gives the same bits, with or without lse, into given buffers and workspace, whatever they hold."""
    b = make_batch([(4000, 8), (900, 3), (17, 1)], 16, 2, 128, 16, BF16, "tree", seed=8)
    out, lse = attend(b)
    ws = torch.full((ra.tree_attn_workspace_size(b.q.shape[0], 3, 16, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    o2, l2 = torch.full_like(out, math.nan), torch.full_like(lse, math.nan)
    for _ in range(3):
        attend(b, out=o2, lse=l2, workspace=ws)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    o3, none = attend(b, want_lse=False)
    assert none is None and torch.equal(out, o3)


def test_tree_attn_refuses_on_the_device():
    """A bad page reads as zeros, a bad length or offset skips its sequence; each is reported, the rest is right."""
    b = make_batch([(200, 2), (100, 3), (50, 1)], 4, 2, 64, 16, BF16, seed=9)
    ref, _, e_out, _ = attention(b)
    c = b.cuda()
    for what in ("page", "page high", "length", "length negative", "offset"):
        pages, lens, offs = c.pages.clone(), c.lens.clone(), c.offs.clone()
        if what == "page":
            pages[1, 2] = -1
        elif what == "page high":
            pages[1, 0] = c.k_pages.shape[0]
        elif what == "length":
            lens[1] = pages.shape[1] * 16 + 1
        elif what == "length negative":
            lens[1] = -3
        else:
            offs[1], offs[2] = 5, 2
        out = torch.full_like(c.q, 7.0)
        ra.tree_attn(c.q, offs, c.k_pages, c.v_pages, pages, lens, out=out)
        with pytest.raises(ra.RAError) as e:
            ra.device_status()
        assert e.value.status == rab.RA_ERR_INVALID_ARG
        if what != "offset":
            within(out[[0, 1, 5]], ref[[0, 1, 5]], e_out[[0, 1, 5]], what)
        if what.startswith("length"):
            assert (out[2:5] == 7.0).all()
        ra.device_status()   # cleared


def test_tree_attn_in_a_graph():
    """Captured once, replayed on other lengths, pages and rows; two graphs with workspaces of their own."""
    big = make_batch([(1500, 4), (1500, 4)], 8, 2, 128, 16, BF16, seed=10)
    c = big.cuda()
    q, offs, pages, lens = c.q.clone(), c.offs.clone(), c.pages.clone(), c.lens.clone()
    out, lse = torch.empty_like(q), torch.empty(8, 8, device="cuda")
    ra.tree_attn(q, offs, c.k_pages, c.v_pages, pages, lens, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.tree_attn(q, offs, c.k_pages, c.v_pages, pages, lens, out=out, lse=lse)
    for seqs in ([(1500, 4), (1500, 4)], [(700, 1), (37, 7)], [(9, 8), (1400, 0)]):
        part = make_batch([(1500, 4), (1500, 4)], 8, 2, 128, 16, BF16, seed=10)
        part.offs = torch.tensor([0, seqs[0][1], seqs[0][1] + seqs[1][1]], dtype=torch.int32)
        part.lens = torch.tensor([s[0] for s in seqs], dtype=torch.int32)
        part.k = [k[:s[0]] for k, s in zip(part.k, seqs)]
        part.v = [v[:s[0]] for v, s in zip(part.v, seqs)]
        offs.copy_(part.offs)
        lens.copy_(part.lens)
        graph.replay()
        ra.device_status()
        ref, ref_lse, e_out, e_lse = attention(part)
        within(out, ref, e_out, "out")
        within(lse, ref_lse, e_lse, "lse")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_inputs_written_just_before_the_call(dtype):
    """Lengths, offsets, page lists and rows that the kernels before on the stream have just written, call after call
    without a wait: a launch that starts early may not read early."""
    batches = [make_batch(seqs, 8, 2, 128, 16, dtype, "chain", seed=13) for seqs in ([(900, 3), (40, 2)], [(64, 1), (700, 4)], [(5, 5), (300, 0)])]
    cs = [b.cuda() for b in batches]
    want = []
    for b, c in zip(batches, cs):
        o, l = attend(b)
        mo = torch.zeros(2, 2, 1000, device="cuda")
        ra.key_mass(c.q, l, c.offs, c.k_pages, c.pages, c.lens, mo)
        want.append((o, l, mo))
    R, P, N = 5, max(c.pages.shape[1] for c in cs), max(c.k_pages.shape[0] for c in cs)
    q, offs, lens = torch.zeros_like(cs[0].q), torch.zeros_like(cs[0].offs), torch.zeros_like(cs[0].lens)
    pages = torch.zeros(2, P, dtype=torch.int32, device="cuda")
    k, v = (torch.zeros(N, 16, 2, 128, dtype=dtype, device="cuda") for _ in range(2))
    big = torch.zeros(1 << 26, device="cuda")
    got = []
    for it in range(30):
        c = cs[it % 3]
        if it % 5 == 0:
            big.add_(1)   # a long kernel ahead
        n = c.q.shape[0]
        k[:c.k_pages.shape[0]].copy_(c.k_pages)
        v[:c.v_pages.shape[0]].copy_(c.v_pages)
        pages[:, :c.pages.shape[1]].copy_(c.pages)
        q[:n].copy_(c.q)
        offs.copy_(c.offs)
        lens.copy_(c.lens)
        o, l = ra.tree_attn(q[:n], offs, k, v, pages, lens)
        mo = torch.zeros(2, 2, 1000, device="cuda")
        ra.key_mass(q[:n], l, offs, k, pages, lens, mo)
        got.append((o, l, mo))
    ra.device_status()
    for it, (o, l, mo) in enumerate(got):
        a, b, c = want[it % 3]
        assert torch.equal(o, a) and torch.equal(l, b) and torch.equal(mo, c), it


def test_tree_attn_on_two_streams():
    batches = [make_batch([(3000, 8), (10, 2)], 16, 2, 128, 16, BF16, "tree", seed=s) for s in (11, 12)]
    want = [attend(b) for b in batches]
    cs = [b.cuda() for b in batches]
    streams = [torch.cuda.Stream() for _ in batches]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for c, st in zip(cs, streams):
            with torch.cuda.stream(st):
                got.append(ra.tree_attn(c.q, c.offs, c.k_pages, c.v_pages, c.pages, c.lens, tree_mask=c.mask))
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_tree_attn_from_two_threads():
    """Two threads, each on a stream of its own, call at the same time."""
    batches = [make_batch([(3000, 8), (10, 2)], 16, 2, 128, 16, BF16, "tree", seed=s) for s in (11, 12)]
    want = [attend(b) for b in batches]
    cs = [b.cuda() for b in batches]
    torch.cuda.synchronize()

    def run(c):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [ra.tree_attn(c.q, c.offs, c.k_pages, c.v_pages, c.pages, c.lens, tree_mask=c.mask) for _ in range(50)]
            torch.cuda.current_stream().synchronize()
        return got

    with ThreadPoolExecutor(2) as pool:
        for got, (out, lse) in zip(pool.map(run, cs), want):
            assert all(torch.equal(o, out) and torch.equal(l, lse) for o, l in got)
    ra.device_status()


def test_binding_refusals_and_given_tensors():
    """Refused on the host, before any launch; tensors that are given come back as the same objects."""
    b = make_batch([(40, 2)], 4, 2, 64, 8, BF16).cuda()
    args = (b.q, b.offs, b.k_pages, b.v_pages, b.pages, b.lens)
    out, lse = torch.empty_like(b.q), torch.empty(4, 2, device="cuda")
    got = ra.tree_attn(*args, out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    assert ra.tree_attn(*args, want_lse=False)[1] is None
    with pytest.raises(ValueError, match="CUDA"):
        ra.tree_attn(b.q, b.offs.cpu(), *args[2:])
    with pytest.raises(ValueError, match="contiguous"):
        ra.tree_attn(torch.cat([b.q, b.q], 2)[:, :, :64], *args[1:])
    with pytest.raises(ra.RAError) as e:
        ra.tree_attn(*args, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == rab.RA_ERR_WORKSPACE
    with pytest.raises(ra.RAError) as e:
        ra.tree_attn(b.q[:, :3].contiguous(), *args[1:])
    assert e.value.status == rab.RA_ERR_INVALID_ARG
    mass_rows = torch.zeros(1, 2, 42, device="cuda")
    kept = torch.empty(1, 2, 8, device="cuda")
    pos, counts, same = ra.evict_select(mass_rows, b.lens, 8, kept_mass=kept)
    assert same is kept and counts.tolist() == [8] and pos[0, 0].tolist() == list(range(8))
    with pytest.raises(ra.RAError, match="n_first"):
        ra.evict_select(mass_rows, b.lens, 8, n_first=5, n_recent=4)
    assert ra.cache_move(b.k_pages, b.v_pages, b.pages, b.pages, pos, counts) is None
    ra.device_status()


def test_device_status_reads_no_more_without_paged_batches():
    """A program that makes none of these calls pays for none of their status words: nine copies from the device take
    87 us, five 50; and the first call's refusal is still reported."""
    code = """
import time, torch, ring_context_parallelism_gb300 as ra
torch.zeros(1, device="cuda")
def cost():
    got = []
    for _ in range(9):
        a = time.perf_counter()
        for _ in range(100):
            ra.device_status()
        got.append(time.perf_counter() - a)
    return sorted(got)[4]
cost()
before = cost()
ra.evict_select(torch.rand(1, 1, 8, device="cuda"), torch.tensor([9], dtype=torch.int32, device="cuda"), 4)
try:
    ra.device_status()
    raise SystemExit("not reported")
except ra.RAError as e:
    assert "upkeep" in str(e), e
after = cost()
assert before < 0.75 * after, (before, after)
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


# ---------------------------------------------------------------------------
# gathered weight
# ---------------------------------------------------------------------------
def check_mass(b, decay=0.75, cols=None, with_in=True, in_place=False):
    _, lse, _, _ = attention(b)
    lse = lse.float()
    Hkv, n = b.k_pages.shape[2], len(b.k)
    cols = cols or max(1, int(b.lens.max()))
    g = torch.Generator().manual_seed(99)
    old = torch.rand(n, Hkv, cols, generator=g) if with_in else None
    want, err = mass(b, lse, old, decay, cols)
    c = b.cuda()
    out = old.cuda() if in_place else torch.full((n, Hkv, cols), math.nan, device="cuda")
    if in_place:
        want = torch.where(want.isnan(), old.double(), want)
    src = out if in_place else None if old is None else old.cuda()
    got = ra.key_mass(c.q, lse.cuda(), c.offs, c.k_pages, c.pages, c.lens, out, mass_in=src, decay=decay, tree_mask=c.mask)
    ra.device_status()
    assert got is out
    within(got, want, err, "mass")
    return got


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", SEQS)
@pytest.mark.parametrize("mask", ["chain", "tree"])
def test_key_mass_lengths(name, mask, dtype):
    check_mass(make_batch(SEQS[name], 8, 2, 128, 16, dtype, mask, seed=21), cols=max(1, max(k for k, _ in SEQS[name])) + 3)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 8, 64, 8), (32, 4, 128, 64), (14, 2, 64, 32), (128, 1, 128, 16), (66, 2, 128, 1024)])
def test_key_mass_heads_and_pages(Hq, Hkv, D, page, dtype):
    b = make_batch([(300, 9), (40, 40), (130, 1)], Hq, Hkv, D, page, dtype, "random", seed=22)
    check_mass(b, in_place=True)
    check_mass(b, with_in=False)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("mask", ["empty", "narrow"])
def test_key_mass_masks(mask, dtype):
    check_mass(make_batch([(6, 6), (90, 20), (33, 33), (1, 1)], 8, 2, 64, 8, dtype, mask, seed=23))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_key_mass_long_chain_and_many_sequences(dtype):
    check_mass(make_batch([(500, 300), (90, 70)], 8, 2, 128, 16, dtype, seed=24))
    g = torch.Generator().manual_seed(25)
    seqs = [(int(torch.randint(0, 90, (1,), generator=g)), int(torch.randint(0, 3, (1,), generator=g))) for _ in range(700)]
    check_mass(make_batch(seqs, 4, 2, 64, 16, dtype, "chain", seed=25))


@pytest.mark.parametrize("tokens", [1, 5, 9, 20, 40])
def test_key_mass_many_short_runs(tokens):
    """A CTA goes through many sequences and heads, of one, two and more row chunks, between chunks of any width."""
    seqs = [(tokens + 37 * (i % 7), max(0, tokens - i % 3)) for i in range(90)]
    check_mass(make_batch(seqs, 48, 6, 64, 16, BF16, "chain", seed=29))


@pytest.mark.parametrize("tokens,Hkv,mask,D", [(4, 1, "chain", 128), (4, 1, "tree", 64), (4, 3, "tree", 128),
                                               (12, 1, "tree", 128), (12, 3, "tree", 64), (12, 1, "chain", 64),
                                               (20, 1, "tree", 128), (20, 3, "tree", 128), (40, 1, "tree", 128),
                                               (40, 3, "chain", 64)])
def test_key_mass_runs_of_one_and_two_tiles(tokens, Hkv, mask, D):
    """Runs of two key tiles with an odd number of runs of one between them, in chunks of 32 rows (4 tokens) and of
    128 (one, two that stay, three streamed): the lse of a run stays until all of its rows are weighed."""
    seqs = [((250, 100)[i % 2], tokens) for i in range(600 if Hkv == 1 else 300)]
    check_mass(make_batch(seqs, 8 * Hkv, Hkv, D, 16, BF16, mask, seed=60 + tokens))


@pytest.mark.parametrize("Hq,Hkv,D,chunk", [(4, 1, 128, 32), (12, 3, 64, 32), (8, 1, 64, 16), (24, 3, 128, 16),
                                            (8, 1, 128, 4), (24, 3, 64, 4)])
def test_key_mass_runs_past_the_first_chunk(Hq, Hkv, D, chunk):
    """Chains of two row chunks whose last key tile only the second chunk sees, where runs start at that tile; for
    chunks of 32 rows next to single tokens, which keep the batch's mean low."""
    g = torch.Generator().manual_seed(61)
    seqs = []
    for i in range(120):
        n = int(torch.randint(chunk + 1, 2 * chunk, (1,), generator=g))
        last = 128 * int(torch.randint(1, 4, (1,), generator=g))
        seqs.append((last + int(torch.randint(1, n - chunk + 1, (1,), generator=g)), n))
        if chunk == 4:
            seqs.append((last + 60, 1))
    check_mass(make_batch(seqs, Hq, Hkv, D, 16, BF16, seed=62))


def test_key_mass_without_rows_decays():
    b = make_batch([(100, 0), (5, 0)], 4, 2, 64, 16, BF16, seed=26)
    check_mass(b, in_place=True, cols=128)


def test_key_mass_repeats():
    b = make_batch([(2000, 16), (700, 5)], 16, 2, 128, 16, BF16, "tree", seed=27)
    first = check_mass(b)
    assert torch.equal(first.nan_to_num(), check_mass(b).nan_to_num())


def test_key_mass_refuses_on_the_device():
    b = make_batch([(200, 2), (100, 3)], 4, 2, 64, 16, BF16, seed=28)
    c = b.cuda()
    lse = torch.zeros(4, 5, device="cuda")
    out = torch.full((2, 2, 199), 3.0, device="cuda")      # sequence 0 has more keys than columns
    ra.key_mass(c.q, lse, c.offs, c.k_pages, c.pages, c.lens, out)
    with pytest.raises(ra.RAError) as e:
        ra.device_status()
    assert e.value.status == rab.RA_ERR_INVALID_ARG
    assert (out[0] == 3.0).all() and (out[1, :, :100] != 3.0).any() and (out[1, :, 100:] == 3.0).all()
    pages = c.pages.clone()
    pages[1, 1] = 1 << 20
    ra.key_mass(c.q, lse, c.offs, c.k_pages, pages, c.lens, torch.empty(2, 2, 256, device="cuda"))
    with pytest.raises(ra.RAError):
        ra.device_status()


# ---------------------------------------------------------------------------
# choice, moves, writes
# ---------------------------------------------------------------------------
def special(n, H, cols, kind, seed):
    g = torch.Generator().manual_seed(seed)
    m = torch.rand(n, H, cols, generator=g)
    if kind == "ties":
        m = torch.floor(m * 4)
    elif kind == "zeros":
        m.zero_()
        m[..., ::2] = -0.0
    elif kind == "odd values":
        m = torch.randn(n, H, cols, generator=g)
        pick = torch.randint(0, 8, m.shape, generator=g)
        for i, x in enumerate((math.nan, math.inf, -math.inf, 1e-45, -1e-45)):
            m[pick == i] = x
    elif kind == "wide":
        m = torch.exp(40 * (m - 0.5))
    return m


@pytest.mark.parametrize("kind", ["plain", "ties", "zeros", "odd values", "wide"])
@pytest.mark.parametrize("lens,cols,budget,first,recent", [
    ([1], 1, 1, 0, 0), ([0, 1, 5], 8, 4, 1, 1), ([100, 64, 63, 65], 100, 64, 4, 16), ([2000, 1999, 3], 2048, 512, 0, 0),
    ([1500, 1025], 1600, 1024, 512, 512), ([5000], 5000, 1, 0, 0), ([5000], 5001, 4999, 4, 8), ([70, 71], 80, 16, 16, 0),
    ([33000, 9], 33000, 8000, 4, 100), ([140000], 140001, 5000, 3, 50), ([131072, 8193], 131072, 8192, 16, 1024)])
def test_evict_select(kind, lens, cols, budget, first, recent):
    m = special(len(lens), 2, cols, kind, seed=sum(lens))
    lens_t = torch.tensor(lens, dtype=torch.int32)
    want = select(m, lens_t, budget, first, recent)
    kept = torch.full((len(lens), 2, budget + 5), math.nan, device="cuda")
    pos, counts, got = ra.evict_select(m.cuda(), lens_t.cuda(), budget, first, recent, kept_mass=kept)
    ra.device_status()
    assert torch.equal(pos.cpu(), want[0]) and torch.equal(counts.cpu(), want[1])
    bits = got.cpu()[..., :budget].contiguous().view(torch.int32)
    assert torch.equal(bits, want[2].view(torch.int32)) and (got[..., budget:] == 0).all()


def test_evict_select_refuses_on_the_device():
    m = torch.rand(3, 2, 50, device="cuda")
    pos, counts, kept = ra.evict_select(m, torch.tensor([40, 51, -1], dtype=torch.int32, device="cuda"), 30, 2, 2)
    with pytest.raises(ra.RAError) as e:
        ra.device_status()
    assert e.value.status == rab.RA_ERR_INVALID_ARG
    assert counts.tolist() == [30, 0, 0] and (pos[1:] == -1).all() and (kept[1:] == 0).all() and (pos[0] >= 0).all()


def rows_of(pool, pages, page):
    """[sequences, keys, Hkv, D] through the page lists (CPU)."""
    j = torch.arange(pages.shape[1] * page)
    at = pages.long()[:, j // page] * page + j % page
    return pool.reshape(-1, *pool.shape[2:])[at]


def pool_of(n, Hkv, D, page, src, dst, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n_pages = n * (src + dst) + 1
    k, v = (torch.randn(n_pages, page, Hkv, D, generator=g).to(dtype) for _ in range(2))
    order = torch.randperm(n_pages, generator=g).to(torch.int32)
    return k, v, order[:n * src].reshape(n, src).contiguous(), order[n * src:n * (src + dst)].reshape(n, dst).contiguous(), g


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,Hkv,D,page,src,dst,heads,start", [(1, 1, 64, 8, 2, 2, 1, None), (3, 2, 128, 16, 7, 5, 2, None),
                                                              (2, 4, 64, 64, 4, 3, 1, [5, 64]), (5, 8, 128, 8, 40, 40, 8, None)])
def test_cache_move_to_other_pages(n, Hkv, D, page, src, dst, heads, start, dtype):
    k, v, sp, dp, g = pool_of(n, Hkv, D, page, src, dst, dtype, 31)
    first = start or [0] * n
    most = dst * page - max(first)
    pos = torch.randint(0, src * page, (n, heads, most), generator=g, dtype=torch.int32)   # any order, repeats too
    counts = torch.tensor([most + 3 if b == 0 else int(torch.randint(0, most + 1, (1,), generator=g)) for b in range(n)], dtype=torch.int32)
    want = []
    for pool in (k, v):
        w, old = pool.clone().reshape(-1, Hkv, D), rows_of(pool, sp, page)
        for b in range(n):
            for i in range(min(most, int(counts[b]))):
                slot = first[b] + i
                at = int(dp[b, slot // page]) * page + slot % page
                for h in range(Hkv):
                    w[at, h] = old[b, int(pos[b, h if heads > 1 else 0, i]), h]
        want.append(w.reshape(pool.shape))
    kc, vc = k.cuda(), v.cuda()
    ra.cache_move(kc, vc, sp.cuda(), dp.cuda(), pos.cuda(), counts.cuda(),
                  None if start is None else torch.tensor(start, dtype=torch.int32).cuda())
    ra.device_status()
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("n,Hkv,D,page,src,heads", [(1, 2, 64, 8, 3, 2), (4, 2, 128, 16, 20, 1), (2, 8, 64, 64, 30, 8)])
def test_cache_move_in_place(n, Hkv, D, page, src, heads, dtype):
    k, v, sp, _, g = pool_of(n, Hkv, D, page, src, 1, dtype, 32)
    keys = src * page
    start = [0 if b == 0 else int(torch.randint(0, keys // 2, (1,), generator=g)) for b in range(n)]
    most = keys // 2
    pos = torch.full((n, heads, most), -1, dtype=torch.int32)
    counts = torch.zeros(n, dtype=torch.int32)
    for b in range(n):
        counts[b] = most - b
        for h in range(heads):
            pick = torch.randperm(keys - start[b], generator=g)[:int(counts[b])].sort().values + start[b]
            pos[b, h, :int(counts[b])] = pick.to(torch.int32)
    want = []
    for pool in (k, v):
        w, old = pool.clone().reshape(-1, Hkv, D), rows_of(pool, sp, page)
        for b in range(n):
            for i in range(int(counts[b])):
                slot = start[b] + i
                for h in range(Hkv):
                    w[int(sp[b, slot // page]) * page + slot % page, h] = old[b, int(pos[b, h if heads > 1 else 0, i]), h]
        want.append(w.reshape(pool.shape))
    kc, vc, spc = k.cuda(), v.cuda(), sp.cuda()
    ra.cache_move(kc, vc, spc, spc, pos.cuda(), counts.cuda(), torch.tensor(start, dtype=torch.int32).cuda())
    ra.device_status()
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


@pytest.mark.parametrize("what", ["position", "negative position", "source page", "target page", "slot", "count", "start"])
@pytest.mark.parametrize("in_place", [False, True])
def test_cache_move_refuses_on_the_device(what, in_place):
    """What is out of range is not moved and reported; every other row is moved."""
    k, v, sp, dp, g = pool_of(2, 2, 64, 8, 4, 4, F32, 33)
    if in_place:
        dp = sp
    pos = torch.arange(0, 32, 2, dtype=torch.int32).reshape(1, 1, 16).repeat(2, 2, 1).contiguous()
    counts, start = torch.tensor([16, 16], dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    bad = []          # (sequence, slot) not written
    if what == "position":
        pos[1, :, 15] = 32
        bad = [(1, 15)]
    elif what == "negative position":
        pos[1, :, 0] = -1
        bad = [(1, 0)]
    elif what == "source page":
        sp = sp.clone()
        sp[1, 3] = 1000
        dp = sp if in_place else dp
        bad = [(1, i) for i in range(12, 16)]
    elif what == "target page":
        dp = dp.clone()
        dp[1, 1] = -2
        sp = dp if in_place else sp
        bad = [(1, i) for i in range(8, 16)] + ([(1, i) for i in range(4, 8)] if in_place else [])
    elif what == "slot":
        start[1] = 20
        if in_place:
            pos[1] = torch.arange(16, 32, dtype=torch.int32)   # below their slots: only what is out of range matters here
            start[1] = 32
        bad = [(1, i) for i in (range(16) if in_place else range(12, 16))]
    elif what == "count":
        counts[1] = -1
        bad = [(1, i) for i in range(16)]
    else:
        start[1] = -1
        bad = [(1, i) for i in range(16)]
    want = []
    for pool in (k, v):
        w, flat = pool.clone().reshape(-1, 2, 64), pool.reshape(-1, 2, 64)
        for b in range(2):
            for i in range(16):
                if (b, i) in bad:
                    continue
                slot, j = int(start[b]) + i, int(pos[b, 0, i])
                w[int(dp[b, slot // 8]) * 8 + slot % 8] = flat[int(sp[b, j // 8]) * 8 + j % 8]
        want.append(w.reshape(pool.shape))
    kc, vc, spc = k.cuda(), v.cuda(), sp.cuda()
    ra.cache_move(kc, vc, spc, spc if in_place else dp.cuda(), pos.cuda(), counts.cuda(), start.cuda())
    with pytest.raises(ra.RAError) as e:
        ra.device_status()
    assert e.value.status == rab.RA_ERR_INVALID_ARG
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("seqs,Hkv,D,page", [([(1, 1)], 1, 64, 8), ([(100, 3), (40, 40), (7, 0), (3, 5), (0, 2), (65, 1)], 2, 128, 16),
                                             ([(5000, 3000), (17, 16)], 8, 64, 64), ([(9, 1)] * 300, 3, 64, 8)])
def test_cache_append(seqs, Hkv, D, page, dtype):
    b = make_batch(seqs, Hkv, Hkv, D, page, dtype, seed=41)
    g = torch.Generator().manual_seed(42)
    R = int(b.offs[-1])
    kr, vr = (torch.randn(R, Hkv, D, generator=g).to(dtype) for _ in range(2))
    want = [b.k_pages.clone(), b.v_pages.clone()]
    for s, (kv, n) in enumerate(seqs):
        for t in range(n):
            j = kv - n + t
            if j >= 0:
                for w, r in zip(want, (kr, vr)):
                    w[int(b.pages[s, j // page]), j % page] = r[int(b.offs[s]) + t]
    c = b.cuda()
    ra.cache_append(kr.cuda(), vr.cuda(), c.offs, c.k_pages, c.v_pages, c.pages, c.lens)
    ra.device_status()
    for got, w in zip((c.k_pages, c.v_pages), want):
        assert torch.equal(got.cpu().nan_to_num(777.0), w.nan_to_num(777.0))


def test_cache_append_refuses_on_the_device():
    b = make_batch([(20, 2), (30, 3), (9, 1)], 2, 2, 64, 8, F32, seed=43)
    c = b.cuda()
    rows = torch.ones(6, 2, 64, device="cuda")
    for what in ("page", "length", "offset"):
        pages, lens, offs = c.pages.clone(), c.lens.clone(), c.offs.clone()
        if what == "page":
            pages[1, 3] = -1
        elif what == "length":
            lens[1] = 33
        else:
            offs[1] = 9
        k, v = c.k_pages.clone(), c.v_pages.clone()
        ra.cache_append(rows, rows, offs, k, v, pages, lens)
        with pytest.raises(ra.RAError):
            ra.device_status()
        last = int(c.pages[2, 1])
        assert (k[last, 0] == 1).all() and (v[last, 0] == 1).all()   # sequence 2 is written
        changed = (k != c.k_pages) & ~(k.isnan() & c.k_pages.isnan())
        keep = torch.ones(k.shape[0], dtype=torch.bool, device="cuda")
        keep[last] = False
        keep[c.pages[0, 2].long()] = False
        assert not changed[keep].any() or what == "page" and not changed[c.pages[1, 3].long()].any()


@pytest.mark.parametrize("what,skipped", [("page", [1]), ("high page", [1]), ("length", [1]), ("offset", [0, 1])])
def test_cache_append_writes_nothing_else_when_it_refuses(what, skipped):
    """Both pools hold the rows of the sequences that are right and are otherwise as they were."""
    seqs = [(20, 2), (30, 3), (9, 1)]
    b = make_batch(seqs, 2, 2, 64, 8, F32, seed=44)
    g = torch.Generator().manual_seed(45)
    kr, vr = (torch.randn(6, 2, 64, generator=g) for _ in range(2))
    want = [b.k_pages.clone(), b.v_pages.clone()]
    for s, (kv, n) in enumerate(seqs):
        for t in range(n if s not in skipped else 0):
            j = kv - n + t
            for w, r in zip(want, (kr, vr)):
                w[int(b.pages[s, j // 8]), j % 8] = r[int(b.offs[s]) + t]
    c = b.cuda()
    if what == "page":
        c.pages[1, 3] = -1
    elif what == "high page":
        c.pages[1, 3] = c.k_pages.shape[0]
    elif what == "length":
        c.lens[1] = 33
    else:
        c.offs[1] = 9
    ra.cache_append(kr.cuda(), vr.cuda(), c.offs, c.k_pages, c.v_pages, c.pages, c.lens)
    with pytest.raises(ra.RAError) as e:
        ra.device_status()
    assert e.value.status == rab.RA_ERR_INVALID_ARG
    for got, w in zip((c.k_pages, c.v_pages), want):
        assert torch.equal(got.cpu().nan_to_num(777.0), w.nan_to_num(777.0))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_pages_past_32_bit_offsets(dtype):
    """Pools of more than 2^32 bytes and 2^31 elements, the pages in use at their end."""
    Hq, Hkv, D, page = 16, 8, 128, 16
    b = make_batch([(300, 5), (70, 1)], Hq, Hkv, D, page, dtype, "tree", seed=71)
    used, total = b.k_pages.shape[0], (1 << 21) // page + 64
    lo = total - used
    c = b.cuda()
    c.pages = torch.where(c.pages >= 0, c.pages + lo, c.pages)
    pools = []
    for small in (c.k_pages, c.v_pages):
        pool = torch.empty(total, page, Hkv, D, dtype=dtype, device="cuda")
        pool[lo - 64:] = math.nan
        pool[lo:] = small
        pools.append(pool)
    k, v = pools
    rows = [torch.cat([x[-n:] for x, n in zip(xs, (5, 1))]).cuda() for xs in (b.k, b.v)]
    for s, (kv, n) in enumerate([(300, 5), (70, 1)]):
        for j in range(kv - n, kv):
            k[int(c.pages[s, j // page]), j % page] = v[int(c.pages[s, j // page]), j % page] = math.nan
    ra.cache_append(*rows, c.offs, k, v, c.pages, c.lens)
    out, lse = ra.tree_attn(c.q, c.offs, k, v, c.pages, c.lens, tree_mask=c.mask)
    ref, ref_lse, e_out, e_lse = attention(b)
    within(out, ref, e_out, "out")
    within(lse, ref_lse, e_lse, "lse")
    m = torch.zeros(2, Hkv, 300, device="cuda")
    ra.key_mass(c.q, lse, c.offs, k, c.pages, c.lens, m, tree_mask=c.mask)
    want, err = mass(b, lse.cpu(), None, 1.0, 300)
    within(m, torch.where(want.isnan(), torch.zeros_like(want), want), err, "mass")
    dst = (lo - 8 + torch.arange(8, dtype=torch.int32, device="cuda")).reshape(2, 4)
    pos, counts, _ = ra.evict_select(m, c.lens, 64, 2, 8)
    ra.cache_move(k, v, c.pages, dst, pos, counts)
    ra.device_status()
    for s, n in enumerate((64, 64)):
        for h in range(Hkv):
            keep = pos[s, h, :n].cpu().long()
            for pool, src in ((k, b.k), (v, b.v)):
                assert torch.equal(pool[dst[s].long()].reshape(-1, Hkv, D)[:n, h].cpu(), src[s][keep, h])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_a_serving_round(dtype):
    """Drafts written, verified, the accepted path kept, weights gathered, the cache cut to its budget in other
    pages, the next token attended: each step against the definition on what the steps before left."""
    Hq, Hkv, D, page, budget = 8, 2, 64, 8, 60
    n_ctx, n_draft = [90, 41, 70], [6, 5, 6]
    seqs = [(c + d, d) for c, d in zip(n_ctx, n_draft)]
    b = make_batch(seqs, Hq, Hkv, D, page, dtype, "tree", seed=51, max_pages=16)
    n = len(seqs)
    extra = -(-(budget + 1) // page)
    grow = torch.full((n * extra, page, Hkv, D), math.nan, dtype=dtype)
    first_new = b.k_pages.shape[0]
    b.k_pages, b.v_pages = torch.cat([b.k_pages, grow]), torch.cat([b.v_pages, grow])
    dst = (first_new + torch.arange(n * extra, dtype=torch.int32)).reshape(n, extra)
    c = b.cuda()
    # the drafts' rows are written by append: blank them first
    rows_k = torch.cat([k[ctx:] for k, ctx in zip(b.k, n_ctx)])
    rows_v = torch.cat([v[ctx:] for v, ctx in zip(b.v, n_ctx)])
    for s in range(n):
        for j in range(n_ctx[s], seqs[s][0]):
            c.k_pages[int(b.pages[s, j // page]), j % page] = math.nan
            c.v_pages[int(b.pages[s, j // page]), j % page] = math.nan
    ra.cache_append(rows_k.cuda(), rows_v.cuda(), c.offs, c.k_pages, c.v_pages, c.pages, c.lens)
    out, lse = ra.tree_attn(c.q, c.offs, c.k_pages, c.v_pages, c.pages, c.lens, tree_mask=c.mask)
    ra.device_status()
    ref, ref_lse, e_out, e_lse = attention(b)
    within(out, ref, e_out, "verify")
    within(lse, ref_lse, e_lse, "verify lse")
    # accept the path to the last draft of each tree
    paths = [b.mask[int(b.offs[s + 1]) - 1, :n_draft[s]].nonzero()[:, 0] for s in range(n)]
    most = max(len(p) for p in paths)
    pos = torch.full((n, 1, most), -1, dtype=torch.int32)
    for s, p in enumerate(paths):
        pos[s, 0, :len(p)] = (p + n_ctx[s]).to(torch.int32)
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32)
    start = torch.tensor(n_ctx, dtype=torch.int32)
    ra.cache_move(c.k_pages, c.v_pages, c.pages, c.pages, pos.cuda(), counts.cuda(), start.cuda())
    # the accepted tokens as a chain: their weights
    rows = torch.cat([p + int(b.offs[s]) for s, p in enumerate(paths)])
    lens = start + counts
    chain = make_batch([(int(l), int(k)) for l, k in zip(lens, counts)], Hq, Hkv, D, page, dtype, seed=52)
    chain.q, chain.mask = b.q[rows], None
    chain.k = [torch.cat([k[:ctx], k[ctx:][p]]) for k, ctx, p in zip(b.k, n_ctx, paths)]
    chain.v = [torch.cat([v[:ctx], v[ctx:][p]]) for v, ctx, p in zip(b.v, n_ctx, paths)]
    old = torch.rand(n, Hkv, 128, generator=torch.Generator().manual_seed(53))
    got = old.cuda()
    lse_rows = lse[:, rows.cuda()].contiguous()
    ra.key_mass(chain.q.cuda(), lse_rows, chain.offs.cuda(), c.k_pages, c.pages, lens.cuda(), got, mass_in=got, decay=0.5)
    ra.device_status()
    want, err = mass(chain, lse_rows.cpu(), old, 0.5, 128)
    within(got, torch.where(want.isnan(), old.double(), want), err, "mass")
    # to the budget, in other pages
    positions, kept, _ = ra.evict_select(got, lens.cuda(), budget, 2, 8)
    want_pos, want_counts, _ = select(got.cpu(), lens, budget, 2, 8)
    assert torch.equal(positions.cpu(), want_pos) and torch.equal(kept.cpu(), want_counts)
    ra.cache_move(c.k_pages, c.v_pages, c.pages, dst.cuda(), positions, kept)
    # the next token
    g = torch.Generator().manual_seed(54)
    nk, nv = (torch.randn(n, Hkv, D, generator=g).to(dtype) for _ in range(2))
    q = torch.randn(n, Hq, D, generator=g).to(dtype)
    one = torch.arange(n + 1, dtype=torch.int32)
    now = want_counts + 1
    ra.cache_append(nk.cuda(), nv.cuda(), one.cuda(), c.k_pages, c.v_pages, dst.cuda(), now.cuda())
    out, _ = ra.tree_attn(q.cuda(), one.cuda(), c.k_pages, c.v_pages, dst.cuda(), now.cuda())
    ra.device_status()
    last = make_batch([(int(x), 1) for x in now], Hq, Hkv, D, page, dtype, seed=55)
    last.q = q
    for s in range(n):
        keep = want_pos[s, :, :int(want_counts[s])].long()
        for lst, src, new in ((last.k, chain.k, nk), (last.v, chain.v, nv)):
            per_head = torch.stack([src[s][keep[h], h] for h in range(Hkv)], 1)
            lst[s] = torch.cat([per_head, new[s][None]])
    ref, _, e_out, _ = attention(last)
    within(out, ref, e_out, "decode after eviction")
