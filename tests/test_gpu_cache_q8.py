"""GPU parity of the 8-bit cache -- write, read, attention -- against its 64-bit definitions (cache_q8_cases.py)."""
import math
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300 import ra as rab
from ring_context_parallelism_gb300.build import build
from cache_cases import make_batch
from cache_q8_cases import E4M3, Batch8, attention_q8, codes, scale_bytes, value

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


# ---------------------------------------------------------------------------
# write and read
# ---------------------------------------------------------------------------
def rows_of(R, Hkv, D, dtype, seed):
    """Rows of every kind: ordinary, with channels far larger, zero, tiny, huge, on ties, at the scale's borders."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, Hkv, D, generator=g)
    x[..., ::37] *= 30
    kind = torch.randint(0, 12, (R, Hkv), generator=g)
    x[kind == 0] = 0.0
    x[kind == 1] *= 1e-39
    x[kind == 2] *= 1e36
    ties = (torch.randint(16, 32, (R, Hkv, D), generator=g) + 0.5) * 2.0 ** torch.randint(-12, 4, (R, Hkv, D), generator=g)
    x = torch.where((kind == 3)[..., None], ties, x)
    border = 448.0 * 2.0 ** torch.randint(-20, 20, (R, Hkv), generator=g)
    for k, f in ((4, 1.0), (5, 1 + 2.0 ** -7), (6, 1 - 2.0 ** -8)):
        x = torch.where((kind == k)[..., None], x.clamp(-0.9, 0.9) * border[..., None], x)
        x[..., D // 2] = torch.where(kind == k, border * f, x[..., D // 2])
    x[kind == 7] = -x[kind == 7].abs()
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("seqs,Hkv,D,page", [
    ([(1, 1)], 1, 64, 8), ([(40, 40), (7, 3), (0, 0), (100, 1)], 2, 128, 16), ([(3, 5), (0, 2), (9, 9)], 3, 64, 8),
    ([(300, 300), (1000, 77)], 8, 128, 64), ([(50, 20)] * 90, 5, 64, 32), ([(5000, 1)], 4, 128, 1024)])
def test_append_and_read(seqs, Hkv, D, page, dtype):
    b = make_batch(seqs, Hkv, Hkv, D, page, F32, seed=1)
    R = b.q.shape[0]
    rows = [rows_of(R, Hkv, D, dtype, s) for s in (2, 3)]
    g = torch.Generator().manual_seed(4)
    n = b.k_pages.shape[0]
    pools = [torch.randint(0, 127, (n, page, Hkv, D), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randint(1, 250, (n, Hkv, page), generator=g, dtype=torch.uint8) for _ in range(2)]
    dev = [p.clone().view(E4M3).cuda() for p in pools] + [s.clone().cuda() for s in scales]
    offs, pages, lens = b.offs.cuda(), b.pages.cuda(), b.lens.cuda()
    ra.cache_append_q8(rows[0].cuda(), rows[1].cuda(), offs, *dev, pages, lens)
    ra.device_status()
    back = [torch.zeros(R, Hkv, D, dtype=torch.float64) for _ in range(2)]
    for t in range(2):
        e = scale_bytes(rows[t])
        c = codes(rows[t], e)
        for s, (kv, m) in enumerate(seqs):
            for i in range(m):
                r, j = int(b.offs[s]) + i, kv - m + i
                if j >= 0:
                    pg = int(b.pages[s, j // page])
                    pools[t][pg, j % page] = c[r]
                    scales[t][pg, :, j % page] = e[r]
                    back[t][r] = value(c[r], e[r])
    for got, want in zip(dev, pools + scales):   # whole pools: nothing else is written
        assert torch.equal(got.view(torch.uint8).cpu(), want)
    for out in (BF16, F32):
        for got, want in zip(ra.cache_read_q8(offs, R, *dev, pages, lens, dtype=out), back):
            assert got.dtype == out
            fits = (want.abs() >= 2.0 ** -126) | (want == 0)   # a smaller one may not be held exactly
            off = (got.double().cpu() - want).abs()
            assert (off[fits] == 0).all() and (off <= 2.0 ** -126).all()
    ra.device_status()


def test_append_of_values_that_are_not_numbers():
    b = make_batch([(8, 8)], 2, 2, 64, 8, F32, seed=1)
    x = torch.ones(8, 2, 64)
    x[1, 0, 3], x[2, 1, 7], x[3, 0, 9] = math.nan, math.inf, -math.inf
    dev = [torch.zeros(b.k_pages.shape, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.zeros(b.k_pages.shape[0], 2, 8, dtype=torch.uint8, device="cuda") for _ in range(2)]
    offs, pages, lens = b.offs.cuda(), b.pages.cuda(), b.lens.cuda()
    ra.cache_append_q8(x.cuda(), x.cuda(), offs, *dev, *scales, pages, lens)
    k, v = (t.cpu() for t in ra.cache_read_q8(offs, 8, *dev, *scales, pages, lens, dtype=F32))
    ra.device_status()
    assert torch.equal(k.nan_to_num(7.0), v.nan_to_num(7.0))
    assert k[1, 0, 3].isnan() and k[2, 1, 7] == math.inf and k[3, 0, 9] == -math.inf
    for r, h, d in ((1, 0, 3), (2, 1, 7), (3, 0, 9)):
        rest = k[r, h].clone()
        rest[d] = 0
        assert (rest == 0).all()
        k[r, h] = 1
    assert (k == 1).all()


@pytest.mark.parametrize("what", ["page", "page high", "length", "offset"])
def test_append_and_read_refuse_on_the_device(what):
    """A bad page's rows are not written and read as zeros, a bad sequence is skipped; each is reported, the rest is right."""
    b = make_batch([(40, 5), (60, 50), (30, 4)], 2, 2, 64, 16, F32, seed=5)
    R = b.q.shape[0]
    x = torch.randn(R, 2, 64).bfloat16()
    e = scale_bytes(x)
    good = value(codes(x, e), e)
    offs, pages, lens = b.offs.clone(), b.pages.clone(), b.lens.clone()
    if what == "page":
        pages[1, 2] = -1
    elif what == "page high":
        pages[1, 2] = b.k_pages.shape[0]
    elif what == "length":
        lens[1] = pages.shape[1] * 16 + 1
    else:
        offs[1], offs[2] = 50, 5
    pools = [torch.zeros(b.k_pages.shape, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.ones(b.k_pages.shape[0], 2, 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    args = (offs.cuda(), *pools, *scales, pages.cuda(), lens.cuda())
    ra.cache_append_q8(x.cuda(), x.cuda(), *args)
    with pytest.raises(ra.RAError) as err:
        ra.device_status()
    assert err.value.status == rab.RA_ERR_INVALID_ARG
    k, v = torch.full((R, 2, 64), 9.0, device="cuda"), torch.full((R, 2, 64), 9.0, device="cuda")
    got = ra.cache_read_q8(args[0], R, *args[1:], dtype=F32, k_rows=k, v_rows=v)
    assert got[0] is k and got[1] is v
    with pytest.raises(ra.RAError):
        ra.device_status()
    ra.device_status()   # cleared
    same = torch.equal(k, v)
    k = k.double().cpu()
    if what != "offset":   # there two sequences own some rows: K's may be one's and V's the other's
        assert same and torch.equal(k[:5], good[:5]) and torch.equal(k[55:], good[55:])
    if what.startswith("page"):
        at = torch.arange(10, 60)   # keys of the second sequence's rows
        bad = (at // 16 == 2)
        assert (k[5:55][bad] == 0).all() and torch.equal(k[5:55][~bad], good[5:55][~bad])
    if what == "length":
        assert (k[5:55] == 9.0).all()
        for s in scales:
            for pg in b.pages[1].tolist():
                assert (s[pg] == 1).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attend(b8, **kw):
    out, lse = ra.tree_attn_q8(*b8.args(), tree_mask=b8.mask(), **kw)
    ra.device_status()
    return out, lse


def check_attention(b8):
    out, lse = attend(b8)
    ref, ref_lse, e_out, e_lse = attention_q8(b8)
    within(lse, ref_lse, e_lse, "lse")
    within(out, ref, e_out, "out")


SEQS = {
    "one key": [(1, 1)],
    "no key": [(0, 1)],
    "no key at all": [(0, 0), (0, 2), (7, 0)],
    "one token": [(1000, 1)],
    "fewer keys than tokens": [(3, 5), (70, 71)],
    "only new tokens": [(64, 64), (1, 1), (129, 129)],
    "tile ends": [(63, 1), (64, 2), (65, 3), (127, 1), (128, 4), (129, 1), (191, 2), (255, 1), (256, 5), (257, 1)],
    "ragged": [(257, 33), (5, 1), (0, 0), (128, 1), (700, 17), (1, 1), (31, 8)],
    "long": [(20000, 1), (3, 1)],
}


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", SEQS)
@pytest.mark.parametrize("mask", ["chain", "tree"])
def test_lengths(name, mask, dtype):
    check_attention(Batch8(SEQS[name], 8, 2, 128, 16, dtype, mask, seed=1))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 8, 64, 8), (32, 4, 128, 64), (14, 2, 64, 32), (5, 1, 128, 128),
                                           (128, 1, 64, 16), (12, 4, 128, 256), (66, 2, 128, 1024), (7, 1, 128, 8)])
@pytest.mark.parametrize("mask", ["chain", "random"])
def test_heads_and_pages(Hq, Hkv, D, page, mask, dtype):
    check_attention(Batch8([(300, 9), (40, 40), (130, 1)], Hq, Hkv, D, page, dtype, mask, seed=2))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D", [(2, 2, 128), (8, 2, 64), (16, 2, 128), (64, 2, 64)])
@pytest.mark.parametrize("tokens", [1, 4, 7, 16, 33])
def test_rows_of_a_sequence(tokens, Hq, Hkv, D, dtype):
    """From one row to hundreds: each way of cutting them into tiles."""
    check_attention(Batch8([(500, tokens), (140, tokens)], Hq, Hkv, D, 16, dtype, "tree", seed=tokens))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("mask", ["empty", "narrow", "random"])
def test_masks(mask, dtype):
    """Rows without a key (no earlier key, no bit set) give O = 0 and lse = -inf; columns the mask lacks are not seen."""
    check_attention(Batch8([(6, 6), (90, 20), (33, 33), (1, 1), (200, 130)], 8, 2, 64, 8, dtype, mask, seed=4))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_many_sequences(dtype):
    g = torch.Generator().manual_seed(5)
    seqs = [(int(torch.randint(0, 200, (1,), generator=g)), int(torch.randint(0, 3, (1,), generator=g))) for _ in range(700)]
    check_attention(Batch8(seqs, 4, 2, 64, 16, dtype, "chain", seed=5, max_pages=40))


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 128), (12, 3, 64), (16, 2, 128)])
def test_few_rows_on_the_mean(Hq, Hkv, D):
    """The cut goes by the mean: one sequence of many rows among decodes, in many units of 8 or 16."""
    check_attention(Batch8([(300, 1)] * 30 + [(400, 41)] + [(777, 1)] * 9, Hq, Hkv, D, 16, BF16, "tree", seed=14))


@pytest.mark.parametrize("keys", [128, 129, 256, 384, 640])
@pytest.mark.parametrize("tokens", [1, 8, 20])
def test_many_equal_sequences(keys, tokens):
    """Several units per CTA with whole tiles only: nothing but the pipeline's own waits orders them."""
    one = Batch8([(keys, tokens)], 8, 2, 64, 64, BF16, seed=keys)
    ref, _, e_out, _ = attention_q8(one)
    q, offs, *pools, pages, lens = one.args()
    n = 700
    out, _ = ra.tree_attn_q8(q.repeat(n, 1, 1), torch.arange(n + 1, dtype=torch.int32, device="cuda") * tokens, *pools,
                             pages.expand(n, -1).contiguous(), lens.expand(n).contiguous())
    ra.device_status()
    within(out, ref.repeat(n, 1, 1), e_out.repeat(n, 1, 1), "out")


@pytest.mark.parametrize("tokens", [1, 20, 140])
@pytest.mark.parametrize("Hkv", [3, 155, 307])
def test_more_heads_than_ctas(Hkv, tokens):
    """Heads that do not divide the CTAs, and more heads than CTAs: a column of heads may end past the last."""
    check_attention(Batch8([(150, tokens), (145, tokens)], Hkv, Hkv, 64, 16, BF16, "chain", seed=Hkv))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_long_chain(dtype):
    check_attention(Batch8([(500, 300), (90, 70)], 8, 2, 128, 16, dtype, "chain", seed=6))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 6, 40])
def test_rows_behind_the_last_sequence(tokens, dtype):
    """A batch padded to a fixed number of rows: a last sequence without keys owns them.  Rows that no sequence owns are
    refused with the sequence before them (row_offsets end with R): both are left as they were, the rest is right."""
    b = Batch8([(300, tokens), (90, 1), (17, tokens)], 16, 2, 128, 16, dtype, "tree", seed=12)
    ref, ref_lse, e_out, e_lse = attention_q8(b)
    q, offs, *pools, pages, lens = b.args()
    R, more = q.shape[0], 37
    pad = lambda t, v, n=more: torch.cat([t, torch.full((n, *t.shape[1:]), v, dtype=t.dtype, device="cuda")])  # noqa: E731
    mask = pad(b.mask(), True)

    def call(offs, pages, lens):
        out, lse = torch.full((R + more, 16, 128), 9.0, dtype=dtype, device="cuda"), torch.full((16, R + more), 9.0, device="cuda")
        ra.tree_attn_q8(pad(q, math.nan), offs, *pools, pages, lens, tree_mask=mask, out=out, lse=lse)
        rows = [torch.full((R + more, 2, 128), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
        ra.cache_read_q8(offs, R + more, *pools, pages, lens, dtype=dtype, k_rows=rows[0], v_rows=rows[1])
        before = [p.view(torch.uint8).clone() for p in pools]
        new = [torch.cat([r[:R].nan_to_num(0.0), r[R:] * math.nan]) for r in rows]
        ra.cache_append_q8(*new, offs, *pools, pages, lens)   # what was read: the same values
        again = ra.cache_read_q8(offs, R + more, *pools, pages, lens, dtype=dtype, k_rows=torch.full_like(rows[0], 9.0),
                                 v_rows=torch.full_like(rows[1], 9.0))
        assert all(torch.equal(x, y) for x, y in zip(again, rows))
        used = sorted(set(b.base.pages.flatten().tolist()) - {-7})
        for x, y in zip(pools, before):   # pages of no sequence are as they were
            x = x.view(torch.uint8).clone()
            x[used] = y[used]
            assert torch.equal(x, y)
        return out, lse, rows

    out, lse, rows = call(pad(offs, R + more, 1), pad(pages, 0, 1), pad(lens, 0, 1))
    ra.device_status()
    within(out[:R], ref, e_out, "out")
    within(lse[:, :R], ref_lse, e_lse, "lse")
    assert (out[R:] == 0).all() and (lse[:, R:] == -math.inf).all() and all((r[R:] == 0).all() for r in rows)
    for s, n in enumerate((tokens, 1, tokens)):
        at, kv = int(b.base.offs[s]) + n, b.k[s].shape[0]
        m = min(n, kv)
        assert torch.equal(rows[0][at - m:at].double().cpu(), b.k[s][kv - m:])
        assert torch.equal(rows[1][at - m:at].double().cpu(), b.v[s][kv - m:])
    out, lse, rows = call(offs, pages, lens)
    for _ in range(2):   # one record of the writes and reads, one of the attention
        with pytest.raises(ra.RAError) as err:
            ra.device_status()
        assert err.value.status == rab.RA_ERR_INVALID_ARG
    ra.device_status()
    last = int(b.base.offs[2])
    within(out[:last], ref[:last], e_out[:last], "out")
    within(lse[:, :last], ref_lse[:, :last], e_lse[:, :last], "lse")
    assert (out[last:] == 9).all() and (lse[:, last:] == 9).all() and all((r[last:] == 9).all() for r in rows)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 12, 40])
def test_pages_listed_more_than_once(tokens, dtype):
    """Two sequences on the same first pages, one of which is listed twice in one of them."""
    b = Batch8([(330, tokens), (280, tokens), (170, 1)], 16, 2, 64, 32, dtype, "chain", seed=13)
    pages = b.base.pages
    for s, i, s0, i0 in ((1, 0, 0, 0), (1, 1, 0, 1), (2, 0, 0, 0), (2, 2, 0, 0)):
        pages[s, i] = pages[s0, i0]
        for rows in (b.k, b.v):
            rows[s][32 * i:32 * i + 32] = rows[s0][32 * i0:32 * i0 + 32]
    check_attention(b)
    q, offs, *pools, pages, lens = b.args()
    ends = torch.tensor([0, 330, 610, 780], dtype=torch.int32, device="cuda")
    for got, want in zip(ra.cache_read_q8(ends, 780, *pools, pages, lens, dtype=dtype), (b.k, b.v)):
        assert torch.equal(got.double().cpu(), torch.cat(want))
    ra.device_status()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_sharp_scores(dtype):
    """Scores of tens: the running maximum moves from tile to tile and across cut units."""
    check_attention(Batch8([(3000, 2), (900, 4), (1500, 20)], 8, 2, 64, 16, dtype, "tree", seed=7, scale=8.0))


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 12])
def test_scales_far_apart(dtype, tokens):
    """Keys and values whose scales lie many powers of two apart, rows of zeros among them, queries of unlike sizes."""
    def edit(b):
        g = torch.Generator().manual_seed(9)
        for s in range(len(b.k)):
            n = b.k[s].shape[0]
            b.v[s] *= torch.exp2(torch.randint(-30, 12, (n, 1, 1), generator=g).float())
            b.k[s] *= torch.exp2(torch.randint(-12, 2, (n, 1, 1), generator=g).float())
            b.v[s][::7] = 0
            b.k[s][::11] = 0
        b.q *= torch.exp2(torch.randint(-20, 2, (*b.q.shape[:2], 1), generator=g).float()).to(b.q.dtype)
        b.q[0, 0] = 0
        b.q[-1, 1, ::2] *= 2.0 ** -9
    check_attention(Batch8([(2000, tokens), (300, tokens)], 8, 2, 128, 16, dtype, "chain", seed=9, edit=edit))


@pytest.mark.parametrize("tokens", [1, 12])
def test_one_key_above_many_equal_ones(tokens):
    """One key of weight near one half, the rest shared by thousands of equal ones: their weights must not vanish."""
    def edit(b):
        for s in range(len(b.k)):
            b.k[s][1:] = 0
            b.k[s][0] = 1.0
            b.v[s][1:] = 1.0
            b.v[s][0] = -1.0
        b.q[:] = math.log(16000) / math.sqrt(128)   # its score: log of their number
    check_attention(Batch8([(16000, tokens)], 8, 2, 128, 64, BF16, "chain", seed=10, edit=edit))


def test_values_that_are_not_numbers():
    """A query that is none reaches its own row, and no other."""
    b8 = Batch8([(300, 4), (200, 2)], 8, 2, 128, 16, BF16, "chain", seed=11)
    ref, ref_lse, e_out, e_lse = attention_q8(b8)
    args = list(b8.args())
    args[0][1, 3, 7], args[0][2, 5, 0] = math.nan, math.inf
    out, lse = ra.tree_attn_q8(*args)
    ra.device_status()
    assert out[1, 3].isnan().all() and out[2, 5].isnan().all()
    ok = torch.ones(out.shape[:2], dtype=torch.bool)
    ok[1, 3] = ok[2, 5] = False
    within(out.cpu()[ok], ref[ok], e_out[ok], "out")
    within(lse.cpu().T[ok], ref_lse.T[ok], e_lse.T[ok], "lse")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 3, 8])
def test_repeats_and_options(dtype, tokens):
    """The same call gives the same bits, with or without lse, into given buffers and workspace, whatever they hold."""
    b = Batch8([(4000, tokens), (900, 3), (17, 1)], 16, 2, 128, 16, dtype, "tree", seed=8)
    out, lse = attend(b)
    ws = torch.full((ra.tree_attn_q8_workspace_size(out.shape[0], 3, 16, 2, 128, dtype),), 255, dtype=torch.uint8, device="cuda")
    o2, l2 = torch.full_like(out, math.nan), torch.full_like(lse, math.nan)
    for _ in range(3):
        got = attend(b, out=o2, lse=l2, workspace=ws)
        assert got[0] is o2 and got[1] is l2 and torch.equal(out, o2) and torch.equal(lse, l2)
    o3, none = attend(b, want_lse=False)
    assert none is None and torch.equal(out, o3)
    with pytest.raises(ra.RAError) as e:
        attend(b, workspace=ws[:256])
    assert e.value.status == rab.RA_ERR_WORKSPACE


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_refuses_on_the_device(dtype):
    """A bad page reads as zeros, a bad length or offset skips its sequence; each is reported, the rest is right."""
    b = Batch8([(200, 2), (100, 3), (50, 1)], 4, 2, 64, 16, dtype, seed=9)
    ref, _, e_out, _ = attention_q8(b)
    q, offs0, *pools, pages0, lens0 = b.args()
    for what in ("page", "page high", "length", "length negative", "offset"):
        pages, lens, offs = pages0.clone(), lens0.clone(), offs0.clone()
        if what == "page":
            pages[1, 2] = -1
        elif what == "page high":
            pages[1, 0] = pools[0].shape[0]
        elif what == "length":
            lens[1] = pages.shape[1] * 16 + 1
        elif what == "length negative":
            lens[1] = -3
        else:
            offs[1], offs[2] = 5, 2
        out = torch.full_like(q, 7.0)
        ra.tree_attn_q8(q, offs, *pools, pages, lens, out=out)
        with pytest.raises(ra.RAError) as e:
            ra.device_status()
        assert e.value.status == rab.RA_ERR_INVALID_ARG
        if what != "offset":
            within(out[[0, 1, 5]], ref[[0, 1, 5]], e_out[[0, 1, 5]], what)
        if what.startswith("length"):
            assert (out[2:5] == 7.0).all()
        ra.device_status()   # cleared
    # keys of a bad page: zeros, as keys and as values
    pages = pages0.clone()
    pages[1, 2] = -1
    out, lse = ra.tree_attn_q8(q, offs0, *pools, pages, lens0)
    with pytest.raises(ra.RAError):
        ra.device_status()
    b.base.k[1][32:48] = 0
    b.base.v[1][32:48] = 0
    ref, ref_lse, e_out, e_lse = attention_q8(b)
    within(out, ref, e_out, "out")
    within(lse, ref_lse, e_lse, "lse")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_in_a_graph(dtype):
    """Captured once, replayed on other lengths, offsets and rows."""
    seqs0 = [(1500, 4), (1500, 4)]
    big = Batch8(seqs0, 8, 2, 128, 16, dtype, seed=10)
    q, offs, *pools, pages, lens = big.args()
    out, lse = torch.empty_like(q), torch.empty(8, 8, device="cuda")
    ra.tree_attn_q8(q, offs, *pools, pages, lens, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra.tree_attn_q8(q, offs, *pools, pages, lens, out=out, lse=lse)
    for seqs in (seqs0, [(700, 1), (37, 7)], [(9, 8), (1400, 0)]):
        part = Batch8(seqs0, 8, 2, 128, 16, dtype, seed=10)
        p = part.base
        p.offs = torch.tensor([0, seqs[0][1], seqs[0][1] + seqs[1][1]], dtype=torch.int32)
        p.lens = torch.tensor([s[0] for s in seqs], dtype=torch.int32)
        p.k = [k[:s[0]] for k, s in zip(p.k, seqs)]
        p.v = [v[:s[0]] for v, s in zip(p.v, seqs)]
        offs.copy_(p.offs)
        lens.copy_(p.lens)
        graph.replay()
        ra.device_status()
        ref, ref_lse, e_out, e_lse = attention_q8(part)
        within(out, ref, e_out, "out")
        within(lse, ref_lse, e_lse, "lse")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_decode_loop_without_waits(dtype):
    """Norm and rotation, write, attention and read call after call on one stream, each on what the one before has just
    written; replayed from a graph; the results are those of the same calls with a wait between them."""
    b = Batch8([(900, 3), (40, 2), (130, 1)], 8, 2, 128, 16, dtype, seed=13)
    q, offs, *pools, pages, lens = b.args()
    g = torch.Generator().manual_seed(14)
    qkv = torch.randn(6, 12, 128, generator=g).to(dtype).cuda()
    w = [(1 + 0.1 * torch.randn(128, generator=g)).to(dtype).cuda() for _ in range(2)]
    freq = (1e4 ** (-torch.arange(64).double() / 64)).float().cuda()
    pos = torch.tensor([897, 898, 899, 38, 39, 129], dtype=torch.int32, device="cuda")
    big = torch.zeros(1 << 26, device="cuda")

    def step(wait):
        hold = torch.cuda.synchronize if wait else lambda: None
        qn, kn = ra.qk_norm_rope(qkv[:, :8], qkv[:, 8:10], *w, pos, freq)
        hold()
        ra.cache_append_q8(kn, qkv[:, 10:].contiguous(), offs, *pools, pages, lens)
        hold()
        out, lse = ra.tree_attn_q8(qn, offs, *pools, pages, lens)
        hold()
        k, v = ra.cache_read_q8(offs, 6, *pools, pages, lens, dtype=dtype)
        hold()
        return out, lse, k, v

    first = qkv.clone()
    want = []
    for i in range(3):
        qkv.copy_(first * (i + 1) + i)
        want.append([t.clone() for t in step(True)])
    got = []
    for it in range(15):
        if it % 4 == 0:
            big.add_(1)
        i = it % 3
        qkv.copy_(first * (i + 1) + i)
        got.append([t.clone() for t in step(False)])
    ra.device_status()
    for it, g3 in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g3, want[it % 3])), it
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(False)
    for i in (1, 2, 0):
        qkv.copy_(first * (i + 1) + i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want[i])), i


def test_on_two_streams_and_threads():
    batches = [Batch8([(3000, 8), (10, 2)], 16, 2, 128, 16, BF16, "tree", seed=s) for s in (11, 12)]
    want = [attend(b) for b in batches]
    args = [(b.args(), b.mask()) for b in batches]
    torch.cuda.synchronize()

    def run(a):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [ra.tree_attn_q8(*a[0], tree_mask=a[1]) for _ in range(30)]
            torch.cuda.current_stream().synchronize()
        return got

    with ThreadPoolExecutor(2) as pool:
        for got, (out, lse) in zip(pool.map(run, args), want):
            assert all(torch.equal(o, out) and torch.equal(l, lse) for o, l in got)
    ra.device_status()


def test_against_the_cache_in_16_bits():
    """The codes' values in bf16 pools, through tree_attn: the same attention, off by both calls' bounds."""
    b8 = Batch8([(700, 5), (64, 3), (2000, 1)], 16, 4, 128, 32, BF16, "tree", seed=15)
    out, lse = attend(b8)
    q, offs, *pools, pages, lens = b8.args()
    n, page, Hkv, D = pools[0].shape
    dense = [torch.ldexp(p.float(), s.transpose(1, 2).int()[..., None] - 127).bfloat16() for p, s in zip(pools[:2], pools[2:])]
    o16, l16 = ra.tree_attn(q, offs, *dense, pages, lens, tree_mask=b8.mask())
    ra.device_status()
    _, _, e_out, e_lse = attention_q8(b8)
    within(out, o16.double(), 2 * e_out, "out")
    within(lse, l16.double(), 2 * e_lse, "lse")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_pages_past_32_bit_offsets(dtype):
    """Pools of more than 2^32 bytes: one sequence on their last pages, one on their first."""
    b = Batch8([(300, 2), (150, 9)], 8, 2, 128, 64, dtype, seed=16)
    ref, ref_lse, e_out, e_lse = attention_q8(b)
    n = (1 << 32) // (64 * 2 * 128) + 512
    q, offs, k, v, ks, vs, pages, lens = b.args()
    m = k.shape[0]
    pools = []
    for p in (k, v):
        t = torch.empty((n, 64, 2, 128), dtype=torch.uint8, device="cuda")
        t[-m:] = p.view(torch.uint8)
        pools.append(t.view(E4M3))
    scales = []
    for s in (ks, vs):
        t = torch.zeros((n, 2, 64), dtype=torch.uint8, device="cuda")
        t[-m:] = s
        scales.append(t)
    pages = torch.where(pages >= 0, pages + (n - m), pages)
    out, lse = ra.tree_attn_q8(q, offs, *pools, *scales, pages, lens)
    ra.device_status()
    within(out, ref, e_out, "out")
    within(lse, ref_lse, e_lse, "lse")
    rows = torch.randn(q.shape[0], 2, 128).cuda()
    ra.cache_append_q8(rows, -rows, offs, *pools, *scales, pages, lens)
    kr, vr = ra.cache_read_q8(offs, q.shape[0], *pools, *scales, pages, lens, dtype=F32)
    ra.device_status()
    e = scale_bytes(rows.cpu())
    assert torch.equal(kr.double().cpu(), value(codes(rows.cpu(), e), e)) and torch.equal(kr, -vr)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_a_drafted_tree_round(dtype):
    """As a server uses them: a tree's rows normed, rotated, written and attended; the accepted path's rows appended again
    behind the context; the next token attends to exactly those."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    b = Batch8([(200, 6), (75, 6)], Hq, Hkv, D, page, dtype, "tree", seed=17, max_pages=20)
    q, offs, *pools, pages, lens = b.args()
    g = torch.Generator().manual_seed(18)
    qkv = torch.randn(12, Hq + 2 * Hkv, D, generator=g).to(dtype).cuda()
    w = [(1 + 0.1 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]
    freq = (1e4 ** (-torch.arange(D // 2).double() / (D // 2))).float().cuda()
    mask = b.base.mask
    depth = torch.cat([mask[s * 6:(s + 1) * 6, :6].sum(1) - 1 for s in range(2)])
    ctx = torch.tensor([194, 69]).repeat_interleave(6)
    qn, kn = ra.qk_norm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], *w, (ctx + depth).int().cuda(), freq)
    vn = qkv[:, Hq + Hkv:].contiguous()
    ra.cache_append_q8(kn, vn, offs, *pools, pages, lens)
    # what the definition says is in the cache now
    for s in range(2):
        for rows, dense in ((kn, b.base.k), (vn, b.base.v)):
            r = rows[s * 6:(s + 1) * 6].cpu()
            e = scale_bytes(r)
            dense[s][-6:] = value(codes(r, e), e)
    b.base.q = qn.cpu()
    out, lse = ra.tree_attn_q8(qn, offs, *pools, pages, lens, tree_mask=mask.cuda())
    ra.device_status()
    ref, ref_lse, e_out, e_lse = attention_q8(b)
    within(out, ref, e_out, "tree")
    within(lse, ref_lse, e_lse, "tree lse")
    paths = [mask[s * 6 + 5, :6].nonzero()[:, 0] for s in range(2)]   # the path to the last token is accepted
    n_acc = [len(p) for p in paths]
    take = torch.cat([p + 6 * s for s, p in enumerate(paths)]).cuda()
    lens2 = torch.tensor([194 + n_acc[0], 69 + n_acc[1]], dtype=torch.int32, device="cuda")
    offs2 = torch.tensor([0, n_acc[0], sum(n_acc)], dtype=torch.int32, device="cuda")
    ra.cache_append_q8(kn[take].contiguous(), vn[take].contiguous(), offs2, *pools, pages, lens2)
    # the last accepted token attends again, as a single token over the kept path
    last = torch.tensor([5, 11])
    out2, _ = ra.tree_attn_q8(qn[last.cuda()].contiguous(), torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), *pools,
                              pages, lens2)
    ra.device_status()
    b.base.q, b.base.mask = b.base.q[last], None
    b.base.offs, b.base.lens = torch.tensor([0, 1, 2], dtype=torch.int32), lens2.cpu()
    for s in range(2):
        for dense in (b.base.k, b.base.v):
            dense[s] = torch.cat([dense[s][:-6], dense[s][-6:][paths[s]]])
    ref2, _, e_out2, _ = attention_q8(b)
    within(out2, ref2, e_out2, "kept path")
    within(out2, ref[last], e_out2 + e_out[last], "the same keys in another order of pages")
