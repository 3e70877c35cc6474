"""Attention over the 8-bit cache where weights, and the scales of values, lie far apart: what is small adds up to what
it should, what is hidden takes nothing with it, and rows that are not numbers say so."""
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300.build import build
from cache_cases import attention, make_batch, visible
from cache_q8_cases import Batch8

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
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {(off / bound)[bad].max().item():.3g} times "
                           f"the bound; first at {bad.nonzero()[0].tolist()}")


def definition(b8):
    """(out, lse, their bounds).  Relative to the sizes that a row adds up, A = sum p |v|, never to the largest value of a
    sequence:
      each weight: one rounding of its own (attention()'s, 2^-8 in bf16), the scores' roundings, and exponents that hold the
        sum of a score and a scale's exponent (at most 2^8: 2^-17, its exponential 2^-17 of the weight);
      queries in two 8-bit parts leave out 2^-17 of the row's largest;
      a weight times its value's scale has a least step, 2^-28 of the row's largest such product, which a code of at most
        448 multiplies; 448 scales are at most twice the largest value of the key: n 2^-27 max (p |v|) for n keys."""
    b = b8.base
    out, lse, e_out, e_lse = attention(b)
    if b.q.dtype != BF16:
        return out, lse, e_out, e_lse
    R, Hq, D = b.q.shape
    G = Hq // b.k_pages.shape[2]
    for s in range(len(b.k)):
        lo, hi = int(b.offs[s]), int(b.offs[s + 1])
        see = visible(b, s)
        n, kv = see.shape
        if not n or not kv:
            continue
        for h in range(Hq):
            q, k, v = b.q[lo:hi, h].double(), b.k[s][:, h // G].double(), b.v[s][:, h // G].double()
            x = ((q @ k.T) / math.sqrt(D)).masked_fill(~see, -math.inf)
            some = see.any(1)
            p = torch.where(some[:, None], torch.exp(x - lse[h, lo:hi, None]), torch.zeros_like(x))
            A, most = p @ v.abs(), (p * v.abs().amax(-1)).amax(-1)
            left_out = 2.0 ** -17 * q.abs().amax(-1) * k.abs().sum(-1).amax() / math.sqrt(D)
            e_out[lo:hi, h] += ((2 * left_out + 2.0 ** -16)[:, None] * A + (kv * 2.0 ** -27 * most)[:, None]) * 1.01
            e_lse[h, lo:hi] += left_out * some + 2.0 ** -20
    return out, lse, e_out, e_lse


def check(b8):
    out, lse = ra.tree_attn_q8(*b8.args(), tree_mask=b8.mask())
    ra.device_status()
    ref, ref_lse, e_out, e_lse = definition(b8)
    within(lse, ref_lse, e_lse, "lse")
    within(out, ref, e_out, "out")
    return out, ref


def with_sink(keys, share, deviation, value, D):
    """One key that holds `share` of the weight, its value `value` times the others', which are positive."""
    def edit(b):
        g = torch.Generator().manual_seed(3)
        score = math.log(share / (1 - share) * keys) + deviation ** 2 / 2
        b.q[:] = 1.0
        for s in range(len(b.k)):
            b.k[s][1:] = deviation * torch.randn(b.k[s][1:].shape, generator=g)
            b.k[s][0] = score / math.sqrt(D)
            b.v[s][:] = 0.5 + 0.5 * torch.rand(b.v[s].shape, generator=g)
            b.v[s][0] *= value
    return edit


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("share", [0.5, 0.99, 0.999, 0.9999])
@pytest.mark.parametrize("deviation", [0.0, 1.0], ids=["equal", "spread"])
@pytest.mark.parametrize("tokens", [1, 4, 8, 40])
def test_a_sink_of_no_value(tokens, deviation, share, dtype):
    """The output is what the other keys add up to, however small their weights (4, 16, 32 and 160 rows a head)."""
    D = 128
    out, ref = check(Batch8([(16000, tokens)], 8, 2, D, 64, dtype, "chain", seed=21, edit=with_sink(16000, share, deviation, 0.0, D)))
    assert ((out.double().cpu() - ref).abs().amax(-1) <= 2.0 ** -6 * ref.abs().amax(-1)).all()


@pytest.mark.parametrize("value", [2.0 ** -12, 2.0 ** -5, 1.0, 2.0 ** 20])
@pytest.mark.parametrize("tokens", [1, 8, 40])
def test_a_sink_of_any_value(tokens, value):
    check(Batch8([(9000, tokens)], 8, 2, 64, 16, BF16, "chain", seed=22, edit=with_sink(9000, 0.9999, 1.0, value, 64)))


@pytest.mark.parametrize("tokens", [1, 4, 8, 40])
@pytest.mark.parametrize("keys,share,deviation", [(3000, 0.9998, 0.0), (12000, 0.9999, 0.0), (12000, 0.9999, 1.0)])
def test_sinks_of_many_sequences(keys, share, deviation, tokens):
    """Units that are walked from the first key to the last by one CTA: the sink weighs on all of them."""
    one = Batch8([(keys, tokens)], 8, 2, 64, 64, BF16, seed=23, edit=with_sink(keys, share, deviation, 0.0, 64))
    ref, _, e_out, _ = definition(one)
    q, offs, *pools, pages, lens = one.args()
    n = 400
    out, _ = ra.tree_attn_q8(q.repeat(n, 1, 1), torch.arange(n + 1, dtype=torch.int32, device="cuda") * tokens, *pools,
                             pages.expand(n, -1).contiguous(), lens.expand(n).contiguous())
    ra.device_status()
    within(out, ref.repeat(n, 1, 1), e_out.repeat(n, 1, 1), "out")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("power", [20, 40, 100])
@pytest.mark.parametrize("mask", ["chain", "tree"])
@pytest.mark.parametrize("tokens", [2, 4, 8, 40])
def test_a_hidden_value_takes_nothing_with_it(tokens, mask, power, dtype):
    """A later token of a chain, or one on another branch, whose value lies far above the others': the rows that do not
    see it are as if it were not there."""
    def edit(b):
        for s, n in enumerate((tokens, tokens)):
            b.v[s][-1] *= 2.0 ** power
            if n > 2:
                b.v[s][-n + 1] *= 2.0 ** (power // 2)
    check(Batch8([(300, tokens), (70, tokens)], 8, 2, 128, 16, dtype, mask, seed=24, edit=edit))


@pytest.mark.parametrize("tokens", [1, 4, 8, 40])
@pytest.mark.parametrize("order", ["random", "falling", "rising", "tiles"])
def test_values_of_any_size(order, tokens):
    """Scales of values from 2^-60 to 2^60, one key beside the next, falling or rising along the keys, or by tile: a row's
    sum counts every key, its output what the large ones leave."""
    def edit(b):
        g = torch.Generator().manual_seed(25)
        for s in range(len(b.v)):
            n = b.v[s].shape[0]
            e = {"random": torch.randint(-60, 61, (n,), generator=g), "falling": 60 - 120 * torch.arange(n) // n,
                 "rising": 120 * torch.arange(n) // n - 60, "tiles": torch.where(torch.arange(n) // 128 % 2 == 0, 60, -60)}[order]
            b.v[s] *= torch.exp2(e.float())[:, None, None]
            b.v[s][5::97] = 0
    check(Batch8([(1500, tokens), (400, tokens)], 8, 2, 64, 16, BF16, "chain", seed=25, edit=edit))


@pytest.mark.parametrize("tokens", [1, 4, 8, 40])
def test_values_near_the_least(tokens):
    """Values whose scales are the least there are come out with what bf16 holds of them."""
    def edit(b):
        for v in b.v:
            v *= 2.0 ** -117
    b8 = Batch8([(400, tokens), (40, tokens)], 8, 2, 64, 16, BF16, "chain", seed=26, edit=edit)
    out, _ = ra.tree_attn_q8(*b8.args())
    ra.device_status()
    ref, _, e_out, _ = definition(b8)
    # attention() allows 1e-30 for fp32's own least numbers: scaled up, so that it counts for nothing
    up = 2.0 ** 100
    for v in b8.base.v:
        v *= up
    _, _, e_up, _ = definition(b8)
    # below 2^-126 a bf16's step is 2^-133
    within(out.double() * up, ref * up, e_up + 2.0 ** -134 * up, "out")


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("tokens", [1, 4, 8, 40])
@pytest.mark.parametrize("nothing", ["values of zero", "scales of zero", "scales of zero in places"])
def test_values_of_nothing(nothing, tokens, dtype):
    """Zeros as values, or scale bytes that mean zero (under codes of any size): nothing in the output,
    and all of their weight in the sums."""
    def edit(b):
        for v in b.v:
            if nothing == "values of zero":
                v *= 0
    b8 = Batch8([(600, tokens), (40, tokens)], 8, 2, 64, 16, dtype, "chain", seed=28, edit=edit)
    if nothing != "values of zero":
        for s in range(2):
            kv = b8.v[s].shape[0]
            at = torch.arange(kv)[::1 if nothing == "scales of zero" else 3]
            b8.v[s][at] = 0
            b8.scales[1][b8.base.pages[s, at // 16].long(), :, at % 16] = 0
    out, ref = check(b8)
    if "places" not in nothing:
        assert (out == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("cache", ["8 bits", "rows"])
@pytest.mark.parametrize("keys,tokens", [(50, 4), (9000, 1), (9000, 4), (9000, 40)])
def test_lse_of_rows_that_are_not_numbers(keys, tokens, cache, dtype):
    """A row whose output is NaN has lse NaN, not the -inf of a row that saw no key; whole and cut units."""
    seqs = [(keys, tokens), (0, 1), (33, 1)]
    b8 = Batch8(seqs, 8, 2, 128, 16, dtype, "chain", seed=27)
    b = b8.base if cache == "8 bits" else make_batch(seqs, 8, 2, 128, 16, dtype, "chain", seed=27)
    bad = torch.zeros(b.q.shape[:2], dtype=torch.bool)
    for r, h, x in ((0, 3, math.nan), (tokens - 1, 5, math.inf), (tokens + 1, 0, math.nan)):
        b.q[r, h, 7] = x
        bad[r, h] = True
    ref, ref_lse, e_out, e_lse = attention(b) if cache == "rows" else definition(b8)
    if cache == "8 bits":
        out, lse = ra.tree_attn_q8(*b8.args())
    else:
        c = b.cuda()
        out, lse = ra.tree_attn(c.q, c.offs, c.k_pages, c.v_pages, c.pages, c.lens)
    ra.device_status()
    out, lse = out.cpu(), lse.cpu().T
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    within(out[~bad], ref[~bad], e_out[~bad], "out")
    within(lse[~bad], ref_lse.T[~bad], e_lse.T[~bad], "lse")
    assert (lse[tokens] == -math.inf).all() and (out[tokens] == 0).all()
