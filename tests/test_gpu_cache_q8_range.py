"""Attention over paged sequences where values are not ordinary: rows that are not numbers say so."""
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300.build import build
from cache_cases import attention, make_batch
from cache_q8_cases import Batch8, attention_q8

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
    ref, ref_lse, e_out, e_lse = attention(b) if cache == "rows" else attention_q8(b8)
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
