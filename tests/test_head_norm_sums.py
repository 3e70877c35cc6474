"""CPU check of the bounds that the head norm's sums are held to: mistakes planted in the definition are outside them."""
import math

import pytest
import torch

from head_norm_cases import backward
from head_norm_sums import SIZES, one_token


@pytest.mark.parametrize("lead,Hq,Hkv,D", SIZES)
@pytest.mark.parametrize("mistake", ["a head left out", "a head twice", "the token before"])
def test_a_planted_mistake_is_outside(lead, Hq, Hkv, D, mistake):
    c, one = one_token(lead, Hq, Hkv, D, torch.float32, math.prod(lead) - 1)
    (_, _, wq, wk), (_, _, eq, ek) = backward(one)
    (_, _, all_q, all_k), _ = backward(c)
    assert (all_q - wq).abs().max() <= 1e-9 and (all_k - wk).abs().max() <= 1e-9   # the other tokens add nothing
    if mistake == "the token before":
        one.q, one.k = (t.flatten(0, -3)[-2:-1].contiguous() for t in (c.q, c.k))
    else:
        one.gq[0, Hq - 1] *= 0 if mistake == "a head left out" else 2
        one.gk[0, 0] *= 0 if mistake == "a head left out" else 2
    (_, _, bad_q, bad_k), _ = backward(one)
    for good, bad, e in ((wq, bad_q, eq), (wk, bad_k, ek)):
        assert ((good - bad).abs() > e).sum() >= D // 2   # a factor of a head may be small in some columns
