"""The norm of the heads and its gradient where one token, one head or one value decides: the weights' gradients with
sums that fp32 holds exactly, and infinities among dims that are not rotated."""
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300.build import build
from head_norm_cases import backward, forward, make_case
from head_norm_sums import SIZES, one_token

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    ra.load()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lead,Hq,Hkv,D", SIZES)
def test_weight_gradients_count_every_head(lead, Hq, Hkv, D, dtype):
    """x = +-1 without an eps: n is x times the root of one, off by 2 steps (2^-22) at most and the same for every head;
    upstream gradients are odd whole numbers.  The sum is whole, at most 3 2^18 in size: the root moves it by less than
    0.2 (partial sums are whole numbers below 2^24 times it), and every head moves every column by one at least.  A head
    left out, taken twice or out of another place shows."""
    c = make_case(lead, Hq, Hkv, D, dtype, rot=0, eps=0.0, seed=31)
    g = torch.Generator().manual_seed(32)
    sign = lambda t: (2 * torch.randint(0, 2, t.shape, generator=g) - 1).to(dtype)  # noqa: E731
    c.q, c.k = sign(c.q), sign(c.k)
    c.gq, c.gk = ((2 * torch.randint(-2, 2, t.shape, generator=g) + 1).to(dtype) for t in (c.gq, c.gk))
    d = c.cuda()
    *_, dwq, dwk = ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how)
    ra.device_status()
    for got, x, gy in ((dwq, c.q, c.gq), (dwk, c.k, c.gk)):
        want = (x.double() * gy.double()).flatten(0, -2).sum(0)
        assert gy.double().abs().flatten(0, -2).sum(0).max() <= 3 * 2 ** 18
        assert ((got.double().cpu() - want).abs() < 0.45).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lead,Hq,Hkv,D", SIZES)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
def test_weight_gradients_of_one_token(lead, Hq, Hkv, D, where, dtype):
    """Upstream gradients of one token only (rotated, with its own angles): the sums are that token's, with its few roundings."""
    n = math.prod(lead)
    c, one = one_token(lead, Hq, Hkv, D, dtype, {"first": 0, "middle": n // 2, "last": n - 1}[where])
    d = c.cuda()
    *_, dwq, dwk = ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how)
    ra.device_status()
    (_, _, wq, wk), (_, _, eq, ek) = backward(one)
    for got, want, e in ((dwq, wq, eq), (dwk, wk, ek)):
        assert ((got.double().cpu() - want).abs() <= e).all()


def same_kind(got, want, what):
    """Finite, infinite and NaN in the same places."""
    got = got.double().cpu()
    for f in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(f(got), f(want)), what


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "next"])
@pytest.mark.parametrize("norm", [True, False], ids=["norm", "no norm"])
@pytest.mark.parametrize("D,rot", [(64, 32), (128, 0), (128, 120)])
def test_infinities_that_are_not_rotated(D, rot, norm, interleaved, dtype):
    """An infinity in a dim that no pair turns is in no pair: what shares its lane is what the formula gives."""
    for dims in ((rot,), (D - 1,), (D - 4, D - 3), (D - 8,)):
        if min(dims) < rot:
            continue
        c = make_case((9,), 6, 2, D, dtype, rot=rot, norm=norm, interleaved=interleaved, seed=34)
        for i, at in enumerate(dims):
            c.q[3, 1, at] = math.inf if i == 0 else -math.inf
            c.k[5, 0, at] = -math.inf
        d = c.cuda()
        want, _ = forward(c)
        for got, w, name in zip(ra.qk_norm_rope(*d.args, **d.how), want, "qk"):
            same_kind(got, w, (name, dims))
        bad = [t.isnan() | t.isinf() for t in want]
        assert all(int(b.sum()) <= 3 for b in bad)   # of the values given, and no others
        # the gradient of an infinite upstream gradient: its own column of dw, no other
        c = make_case((9,), 6, 2, D, dtype, rot=rot, norm=norm, interleaved=interleaved, seed=35)
        c.gq[3, 1, dims[0]], c.gk[5, 0, dims[0]] = math.inf, -math.inf
        d = c.cuda()
        want, _ = backward(c)
        for got, w, name in zip(ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how), want, ("dq", "dk", "dwq", "dwk")):
            if w is None:
                assert got is None
            elif name.startswith("dw"):
                same_kind(got, w, (name, dims))
                assert int((~w.isfinite()).sum()) == 1
            else:   # the head's mean is infinite, and with it every dim of the head with a norm
                heads = ~got.double().cpu().isfinite()
                assert torch.equal(heads, ~w.isfinite()), (name, dims)
    ra.device_status()
