"""The norm of the heads and its gradient with infinities among dims that are not rotated."""
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300.build import build
from head_norm_cases import backward, forward, make_case

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    ra.load()


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
