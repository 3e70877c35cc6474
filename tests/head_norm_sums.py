"""Cases of the head norm's gradient in which one token decides its weights' gradients."""
import math

from head_norm_cases import make_case

SIZES = [((700,), 64, 8, 128), ((301,), 40, 8, 64), ((2111,), 3, 2, 128), ((5003,), 7, 1, 64), ((4, 2049), 32, 8, 128)]


def one_token(lead, Hq, Hkv, D, dtype, at):
    """(a case whose upstream gradients are those of token `at` only, that token alone: its bound counts its few heads)."""
    c = make_case(lead, Hq, Hkv, D, dtype, seed=33, far=1000)
    for t in (c.gq, c.gk):
        rows = t.view(math.prod(lead), *t.shape[-2:])
        keep = rows[at].clone()
        rows.zero_()
        rows[at] = keep
    one = make_case((1,), Hq, Hkv, D, dtype, seed=33, far=1000)
    for name in ("q", "k", "gq", "gk"):
        t = getattr(c, name)
        setattr(one, name, t.view(math.prod(lead), *t.shape[-2:])[at:at + 1].contiguous())
    one.wq, one.wk, one.positions = c.wq, c.wk, c.positions.flatten()[at:at + 1].contiguous()
    return c, one
