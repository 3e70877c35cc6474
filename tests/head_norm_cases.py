"""The norm of the heads with the rotation by position, and its gradient, straight from their definition in 64
bits, with bounds that count the roundings of a kernel whose statistics, angles and products are fp32."""
from dataclasses import dataclass

import torch

U32, U16 = 2.0 ** -24, 2.0 ** -8   # half a step of fp32 and bf16, relative
# cos and sin: the fraction of a turn rounded to 24 bits (pi 2^-25 of a radian at most), 2 steps of the function
# itself, and positions up to 2^28 (2^-22 of a radian)
E_TURN = 3.15 * 2.0 ** -25 + 4 * U32 + 2.0 ** -22


@dataclass
class Case:
    q: torch.Tensor
    k: torch.Tensor
    wq: torch.Tensor | None
    wk: torch.Tensor | None
    positions: torch.Tensor | None
    inv_freq: torch.Tensor | None
    sections: tuple | None
    interleaved: bool
    eps: float
    gq: torch.Tensor
    gk: torch.Tensor

    def cuda(self):
        f = lambda t: t.cuda() if isinstance(t, torch.Tensor) else t  # noqa: E731
        return Case(*(f(getattr(self, n)) for n in self.__dataclass_fields__))

    @property
    def args(self):
        return self.q, self.k, self.wq, self.wk, self.positions, self.inv_freq

    @property
    def how(self):
        return dict(sections=self.sections, eps=self.eps, interleaved=self.interleaved)


def make_case(lead, Hq, Hkv, D, dtype, rot=None, sections=None, interleaved=False, norm=True, eps=1e-6, seed=0, far=1 << 20,
              base=1e4, scale=1.0):
    """lead: the leading dimensions; rot None: the whole head, 0: none."""
    g = torch.Generator().manual_seed(seed)
    lead = tuple(lead)
    normal = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q, k = ((normal(*lead, H, D) * scale).to(dtype) for H in (Hq, Hkv))
    wq, wk = ((1 + 0.2 * normal(D)).to(dtype) if norm else None for _ in range(2))
    rot = D if rot is None else rot
    pos = freq = None
    if rot:
        axes = len(sections) if sections else 1
        pos = torch.randint(-far, far, (axes, *lead), generator=g, dtype=torch.int32)
        if not sections:
            pos = pos[0].contiguous()
        freq = (base ** (-2 * torch.arange(rot // 2, dtype=torch.float64) / rot)).float()
    gq, gk = (normal(*lead, H, D).to(dtype) for H in (Hq, Hkv))
    return Case(q, k, wq, wk, pos, freq, sections, interleaved, eps, gq, gk)


def _angle(c, D):
    """cos, sin [..., 1, pairs] and the dims of the pairs."""
    if c.inv_freq is None:
        return None
    n = c.inv_freq.shape[0]
    pos = c.positions if c.sections else c.positions[None] if c.positions.dim() == c.q.dim() - 2 else c.positions
    axis = torch.tensor([a for a, m in enumerate(c.sections or (n,)) for _ in range(m)])
    angle = (pos.double().movedim(0, -1)[..., axis] * c.inv_freq.double())[..., None, :]
    i = torch.arange(n)
    a, b = (2 * i, 2 * i + 1) if c.interleaved else (i, i + n)
    return torch.cos(angle), torch.sin(angle), a, b


def turned(c, y, turn, back=False):
    if turn is None:
        return y
    cos, sin, a, b = turn
    sin = -sin if back else sin
    z = y.clone()
    z[..., a] = y[..., a] * cos - y[..., b] * sin
    z[..., b] = y[..., b] * cos + y[..., a] * sin
    return z


def _swap(y, turn):
    """The sizes of a value and of the other of its pair, together (the value alone where nothing turns)."""
    z = y.abs().clone()
    if turn is not None:
        _, _, a, b = turn
        both = y[..., a].abs() + y[..., b].abs()
        z[..., a], z[..., b] = both, both
    return z


def _u(c):
    return U16 if c.q.dtype == torch.bfloat16 else U32


def forward(c):
    """((q, k), their bounds)."""
    D = c.q.shape[-1]
    turn = _angle(c, D)
    got, err = [], []
    for x, w in ((c.q, c.wq), (c.k, c.wk)):
        x = x.double()
        y, rel = x, 0.0
        if w is not None:
            y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + c.eps) * w.double()
            # mean of D squares, its square root (half the relative error), its inverse, two products
            rel = (D / 2 + 10) * U32
        z = turned(c, y, turn)
        got.append(z)
        e = _swap(y, turn) * (rel + (E_TURN + 4 * U32 if turn is not None else 0.0))
        err.append(e * 1.01 + _u(c) * z.abs() + 1e-38)
    return got, err


def backward(c):
    """((dq, dk, dwq, dwk), their bounds)."""
    D = c.q.shape[-1]
    turn = _angle(c, D)
    dx, dw, ex, ew = [], [], [], []
    for x, w, g in ((c.q, c.wq, c.gq), (c.k, c.wk, c.gk)):
        x, g = x.double(), g.double()
        e_g = _swap(g, turn) * (E_TURN + 4 * U32) if turn is not None else torch.zeros_like(g)
        g = turned(c, g, turn, back=True)
        if w is None:
            dx.append(g)
            ex.append(e_g * 1.01 + _u(c) * g.abs() + 1e-38)
            dw.append(None)
            ew.append(None)
            continue
        w = w.double()
        r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + c.eps)
        n = x * r
        m = (g * w * n).mean(-1, keepdim=True)
        d = r * (g * w - n * m)
        dx.append(d)
        rel = (D + 20) * U32
        e = r * ((e_g + rel * g.abs()) * w.abs() + n.abs() * ((e_g + rel * g.abs()) * w.abs() * n.abs()).mean(-1, keepdim=True))
        ex.append(e * 1.01 + _u(c) * d.abs() + 1e-38)
        lead = tuple(range(x.dim() - 1))
        terms = x[..., 0].numel()
        dw.append((g * n).sum(lead))
        ew.append(((terms + D + 20) * U32 * (g * n).abs().sum(lead) + (e_g * n.abs()).sum(lead)) * 1.01 + 1e-38)
    return [*dx, *dw], [*ex, *ew]
