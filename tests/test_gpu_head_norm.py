"""GPU parity of the norm of the heads with the rotation by position, and of its gradient, against their 64-bit
definitions, element by element, with bounds that count roundings (head_norm_cases.py)."""
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300 import ra as rab
from ring_context_parallelism_gb300.build import build
from head_norm_cases import Case, backward, forward, make_case

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build()
    ra.load()


def within(got, want, bound, what):
    got = got.double().cpu()
    off = torch.where(got == want, torch.zeros_like(want), (got - want).abs())
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {off[bad].max().item():.3e} "
                           f"where {bound[bad][off[bad].argmax()].item():.3e} is allowed; first at {bad.nonzero()[0].tolist()}")


def check(c, d=None):
    d = d or c.cuda()
    want, err = forward(c)
    for got, w, e, name in zip(ra.qk_norm_rope(*d.args, **d.how), want, err, "qk"):
        assert got.dtype == c.q.dtype and got.is_contiguous()
        within(got, w, e, name)
    want, err = backward(c)
    for got, w, e, name in zip(ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how), want, err, ("dq", "dk", "dwq", "dwk")):
        if w is None:
            assert got is None
        else:
            within(got, w, e, name)
    ra.device_status()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lead,Hq,Hkv,D", [((1,), 1, 1, 64), ((1,), 32, 8, 128), ((7,), 5, 3, 64), ((33,), 7, 1, 128),
                                           ((2, 51), 9, 2, 128), ((301,), 40, 8, 64), ((2, 3, 5), 4, 4, 128),
                                           ((700,), 64, 8, 128), ((2111,), 3, 2, 128)])
def test_sizes(lead, Hq, Hkv, D, dtype):
    check(make_case(lead, Hq, Hkv, D, dtype, seed=1))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "next"])
@pytest.mark.parametrize("D,rot,sections", [(128, 128, (16, 24, 24)), (128, 64, (32,)), (64, 24, (3, 4, 0, 5)), (64, 8, (1, 3)),
                                            (128, 128, (0, 64)), (64, 64, (32, 0, 0, 0)), (128, 0, None)])
def test_rotations(D, rot, sections, interleaved, dtype):
    check(make_case((37,), 6, 2, D, dtype, rot=rot, sections=sections, interleaved=interleaved, seed=2))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rot", [128, 32, 0])
def test_without_a_norm(rot, dtype):
    check(make_case((65,), 6, 2, 128, dtype, rot=rot, norm=False, seed=3))


@pytest.mark.parametrize("scale,eps", [(1e-3, 1e-6), (1e3, 1e-5), (1e-4, 0.0), (1.0, 0.5)])
def test_sizes_of_values(scale, eps):
    check(make_case((50,), 4, 2, 128, F32, scale=scale, eps=eps, seed=4))


@pytest.mark.parametrize("Hq,Hkv,D", [(5, 3, 128), (7, 1, 64), (1, 1, 128), (9, 6, 64)])
def test_heads_that_fill_no_step_without_an_eps(Hq, Hkv, D):
    """Lanes without a head add nothing to the weights' gradients: the root of their zeros is infinite without an eps."""
    check(make_case((21,), Hq, Hkv, D, F32, eps=0.0, seed=20))


def test_far_positions_and_large_frequencies():
    """Positions up to 2^28 either way; a frequency of several turns a token drops them."""
    check(make_case((200,), 2, 1, 64, F32, far=1 << 28, base=1e6, seed=5))
    c = make_case((100,), 2, 1, 64, F32, far=1 << 10, seed=6)
    c.inv_freq[:4] = torch.tensor([1.0, 6.25, 100.5, -3.0])
    check(c)
    d = c.cuda()
    d.positions.fill_(2 ** 31 - 1)
    d.positions[::2] = -2 ** 31
    q, k = ra.qk_norm_rope(*d.args, **d.how)   # lengths hold whatever the angle
    y = c.q.double() / (c.q.double().square().mean(-1, keepdim=True) + c.eps).sqrt() * c.wq.double()
    assert torch.allclose(q.double().cpu().square().sum(-1), y.square().sum(-1), rtol=1e-5)


def test_values_that_are_not_numbers():
    """A NaN or infinity stays in its head; a frequency that is none reaches its pairs alone; zeros stay zeros."""
    c = make_case((40,), 4, 2, 64, F32, seed=7)
    c.q[3, 1, 5], c.q[9, 0, 60], c.k[5, 1, 0] = math.nan, math.inf, -math.inf
    c.q[11, 2] = 0.0
    d = c.cuda()
    q, k = (t.cpu() for t in ra.qk_norm_rope(*d.args, **d.how))
    assert q[3, 1].isnan().all() and k[5, 1].isnan().any() and q[9, 0].isnan().any()
    assert (q[11, 2] == 0).all()
    q[3, 1], q[9, 0], k[5, 1] = 0, 0, 0
    assert q.isfinite().all() and k.isfinite().all()
    c = make_case((40,), 4, 2, 64, F32, rot=32, seed=7)
    c.inv_freq[5] = math.inf
    d = c.cuda()
    q, _ = (t.cpu() for t in ra.qk_norm_rope(*d.args, **d.how))
    bad = torch.zeros(64, dtype=torch.bool)
    bad[[5, 21]] = True
    assert q[..., bad].isnan().all() and q[..., ~bad].isfinite().all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_slices_and_in_place(dtype):
    """Queries and keys as slices of one projection's output, results into slices, in place, and gradients likewise."""
    for lead in ((45,), (3, 15)):
        c = make_case(lead, 6, 2, 128, dtype, seed=8)
        d = c.cuda()
        qkv = torch.cat([d.q, d.k, torch.full_like(d.k, math.nan)], -2)
        d.q, d.k = qkv[..., :6, :], qkv[..., 6:8, :]
        check(c, d)
        want = ra.qk_norm_rope(*d.args, **d.how)
        grads = ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how)
        big = torch.full((*lead, 11, 128), 5.0, dtype=dtype, device="cuda")
        qo, ko = big[..., 1:7, :], big[..., 8:10, :]
        got = ra.qk_norm_rope(*d.args, **d.how, q_out=qo, k_out=ko)
        assert got[0] is qo and got[1] is ko and torch.equal(qo, want[0]) and torch.equal(ko, want[1])
        assert (big[..., [0, 7, 10], :] == 5.0).all()
        big.fill_(5.0)
        dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how, dq=qo, dk=ko)
        assert dq is qo and torch.equal(dq, grads[0]) and torch.equal(dk, grads[1])
        assert torch.equal(dwq, grads[2]) and torch.equal(dwk, grads[3]) and (big[..., [0, 7, 10], :] == 5.0).all()
        gq, gk = d.gq.clone(), d.gk.clone()
        ra.qk_norm_rope_bwd(*d.args, gq, gk, **d.how, dq=gq, dk=gk)   # over the upstream gradients
        assert torch.equal(gq, grads[0]) and torch.equal(gk, grads[1])
        keep = qkv.clone()
        ra.qk_norm_rope(*d.args, **d.how, q_out=d.q, k_out=d.k)
        assert torch.equal(d.q, want[0]) and torch.equal(d.k, want[1]) and qkv[..., 8:, :].isnan().all()
        qkv.copy_(keep)
        ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how, dq=d.q, dk=d.k)
        assert torch.equal(d.q, grads[0]) and torch.equal(d.k, grads[1])


def test_inputs_that_broadcast():
    """One token's values for all (stride 0); the gradient has a row for each."""
    c = make_case((20,), 4, 2, 64, F32, seed=9)
    c.q, c.k = (t[:1].expand(20, *t.shape[1:]).contiguous() for t in (c.q, c.k))
    d = c.cuda()
    d.q, d.k = d.q[:1].expand(20, 4, 64), d.k[:1].expand(20, 2, 64)
    check(c, d)


def test_no_tokens():
    c = make_case((0,), 4, 2, 64, BF16, seed=10)
    d = c.cuda()
    q, k = ra.qk_norm_rope(*d.args, **d.how)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how)
    assert dq.shape == (0, 4, 64) and (dwq == 0).all() and (dwk == 0).all() and dwq.shape == (64,)
    ra.device_status()


def test_gradient_against_differences():
    """fp32 gradient along a direction against the 64-bit function's differences: off by the gradient's own bound."""
    c = make_case((40,), 4, 2, 64, F32, seed=11, far=1000, sections=(10, 10, 12))
    d = c.cuda()
    got = ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how)
    _, err = backward(c)
    base = Case(**{n: (t.double() if isinstance(t, torch.Tensor) and t.is_floating_point() else t)
                   for n, t in vars(c).items()})
    value = lambda: sum((y * g).sum() for y, g in zip(forward(base)[0], (base.gq, base.gk)))  # noqa: E731
    g = torch.Generator().manual_seed(12)
    for name, x, e in zip(("q", "k", "wq", "wk"), got, err):
        v = torch.randn(x.shape, generator=g, dtype=torch.float64)
        at, h = getattr(base, name), 1e-6
        setattr(base, name, at + h * v)
        up = value()
        setattr(base, name, at - h * v)
        down = value()
        setattr(base, name, at)
        diff, mine = (up - down) / (2 * h), (x.double().cpu() * v).sum()
        assert abs(diff - mine) <= (e * v.abs()).sum() + 1e-7 * (1 + abs(mine)), name


def test_repeats_and_workspace():
    """The same bits from call to call, whatever the workspace holds; a workspace that is too small is refused."""
    c = make_case((900,), 16, 4, 128, BF16, seed=13).cuda()
    want = ra.qk_norm_rope_bwd(*c.args, c.gq, c.gk, **c.how)
    size = int(ra.load().ra_qk_norm_rope_bwd_workspace_size(128))
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        got = ra.qk_norm_rope_bwd(*c.args, c.gq, c.gk, **c.how, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(ra.RAError) as e:
        ra.qk_norm_rope_bwd(*c.args, c.gq, c.gk, **c.how, workspace=ws[:256])
    assert e.value.status == rab.RA_ERR_WORKSPACE
    with pytest.raises(ra.RAError) as e:
        ra.qk_norm_rope(c.q, c.k, c.wq, c.wk, c.positions, c.inv_freq, sections=(63,))
    assert e.value.status == rab.RA_ERR_INVALID_ARG


def test_in_a_graph_on_streams_and_after_writes():
    """Captured and replayed on new values; two streams at once; inputs that the stream has just written."""
    cs = [make_case((130,), 8, 2, 128, BF16, seed=s) for s in (14, 15, 16)]
    ds = [c.cuda() for c in cs]
    want = [(*ra.qk_norm_rope(*d.args, **d.how), *ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how)) for d in ds]
    d = ds[0]
    buf = Case(**{n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in vars(d).items()})
    ws = torch.empty(int(ra.load().ra_qk_norm_rope_bwd_workspace_size(128)), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (*ra.qk_norm_rope(*buf.args, **buf.how), *ra.qk_norm_rope_bwd(*buf.args, buf.gq, buf.gk, **buf.how, workspace=ws))
    tensors = lambda c: [t for t in vars(c).values() if isinstance(t, torch.Tensor)]  # noqa: E731
    big = torch.zeros(1 << 26, device="cuda")
    for i in (0, 1, 2, 1, 0):
        big.add_(1)
        for to, src in zip(tensors(buf), tensors(ds[i])):
            to.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i])), i
        for to, src in zip(tensors(buf), tensors(ds[i])):
            to.copy_(src)
        now = (*ra.qk_norm_rope(*buf.args, **buf.how), *ra.qk_norm_rope_bwd(*buf.args, buf.gq, buf.gk, **buf.how))
        assert all(torch.equal(a, b) for a, b in zip(now, want[i])), i
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for d, s in zip(ds, streams):
            with torch.cuda.stream(s):
                got.append((*ra.qk_norm_rope(*d.args, **d.how), *ra.qk_norm_rope_bwd(*d.args, d.gq, d.gk, **d.how)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for i, g in enumerate(got) for a, b in zip(g, want[i % 3]))


def test_strides_past_32_bits():
    """Tokens so far apart that their offsets pass 2^31 elements and 2^32 bytes."""
    c = make_case((3,), 2, 1, 64, BF16, seed=17)
    far = (1 << 30) + 512
    room = torch.empty(2 * far + 4096, dtype=BF16, device="cuda")
    d = c.cuda()
    want = ra.qk_norm_rope(*d.args, **d.how)
    q, k = room.as_strided((3, 2, 64), (far, 64, 1)), room.as_strided((3, 1, 64), (far, 64, 1), 512)
    q.copy_(d.q)
    k.copy_(d.k)
    got = ra.qk_norm_rope(q, k, *d.args[2:], **d.how)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ra.qk_norm_rope(*d.args, **d.how, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])


def test_before_the_attention_and_its_gradient():
    """Norm and rotation, attention, and both gradients, as a training step strings them together, against 64 bits: with
    fp32 throughout, off by the size of their sums' roundings."""
    B, S, Hq, Hkv, D = 1, 128, 2, 1, 64
    c = make_case((B, S), Hq, Hkv, D, F32, seed=18, far=1000)
    g = torch.Generator().manual_seed(19)
    v, do = torch.randn(B, S, Hkv, D, generator=g), torch.randn(B, S, Hq, D, generator=g)
    d = c.cuda()
    q, k = ra.qk_norm_rope(*d.args, **d.how)
    out, lse = ra.attn(q, k, v.cuda(), 2, 64, True)
    dqn, dkn, dv = ra.attn_bwd(q, k, v.cuda(), out, lse, do.cuda(), 2, 64, True)
    dq, dk, dwq, dwk = ra.qk_norm_rope_bwd(*d.args, dqn, dkn, **d.how)
    ra.device_status()
    leaves = [t.double().requires_grad_() for t in (c.q, c.k, c.wq, c.wk, v)]
    n = c.inv_freq.shape[0]
    turn = torch.polar(torch.ones(B, S, n, dtype=torch.float64), c.positions.double()[..., None] * c.inv_freq.double())[..., None, :]

    def one(x, w):
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + c.eps) * w
        z = torch.complex(y[..., :n], y[..., n:]) * turn
        return torch.cat([z.real, z.imag], -1)

    yq, yk = one(leaves[0], leaves[2]), one(leaves[1], leaves[3])
    x = torch.einsum("bthd,bjhd->bhtj", yq, yk.repeat_interleave(2, 2)) / 8
    x = x.masked_fill(torch.ones(S, S).triu(1).bool(), -math.inf)
    o = torch.einsum("bhtj,bjhd->bthd", torch.softmax(x, -1), leaves[4].repeat_interleave(2, 2))
    want = torch.autograd.grad((o * do.double()).sum(), leaves)
    # scores of some tens: their roundings, D + 6 of a size of 40, move a weight by 2^-12 of itself at most
    for got, w in zip((dq, dk, dwq, dwk, dv), want):
        assert (got.double().cpu() - w).abs().max() <= 2.0 ** -11 * w.abs().max()
