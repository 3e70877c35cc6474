"""CPU checks of the norm of the heads with the rotation by position: refusals before any launch, and the 64-bit
definitions the GPU tests use, against closed forms and differences."""
import ctypes
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300 import ra as rab
from ring_context_parallelism_gb300.build import build
from head_norm_cases import backward, forward, make_case

BAD, WS = rab.RA_ERR_INVALID_ARG, rab.RA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build()
    return ra.load()


def ints(*v):
    return (ctypes.c_int * len(v))(*v)


FWD = dict(q=16, qs=2048, k=32, ks=256, wq=16, wk=16, pos=16, freq=16, qo=16, qos=2048, ko=48, kos=256, R=10, Hq=16, Hkv=2,
           D=128, rot=128, sections=ints(64), axes=1, inter=0, eps=1e-6, dt=rab.RA_BF16, stream=None)
BWD = dict(q=16, qs=2048, k=32, ks=256, wq=16, wk=16, pos=16, freq=16, gq=48, gk=64, dq=16, dqs=2048, dk=64, dks=256, dwq=16,
           dwk=16, R=10, Hq=16, Hkv=2, D=128, rot=128, sections=ints(64), axes=1, inter=0, eps=1e-6, dt=rab.RA_BF16, ws=256,
           wsb=1 << 30, stream=None)
BOTH = [dict(dt=7), dict(D=96), dict(Hq=0), dict(Hkv=0), dict(Hq=(1 << 16) + 1), dict(R=-1), dict(R=(1 << 30) + 1),
        dict(R=1 << 28), dict(rot=-8), dict(rot=136), dict(rot=100), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
        dict(wq=None), dict(wk=None), dict(wk=24), dict(axes=0), dict(axes=5, sections=ints(64, 0, 0, 0, 0)),
        dict(sections=None), dict(sections=ints(63)), dict(axes=2, sections=ints(65, -1)), dict(pos=None), dict(freq=None),
        dict(pos=18), dict(freq=18), dict(q=None), dict(k=None), dict(q=24), dict(k=8), dict(qs=2044), dict(ks=-256),
        dict(qs=(1 << 31) + 8)]


@pytest.mark.parametrize("kw", BOTH + [dict(qo=None), dict(ko=None), dict(qo=24), dict(qos=2040), dict(kos=248), dict(kos=0),
                                       dict(qos=4096), dict(qs=0), dict(qo=32), dict(ko=16), dict(qo=48)])
def test_forward_refusals(lib, kw):
    assert lib.ra_qk_norm_rope(*{**FWD, **kw}.values()) == BAD
    assert lib.ra_last_error()


@pytest.mark.parametrize("kw,status", [(kw, BAD) for kw in BOTH] + [
    (dict(gq=None), BAD), (dict(gk=8), BAD), (dict(dq=None), BAD), (dict(dqs=2040), BAD), (dict(dks=128), BAD),
    (dict(dqs=4096), BAD), (dict(dks=512), BAD), (dict(dq=48, dqs=4096), BAD), (dict(dq=32), BAD), (dict(dk=48), BAD),
    (dict(dk=16), BAD), (dict(dwq=None), BAD), (dict(dwk=18), BAD), (dict(ws=None), WS), (dict(ws=128), BAD), (dict(wsb=64), WS)])
def test_backward_refusals(lib, kw, status):
    assert lib.ra_qk_norm_rope_bwd(*{**BWD, **kw}.values()) == status
    assert lib.ra_last_error()


def test_nothing_to_do_launches_nothing(lib):
    none = dict(R=0, q=None, k=None, pos=None, freq=None)
    assert lib.ra_qk_norm_rope(*{**FWD, **none, "qo": None, "ko": None}.values()) == rab.RA_OK
    assert lib.ra_qk_norm_rope_bwd(*{**BWD, **none, "wq": None, "wk": None, "gq": None, "gk": None, "dq": None, "dk": None,
                                     "ws": None}.values()) == rab.RA_OK
    assert lib.ra_last_error() == b""


def test_workspace_size(lib):
    a, b = (int(lib.ra_qk_norm_rope_bwd_workspace_size(D)) for D in (64, 128))
    assert 0 < a and b == 2 * a and lib.ra_qk_norm_rope_bwd_workspace_size(96) == 0


def test_binding_refuses_wrong_shapes_and_types(lib):
    c = make_case((6,), 4, 2, 64, torch.float32)
    run = lambda *a, **kw: ra.qk_norm_rope(*a, **kw)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        run(*c.args)
    with pytest.raises(TypeError, match="dtype"):
        run(c.q.double(), *c.args[1:])
    with pytest.raises(ValueError, match="same tokens"):
        run(c.q[:5], *c.args[1:])
    with pytest.raises(ValueError, match="same tokens"):
        run(c.q, c.k.bfloat16(), *c.args[2:])
    with pytest.raises(ValueError, match="weight"):
        run(c.q, c.k, c.wq[:32], c.wk, *c.args[4:])
    with pytest.raises(ValueError, match="neither"):
        run(c.q, c.k, c.wq, None, *c.args[4:])
    with pytest.raises(ValueError, match="neither"):
        run(*c.args[:5], None)
    with pytest.raises(ValueError, match="int32"):
        run(*c.args[:4], c.positions.long(), c.inv_freq)
    with pytest.raises(ValueError, match="positions"):
        run(*c.args[:4], c.positions[:5], c.inv_freq)
    with pytest.raises(ValueError, match="positions"):
        run(*c.args, sections=(16, 16))
    with pytest.raises(ValueError, match="axes"):
        run(*c.args, sections=())
    with pytest.raises(TypeError, match="sections"):
        run(*c.args, sections=32)
    with pytest.raises(TypeError):
        run(*c.args, sections=("a",))
    with pytest.raises(TypeError):
        run(*c.args, eps="x")
    with pytest.raises(ValueError, match="inv_freq"):
        run(*c.args[:5], torch.ones(33))
    with pytest.raises(ValueError, match="sections"):
        run(*c.args[:4], None, None, sections=(32,))
    with pytest.raises(ValueError, match="dense heads"):
        run(c.q.transpose(0, 1).contiguous().transpose(0, 1), *c.args[1:])
    with pytest.raises(ValueError, match="q_out"):
        run(*c.args, q_out=c.q[:, :2])
    with pytest.raises(TypeError, match="q must be a tensor"):
        run(None, *c.args[1:])
    with pytest.raises(ValueError, match="dq_out"):
        ra.qk_norm_rope_bwd(*c.args, c.gq[:, :2], c.gk)


def test_definition_in_closed_form():
    """Ones with a weight keep it (over sqrt(1 + eps)) and turn by their angle; a turn keeps lengths; position 0 turns nothing."""
    c = make_case((3,), 2, 1, 64, torch.float32, seed=1)
    c.q.fill_(1.0)
    c.wq.fill_(2.0)
    (q, k), _ = forward(c)
    a = c.positions.double()[:, None] * c.inv_freq.double()
    want = 2 / math.sqrt(1 + 1e-6) * torch.cat([torch.cos(a) - torch.sin(a), torch.cos(a) + torch.sin(a)], -1)
    assert torch.allclose(q[:, 0], want, atol=1e-9)
    assert torch.allclose(k.square().sum(-1), (c.k.double() / (c.k.double().square().mean(-1, keepdim=True) + 1e-6).sqrt()
                                               * c.wk.double()).square().sum(-1))
    c.positions.zero_()
    (q, _), _ = forward(c)
    assert torch.allclose(q, torch.full_like(q, 2 / math.sqrt(1 + 1e-6)))


@pytest.mark.parametrize("kw", [dict(), dict(rot=32, interleaved=True, sections=(4, 6, 6)), dict(norm=False), dict(rot=0)])
def test_gradient_definition_against_differences(kw):
    c = make_case((5,), 3, 2, 64, torch.float32, seed=2, far=100, **kw)
    (dq, dk, dwq, dwk), _ = backward(c)
    for name in ("q", "k", "wq", "wk", "gq", "gk"):
        if getattr(c, name) is not None:
            setattr(c, name, getattr(c, name).double())
    value = lambda: sum((y * g).sum() for y, g in zip(forward(c)[0], (c.gq, c.gk)))  # noqa: E731
    g = torch.Generator().manual_seed(3)
    for name, d in (("q", dq), ("k", dk), ("wq", dwq), ("wk", dwk)):
        if d is None:
            continue
        x = getattr(c, name)
        v = torch.randn(x.shape, generator=g, dtype=torch.float64)
        h = 1e-6
        setattr(c, name, x + h * v)
        up = value()
        setattr(c, name, x - h * v)
        down = value()
        setattr(c, name, x)
        assert abs((up - down) / (2 * h) - (d * v).sum()) <= 1e-7 * (1 + (d * v).abs().sum())
