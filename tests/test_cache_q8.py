"""CPU checks of the 8-bit cache: refusals before any launch, workspace sizes, and the 64-bit definitions the GPU
tests use."""
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300 import ra as rab
from ring_context_parallelism_gb300.build import build
from cache_q8_cases import E4M3, Batch8, attention_q8, codes, scale_bytes, value

BAD, UNS, WS = rab.RA_ERR_INVALID_ARG, rab.RA_ERR_UNSUPPORTED, rab.RA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build()
    return ra.load()


APPEND = dict(kr=16, vr=16, offs=16, n_seqs=4, R=10, k=16, v=16, ks=16, vs=16, n_pages=64, page=16, pages=16, max_pages=8,
              lens=16, Hkv=2, D=128, dt=rab.RA_BF16, stream=None)
READ = dict(offs=16, n_seqs=4, R=10, k=16, v=16, ks=16, vs=16, n_pages=64, page=16, pages=16, max_pages=8, lens=16, kr=16, vr=16,
            Hkv=2, D=128, dt=rab.RA_BF16, stream=None)
TREE = dict(q=16, offs=16, n_seqs=4, R=10, k=16, v=16, ks=16, vs=16, n_pages=64, page=16, pages=16, max_pages=8, lens=16,
            mask=None, cols=0, out=16, lse=None, Hq=16, Hkv=2, D=128, dt=rab.RA_BF16, ws=256, wsb=1 << 40, stream=None)
POOL = [dict(k=None), dict(v=None), dict(k=24), dict(v=24), dict(ks=None), dict(vs=None), dict(ks=24), dict(vs=8),
        dict(n_pages=0), dict(page=12), dict(page=4), dict(page=1 << 21), dict(D=96), dict(dt=5), dict(Hkv=0),
        dict(n_pages=1 << 27), dict(n_seqs=0), dict(offs=None), dict(pages=None), dict(lens=None), dict(R=-1),
        dict(max_pages=0), dict(offs=18), dict(n_seqs=(1 << 24) + 1), dict(R=(1 << 30) + 1)]


@pytest.mark.parametrize("kw", POOL + [dict(kr=None), dict(vr=None), dict(vr=24), dict(Hkv=(1 << 16) + 1)])
def test_append_and_read_refusals(lib, kw):
    for fn, base in ((lib.ra_cache_append_paged_q8, APPEND), (lib.ra_cache_read_paged_q8, READ)):
        assert fn(*{**base, **kw}.values()) == BAD
        assert lib.ra_last_error()


@pytest.mark.parametrize("kw,status", [(kw, BAD) for kw in POOL] + [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(out=24), BAD), (dict(q=24), BAD), (dict(Hq=15), BAD), (dict(Hq=258), UNS),
    (dict(R=1 << 30), BAD), (dict(mask=16, cols=0), BAD), (dict(ws=None), WS), (dict(wsb=64), WS), (dict(ws=272), BAD),
    (dict(lse=18), BAD)])
def test_tree_attn_refusals(lib, kw, status):
    assert lib.ra_tree_attn_paged_q8(*{**TREE, **kw}.values()) == status
    assert lib.ra_last_error()


def test_nothing_to_do_launches_nothing(lib):
    assert lib.ra_tree_attn_paged_q8(*{**TREE, "R": 0, "q": None, "out": None, "ws": None}.values()) == rab.RA_OK
    assert lib.ra_cache_append_paged_q8(*{**APPEND, "R": 0, "kr": None, "vr": None}.values()) == rab.RA_OK
    assert lib.ra_cache_read_paged_q8(*{**READ, "R": 0, "kr": None, "vr": None}.values()) == rab.RA_OK
    assert lib.ra_last_error() == b""


def test_workspace_size(lib):
    size = ra.tree_attn_q8_workspace_size
    for dt in (torch.bfloat16, torch.float32):
        assert size(10, 4, 16, 2, 96, dt) == 0 and size(10, 4, 15, 2, 128, dt) == 0 and size(-1, 4, 16, 2, 128, dt) == 0
        a, b = size(1, 1, 8, 8, 128, dt), size(4096, 8, 64, 8, 128, dt)
        assert 0 < a < b and a % 256 == 0 and b % 256 == 0
        assert size(1 << 20, 8, 64, 8, 128, dt) == size(1 << 16, 8, 64, 8, 128, dt)   # bounded by the device


def test_binding_refuses_wrong_shapes_and_types(lib):
    b = Batch8([(20, 2)], 4, 2, 64, 8, torch.float32)
    q, offs, k, v, ks, vs, pages, lens = b.args("cpu")
    rows = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        ra.tree_attn_q8(q, offs, k, v, ks, vs, pages, lens)
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        ra.tree_attn_q8(q, offs, k.float(), v.float(), ks, vs, pages, lens)
    with pytest.raises(ValueError, match="alike"):
        ra.tree_attn_q8(q, offs, k, v.float(), ks, vs, pages, lens)
    with pytest.raises(ValueError, match="scales"):
        ra.tree_attn_q8(q, offs, k, v, ks.transpose(1, 2).contiguous(), vs, pages, lens)
    with pytest.raises(ValueError, match="scales"):
        ra.tree_attn_q8(q, offs, k, v, ks, vs.float(), pages, lens)
    with pytest.raises(ValueError, match="disagree"):
        ra.tree_attn_q8(torch.zeros(2, 4, 128), offs, k, v, ks, vs, pages, lens)
    with pytest.raises(TypeError, match="dtype"):
        ra.tree_attn_q8(q.half(), offs, k, v, ks, vs, pages, lens)
    with pytest.raises(ValueError, match="tree_mask"):
        ra.tree_attn_q8(q, offs, k, v, ks, vs, pages, lens, tree_mask=torch.zeros(2, 0, dtype=torch.bool))
    with pytest.raises(ValueError, match="int32"):
        ra.tree_attn_q8(q, offs.long(), k, v, ks, vs, pages, lens)
    with pytest.raises(ValueError, match="k_rows"):
        ra.cache_append_q8(rows, rows[:, :1], offs, k, v, ks, vs, pages, lens)
    with pytest.raises(ValueError, match="k_rows"):
        ra.cache_append_q8(rows, rows.bfloat16(), offs, k, v, ks, vs, pages, lens)
    with pytest.raises(TypeError, match="dtype"):
        ra.cache_append_q8(rows.half(), rows.half(), offs, k, v, ks, vs, pages, lens)
    with pytest.raises(TypeError, match="dtype"):
        ra.cache_read_q8(offs, 2, k, v, ks, vs, pages, lens, dtype=torch.float16)
    with pytest.raises(ValueError, match="n_rows"):
        ra.cache_read_q8(offs, -1, k, v, ks, vs, pages, lens)
    with pytest.raises(ValueError, match="k_rows"):
        ra.cache_read_q8(offs, 2, k, v, ks, vs, pages, lens, k_rows=rows)
    with pytest.raises(TypeError, match="kv_lens"):
        ra.cache_append_q8(rows, rows, offs, k, v, ks, vs, pages, None)


def test_codes_of_the_definition():
    """Values of the format keep themselves; the scale is the least that fits; ties go to the even code."""
    x = torch.tensor([[448.0, -448.0, 1.0, 0.5, 2.0 ** -9, 0.0, 17.0, 19.0]])
    e = scale_bytes(x)
    assert e.tolist() == [127]
    assert value(codes(x, e), e).tolist() == [[448.0, -448.0, 1.0, 0.5, 2.0 ** -9, 0.0, 16.0, 20.0]]
    assert scale_bytes(torch.tensor([[449.0], [448.0], [224.0], [224.1], [0.0], [1e-45]])).tolist() == [128, 127, 126, 127, 1, 1]
    g = torch.Generator().manual_seed(1)
    y = torch.randn(500, 16, generator=g)
    e = scale_bytes(y)
    assert torch.equal(codes(y, e), (y.double() / torch.exp2(e.double() - 127)[:, None]).float().to(E4M3).view(torch.uint8))
    off = (value(codes(y, e), e) - y.double()).abs()
    step = torch.exp2(e.double() - 127)[:, None]
    assert (off <= torch.maximum(y.double().abs() * 2.0 ** -4, 2.0 ** -10 * step)).all()


def test_attention_bound_adds_to_that_of_16_bits():
    b = Batch8([(40, 3)], 4, 2, 64, 8, torch.bfloat16, seed=2)
    out, lse, e_out, e_lse = attention_q8(b)
    assert out.isfinite().all() and (lse > -math.inf).all() and (e_out < 0.05).all() and (e_lse < 1e-3).all()
