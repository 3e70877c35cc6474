"""CPU checks of the paged-cache operators: refusals before any launch, workspace sizes, and the
64-bit definitions the GPU tests use, against closed forms."""
import math

import pytest
import torch

import ring_context_parallelism_gb300 as ra
from ring_context_parallelism_gb300 import ra as rab
from ring_context_parallelism_gb300.build import build
from cache_cases import attention, make_batch, mass, select

BAD, UNS, WS = rab.RA_ERR_INVALID_ARG, rab.RA_ERR_UNSUPPORTED, rab.RA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    build()
    return ra.load()


def _call(fn, base, kw):
    a = dict(base)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return fn(*a.values())


TREE = dict(q=16, offs=16, n_seqs=4, R=10, k=16, v=16, n_pages=64, page=16, pages=16, max_pages=8, lens=16, mask=None,
            cols=0, out=16, lse=None, Hq=16, Hkv=2, D=128, dt=rab.RA_BF16, ws=256, wsb=1 << 40, stream=None)
MASS = dict(q=16, lse=16, offs=16, n_seqs=4, R=10, k=16, n_pages=64, page=16, pages=16, max_pages=8, lens=16, mask=None,
            cols=0, min=None, mout=16, mcols=128, decay=1.0, Hq=16, Hkv=2, D=128, dt=rab.RA_BF16, stream=None)
SELECT = dict(mass=16, mcols=128, lens=16, n_seqs=4, Hkv=2, budget=64, first=4, recent=8, pos=16, counts=16, kept=32,
              kcols=64, stream=None)
MOVE = dict(k=16, v=16, n_pages=64, page=16, src=16, smax=8, dst=32, dmax=8, pos=16, heads=2, count=64, counts=16,
            start=None, n_seqs=4, Hkv=2, D=128, dt=rab.RA_BF16, stream=None)
APPEND = dict(kr=16, vr=16, offs=16, n_seqs=4, R=10, k=16, v=16, n_pages=64, page=16, pages=16, max_pages=8, lens=16,
              Hkv=2, D=128, dt=rab.RA_BF16, stream=None)

POOL = [(dict(k=None), BAD), (dict(k=24), BAD), (dict(n_pages=0), BAD), (dict(page=12), BAD), (dict(page=4), BAD),
        (dict(page=1 << 21), BAD), (dict(D=96), BAD), (dict(dt=5), BAD), (dict(Hkv=0), BAD),
        (dict(n_pages=1 << 27), BAD), (dict(n_seqs=0), BAD)]
BATCH = [(dict(offs=None), BAD), (dict(pages=None), BAD), (dict(lens=None), BAD), (dict(R=-1), BAD),
         (dict(max_pages=0), BAD), (dict(offs=18), BAD), (dict(n_seqs=(1 << 24) + 1), BAD)]


@pytest.mark.parametrize("kw,status", POOL + BATCH + [
    (dict(q=None), BAD), (dict(out=None), BAD), (dict(v=None), BAD), (dict(out=24), BAD), (dict(Hq=15), BAD),
    (dict(Hq=258), UNS), (dict(R=1 << 30), BAD), (dict(mask=16, cols=0), BAD), (dict(ws=None), WS),
    (dict(wsb=64), WS), (dict(ws=272), BAD), (dict(lse=18), BAD)])
def test_tree_attn_refusals(lib, kw, status):
    assert _call(lib.ra_tree_attn_paged, TREE, kw) == status
    assert lib.ra_last_error()


@pytest.mark.parametrize("kw,status", POOL + BATCH + [
    (dict(q=None), BAD), (dict(lse=None), BAD), (dict(mout=None), BAD), (dict(mcols=0), BAD), (dict(Hq=15), BAD),
    (dict(Hq=258), UNS), (dict(decay=math.inf), BAD), (dict(decay=math.nan), BAD), (dict(mask=16, cols=0), BAD),
    (dict(mout=18), BAD)])
def test_key_mass_refusals(lib, kw, status):
    assert _call(lib.ra_key_mass_paged, MASS, kw) == status
    assert lib.ra_last_error()


@pytest.mark.parametrize("kw", [
    dict(mass=None), dict(lens=None), dict(pos=None), dict(counts=None), dict(mcols=0), dict(n_seqs=0), dict(Hkv=0),
    dict(budget=0), dict(first=-1), dict(recent=-1), dict(first=32, recent=33), dict(kcols=63), dict(kept=16),
    dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), dict(pos=18), dict(mcols=(1 << 30) + 1),
    dict(budget=(1 << 30) + 1, kcols=2 ** 31 - 1), dict(kcols=(1 << 30) + 1)])
def test_evict_select_refusals(lib, kw):
    assert _call(lib.ra_evict_select, SELECT, kw) == BAD
    assert lib.ra_last_error()


@pytest.mark.parametrize("kw,status", POOL + [
    (dict(v=None), BAD), (dict(src=None), BAD), (dict(dst=None), BAD), (dict(pos=None), BAD), (dict(counts=None), BAD),
    (dict(smax=0), BAD), (dict(dmax=0), BAD), (dict(heads=3), BAD), (dict(count=-1), BAD),
    (dict(src=16, dst=16, dmax=9), BAD), (dict(start=18), BAD), (dict(count=(1 << 30) + 1), BAD)])
def test_cache_move_refusals(lib, kw, status):
    assert _call(lib.ra_cache_move_paged, MOVE, kw) == status
    assert lib.ra_last_error()


@pytest.mark.parametrize("kw,status", POOL + BATCH + [(dict(kr=None), BAD), (dict(vr=None), BAD), (dict(vr=24), BAD),
                                                      (dict(v=None), BAD), (dict(Hkv=1 << 20), BAD)])
def test_cache_append_refusals(lib, kw, status):
    assert _call(lib.ra_cache_append_paged, APPEND, kw) == status
    assert lib.ra_last_error()


def test_nothing_to_do_launches_nothing(lib):
    assert _call(lib.ra_tree_attn_paged, TREE, dict(R=0, q=None, out=None, ws=None)) == rab.RA_OK
    assert _call(lib.ra_cache_append_paged, APPEND, dict(R=0, kr=None, vr=None)) == rab.RA_OK
    assert _call(lib.ra_cache_move_paged, MOVE, dict(count=0, pos=None)) == rab.RA_OK
    assert lib.ra_last_error() == b""


def test_tree_workspace_size(lib):
    size = ra.tree_attn_workspace_size
    assert size(10, 4, 16, 2, 96) == 0 and size(10, 4, 15, 2, 128) == 0 and size(-1, 4, 16, 2, 128) == 0
    a, b = size(1, 1, 8, 8, 128), size(4096, 8, 64, 8, 128)
    assert 0 < a < b and a % 256 == 0 and b % 256 == 0
    assert size(1 << 20, 8, 64, 8, 128) == size(1 << 16, 8, 64, 8, 128)   # bounded by the device, not by the rows


def test_binding_refuses_wrong_shapes_and_types():
    b = make_batch([(20, 2)], 4, 2, 64, 8, torch.float32)
    args = (b.q, b.offs, b.k_pages, b.v_pages, b.pages, b.lens)
    with pytest.raises(ValueError, match="CUDA"):
        ra.tree_attn(*args)
    with pytest.raises(ValueError, match="int32"):
        ra.tree_attn(b.q, b.offs.long(), *args[2:])
    with pytest.raises(ValueError, match="tree_mask"):
        ra.tree_attn(*args, tree_mask=torch.ones(3, 2, dtype=torch.bool))
    with pytest.raises(ValueError, match="tree_mask"):
        ra.tree_attn(*args, tree_mask=torch.ones(2, 2))
    with pytest.raises(ValueError, match="dtype"):
        ra.tree_attn(b.q.bfloat16(), *args[1:])
    with pytest.raises(ValueError, match="lse"):
        ra.key_mass(b.q, torch.zeros(2, 4), b.offs, b.k_pages, b.pages, b.lens, torch.zeros(1, 2, 32))
    with pytest.raises(ValueError, match="mass"):
        ra.key_mass(b.q, torch.zeros(4, 2), b.offs, b.k_pages, b.pages, b.lens, torch.zeros(1, 3, 32))
    with pytest.raises(ValueError, match="mass"):
        ra.evict_select(torch.zeros(1, 2), b.lens, 4)
    with pytest.raises(ValueError, match="budget"):
        ra.evict_select(torch.zeros(1, 2, 32), b.lens, 0)
    with pytest.raises(ValueError, match="positions"):
        ra.cache_move(b.k_pages, b.v_pages, b.pages, b.pages, torch.zeros(2, 2, 4, dtype=torch.int32), b.lens)
    with pytest.raises(ValueError, match="k_rows"):
        ra.cache_append(b.q, b.q, b.offs, b.k_pages, b.v_pages, b.pages, b.lens)


def test_binding_refuses_other_objects(lib):
    b = make_batch([(20, 2)], 4, 2, 64, 8, torch.float32)
    with pytest.raises(TypeError, match="kv_lens"):
        ra.tree_attn(b.q, b.offs, b.k_pages, b.v_pages, b.pages, [22])
    with pytest.raises(TypeError, match="q_rows"):
        ra.tree_attn(None, b.offs, b.k_pages, b.v_pages, b.pages, b.lens)
    with pytest.raises(TypeError, match="tree_mask"):
        ra.tree_attn(b.q, b.offs, b.k_pages, b.v_pages, b.pages, b.lens, tree_mask=1)
    with pytest.raises(TypeError):
        ra.key_mass(b.q, torch.zeros(4, 2), b.offs, b.k_pages, b.pages, b.lens, torch.zeros(1, 2, 32), decay="1")
    with pytest.raises(TypeError):
        ra.evict_select(torch.zeros(1, 2, 32), b.lens, 4.5)
    with pytest.raises(ValueError, match="n_first"):
        ra.evict_select(torch.zeros(1, 2, 32), b.lens, 4, n_first=1 << 31)
    with pytest.raises(OverflowError):
        ra.evict_select(torch.zeros(1, 2, 32), b.lens, 1 << 70)
    with pytest.raises(TypeError, match="dtype"):
        ra.cache_append(*(t.double() if t.is_floating_point() else t
                          for t in (b.q[:, :2], b.q[:, 2:], b.offs, b.k_pages, b.v_pages, b.pages, b.lens)))
    with pytest.raises(TypeError, match="arguments"):
        (rab._paged or rab._load_paged()).cache_append(b.q)


def test_binding_refuses_empty_optional_tensors(lib):
    """An empty tensor has no address, which the library would take for an argument left out."""
    b = make_batch([(20, 2)], 4, 2, 64, 8, torch.float32)
    empty = torch.zeros(2, 0, dtype=torch.bool)
    with pytest.raises(ValueError, match="tree_mask"):
        ra.tree_attn(b.q, b.offs, b.k_pages, b.v_pages, b.pages, b.lens, tree_mask=empty)
    with pytest.raises(ValueError, match="tree_mask"):
        ra.key_mass(b.q, torch.zeros(4, 2), b.offs, b.k_pages, b.pages, b.lens, torch.zeros(1, 2, 32), tree_mask=empty)
    with pytest.raises(ValueError, match="kept_mass"):
        ra.evict_select(torch.zeros(1, 2, 32), b.lens, 4, kept_mass=torch.zeros(1, 2, 0))


def test_definitions_against_closed_forms():
    """One visible key gives its value and the scaled score; a chain's weights sum to one per row and head;
    equal scores weigh equally."""
    b = make_batch([(1, 1), (9, 3)], 4, 2, 64, 8, torch.float32, seed=3)
    out, lse, _, _ = attention(b)
    assert torch.allclose(out[0], b.v[0][0].double().repeat_interleave(2, 0))
    x = (b.q[0].double() * b.k[0][0].double().repeat_interleave(2, 0)).sum(-1) / 8
    assert torch.allclose(lse[:, 0], x)
    got, _ = mass(b, lse, None, 1.0, 16)
    assert torch.allclose(got[0, :, 0], torch.full((2,), 2.0, dtype=torch.float64))   # two heads of one row
    assert torch.allclose(got[1, :, :9].sum(1), torch.full((2,), 6.0, dtype=torch.float64))
    b.q[1:] = 0
    out, lse, _, _ = attention(b)
    assert torch.allclose(lse[0, 1:], torch.log(torch.tensor([7.0, 8.0, 9.0], dtype=torch.float64)))
    assert torch.allclose(out[3, 0], b.v[1][:, 0].double().mean(0))
    empty = make_batch([(2, 2)], 2, 2, 64, 8, torch.float32, mask="empty")
    out, lse, _, _ = attention(empty)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_select_definition():
    m = torch.tensor([[[5.0, 1.0, 3.0, 3.0, math.nan, -1.0, 0.0, 9.0]]])
    pos, counts, kept = select(m, torch.tensor([8]), 5, 1, 1)
    assert pos.tolist() == [[[0, 1, 2, 3, 7]]] and counts.tolist() == [5]
    assert kept.tolist() == [[[5.0, 1.0, 3.0, 3.0, 9.0]]]
    pos, counts, _ = select(m, torch.tensor([3]), 5, 1, 1)
    assert pos.tolist() == [[[0, 1, 2, -1, -1]]] and counts.tolist() == [3]
