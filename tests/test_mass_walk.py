"""CPU checks of the order that the roles of the gathered-weight kernel keep: the walk and the rules it uses are
compiled for the host (mass_walk_check.cpp) and followed over batches of many short runs."""
import ctypes
import os
import subprocess

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
NAMES = ("tiles not walked once", "lse overwritten while it may be read", "chunks given back unwaited",
         "chunks taken for others", "places for the lse rule", "places for the chunk rule")


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("mass") / "mass_walk_check.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-o", out,
                    os.path.join(HERE, "mass_walk_check.cpp")], check=True)
    fn = ctypes.CDLL(out).mass_walk_check
    fn.restype = None

    def run(seqs, heads, rpt, tree, ctas):
        kv, n = ((ctypes.c_int * len(seqs))(*x) for x in zip(*seqs))
        got = (ctypes.c_longlong * 6)()
        fn(len(seqs), kv, n, heads, rpt, int(tree), ctas, got)
        return dict(zip(NAMES, got))
    return run


def no_fault(got):
    assert not any(got[x] for x in NAMES[:4]), got


def lengths(kind, count, n):
    """(keys, new tokens) on both sides of one tile of 128 keys."""
    g = torch.Generator().manual_seed(count)
    if kind == "alternating":
        return [((250, 100)[i % 2], min(n, 100)) for i in range(count)]
    keys = torch.randint(1, 400, (count,), generator=g).tolist()
    return [(k, int(torch.randint(0, n + 1, (1,), generator=g))) for k in keys]


@pytest.mark.parametrize("ctas", [148, 152])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kind,count", [("alternating", 600), ("random", 512), ("random", 90)])
@pytest.mark.parametrize("heads", [1, 2, 3, 6])
@pytest.mark.parametrize("n,rpt", [(1, 4), (4, 4), (12, 16), (20, 16), (40, 16), (64, 32)])
def test_lse_sets(check, n, rpt, heads, kind, count, tree, ctas):
    """Warps of a tile wait for one another between two uses of a set of lse."""
    got = check(lengths(kind, count, n), heads, rpt, tree, ctas)
    no_fault(got)
    if kind == "alternating" and heads in (1, 3) and not tree and n <= rpt:
        assert got["places for the lse rule"] > 0


def straddling(count, rpt, seed):
    """Chains of up to two chunks whose new tokens begin in one key tile and end in another."""
    g = torch.Generator().manual_seed(seed)
    seqs = []
    for _ in range(count):
        n = int(torch.randint(rpt + 1, 2 * rpt + 1, (1,), generator=g))
        last = 128 * int(torch.randint(1, 5, (1,), generator=g))   # where the last tile begins
        seqs.append((last + int(torch.randint(1, n - rpt + 1, (1,), generator=g)), n))
    return seqs


@pytest.mark.parametrize("ctas", [148, 152])
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("count", [5, 40, 300])
@pytest.mark.parametrize("rpt", [4, 16, 32])
def test_row_chunks(check, rpt, count, heads, ctas):
    """Every row chunk that is loaded is waited for before it is given back, also where a run starts at a tile that
    the first chunk does not see."""
    got = check(straddling(count, rpt, 7 * count + rpt), heads, rpt, False, ctas)
    no_fault(got)
    assert got["places for the chunk rule"] > 0 or count * heads < 100
