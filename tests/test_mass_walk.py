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
    assert got[NAMES[1]] == 0, got
    assert got[NAMES[0]] == 0, got
    if kind == "alternating" and heads in (1, 3) and not tree and n <= rpt:
        assert got["places for the lse rule"] > 0
