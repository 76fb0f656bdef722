"""Which kernel a grouped product takes, how it cuts a group and how a warp finds
its group, from the library's own code compiled for the host."""
import ctypes
import random

import pytest

from tests import gmm_plan as plan
from tests.test_gmm_tiles import cut, offsets_of  # noqa: F401  (cut is a fixture)

# (step of the MMA's N side, token tile) of every kernel
KERNEL_TILES = [(16, plan.FEW), (32, plan.SWIGLU_PAIRS), (32, plan.NARROW), (32, plan.WIDE_F8),
                (32, plan.WIDE_16)]


@pytest.mark.parametrize("step,nt", KERNEL_TILES)
@pytest.mark.parametrize("nb", [1, 2, 5])
def test_every_kernels_cut(cut, step, nt, nb):  # noqa: F811
    """Every size of one group up to five tiles and two past them: each (row,
    weight tile) once, no more tiles than the launch counts on, no tile empty."""
    for rows in list(range(1, 5 * nt + 3)):
        tiles, ok, bound = cut([3, 3 + rows], rows + 7, nt, nb, step)
        assert ok and len(tiles) <= bound
        seen = []
        for e, nbi, row0, nv, np_ in tiles:
            assert e == 0 and 0 < nv <= np_ <= nt and np_ % step == 0 and np_ - nv < step
            seen += [(nbi, r) for r in range(row0, row0 + nv)]
        assert sorted(seen) == [(b, r) for b in range(nb) for r in range(3, 3 + rows)]


@pytest.mark.parametrize("step,nt", KERNEL_TILES)
@pytest.mark.parametrize("seed", range(4))
def test_every_kernels_cut_of_ragged_groups(cut, step, nt, seed):  # noqa: F811
    g = random.Random(seed)
    E = [3, 33, 64, 257][seed]
    sizes = [g.choice([0, 0, 1, nt - 1, nt, nt + 1, 2 * nt + 1, 3 * nt, g.randint(0, 4 * nt)])
             for _ in range(E)]
    off = offsets_of(sizes, 2)
    tiles, ok, bound = cut(off, off[-1] + 1, nt, 2, step)
    assert ok and len(tiles) <= bound
    rows = sorted((nbi, r) for e, nbi, row0, nv, _ in tiles for r in range(row0, row0 + nv)
                  if off[e] <= r < off[e + 1])
    assert rows == [(b, r) for b in range(2) for r in range(2, off[-1])]


def test_short_last_tile_is_as_stated(cut):  # noqa: F811
    tiles, _, _ = cut([0, 193], 193, 96, 1, 32)
    assert [t[3] for t in tiles] == [96, 96, 1]


@pytest.mark.parametrize("E", [1, 31, 32, 33, 64, 65, 256, 1024])
def test_group_search(E):
    """The search that a warp makes, 32 groups at a step, empty groups among them."""
    g = random.Random(E)
    for _ in range(20):
        n = [g.choice([0, 0, 1, 3]) for _ in range(E)]
        pre = [0]
        for v in n:
            pre.append(pre[-1] + v)
        arr = (ctypes.c_int * (E + 1))(*pre)
        owners = [e for e in range(E) for _ in range(n[e])]
        for t, e in enumerate(owners):
            assert plan.host().group_of_host(t, arr, E) == e


@pytest.mark.parametrize("want,kind,m,n,groups", [
    (plan.FEW, "f8", 1, 4096, None), (plan.FEW, "f8", 32, 151936, None),
    (plan.FEW, "bf16", 8, 768, 128), (plan.FEW, "f8", 600, 1024, None),
    (plan.NARROW, "f8", 33, 20000, None), (plan.NARROW, "f8", 4096, 1024, 64),
    (plan.NARROW, "f8", 260, 4096, None), (plan.WIDE_F8, "f8", 640, 4096, None),
    (plan.WIDE_F8, "f8", 4096, 14336, None), (plan.WIDE_F8, "f8", 32768, 2048, 128),
    (plan.NARROW, "bf16", 260, 4096, 1), (plan.WIDE_16, "bf16", 640, 4096, 1),
    (plan.WIDE_16, "f16", 16384, 4096, 8)])
def test_choice_of_kernel(want, kind, m, n, groups):
    """The documented choices, at 152 SMs."""
    assert plan.kernel(kind, m, n, groups) == want


@pytest.mark.parametrize("want,pairs,n,E", [
    (plan.FEW, 8, 768, 128), (plan.FEW, 600, 256, 3), (plan.SWIGLU_PAIRS, 4096, 1024, 64),
    (plan.SWIGLU_PAIRS, 32768, 768, 128), (plan.SWIGLU_PAIRS, 2800, 640, 4)])
def test_choice_of_kernel_for_swiglu(want, pairs, n, E):
    assert plan.kernel("f8", pairs, n, E, swiglu=True) == want
