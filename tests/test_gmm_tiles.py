"""The grouped products' tile cutting (moe_ffn_gb300/csrc/gmm_tiles.cuh),
compiled for the host: the tiles cover every (row, weight tile) of every group
exactly once, stay inside their group and within the token tile, and number at
most max_tiles; offsets out of order or out of range are clamped, so no tile
leaves [0, M)."""
import ctypes
import os
import random
import subprocess
import tempfile

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def cut():
    so = os.path.join(tempfile.mkdtemp(prefix="gmm_tiles_"), "libgmm_tiles.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-x", "c++", "-o", so,
                    os.path.join(HERE, "host", "gmm_tiles.cpp")], check=True)
    lib = ctypes.CDLL(so)

    def f(offsets, M, nt, nb, step=16):
        E = len(offsets) - 1
        cap = 200000
        out = (ctypes.c_int * (5 * cap))()
        ok, bound = ctypes.c_int(), ctypes.c_longlong()
        n = lib.gmm_tiles_host((ctypes.c_int * (E + 1))(*offsets), E, M, nt, step, nb, out, cap,
                               ctypes.byref(ok), ctypes.byref(bound))
        assert n >= 0
        return [tuple(out[5 * t:5 * t + 5]) for t in range(n)], bool(ok.value), bound.value
    return f


def offsets_of(sizes, start=0):
    o = [start]
    for s in sizes:
        o.append(o[-1] + s)
    return o


@pytest.mark.parametrize("nt,step", [(16, 16), (32, 16), (64, 16), (128, 16), (256, 16), (128, 32), (256, 32)])
@pytest.mark.parametrize("seed", range(6))
def test_tiles_cover_groups_once(cut, nt, step, seed):
    g = random.Random(seed)
    E = [1, 2, 7, 40, 130, 1024][seed]
    sizes = [g.choice([0, 0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 255, 256, 257, 300])
             for _ in range(E)]
    start = g.choice([0, 5])
    off = offsets_of(sizes, start)
    M = off[-1] + g.choice([0, 9])
    nb = g.choice([1, 3])
    if M == 0:
        return
    tiles, ok, bound = cut(off, M, nt, nb, step)
    assert ok and len(tiles) <= bound
    seen = set()
    for e, nbi, row0, nv, np_ in tiles:
        assert 0 < nv <= np_ <= nt and np_ % step == 0 and np_ - nv < step
        assert off[e] <= row0 and row0 + nv <= off[e + 1] and 0 <= nbi < nb
        for r in range(row0, row0 + nv):
            assert (r, nbi) not in seen
            seen.add((r, nbi))
    assert len(seen) == sum(sizes) * nb


@pytest.mark.parametrize("off,M", [
    ([0, 5, 3, 9], 9), ([-4, 2, 6], 6), ([0, 50, 60], 20), ([7, 3, -1], 10),
    ([2**31 - 1, -2**31, 2**31 - 1], 8), ([4, 4, 4], 8),
])
def test_bad_offsets_stay_inside(cut, off, M):
    tiles, ok, _ = cut(off, M, 32, 2)
    in_order = all(0 <= a <= b <= M for a, b in zip(off, off[1:]))
    assert ok == in_order
    for _, _, row0, nv, np_ in tiles:
        assert 0 <= row0 and nv > 0 and row0 + nv <= M and np_ <= 32
