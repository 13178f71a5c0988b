"""CPU check of how the tiles of the 8-bit linear layer's products are dealt out:
for any sizes every unit of both products goes to one cluster once, and the parts
of a tile's K follow each other from its first block to its last."""
import ctypes as C
import random
import subprocess

import pytest

from extreme_label_sparse_gb300 import _build

WALK = r"""
#include "linear8_turns.cuh"
#include <vector>

template <int CG>
static int walk(const Plan &pl, int32_t *info)
{
    LinArgs a = {};
    a.p[0] = pl.p[0], a.p[1] = pl.p[1];
    schedule(a, pl.C);
    std::vector<std::vector<int>> seen(2), at(2);  // how often a unit was met, and the K blocks of each tile
    for (int w = 0; w < 2; ++w)
        seen[w].assign(a.p[w].units, 0);
    Unit t;
    int longest = 0;
    for (int c = 0; c < pl.C; ++c) {
        int i = 0;
        for (; unit_at<CG>(a, c, i, t); ++i) {
            const Prod &p = a.p[t.which];
            if (t.id < 0 || t.id >= p.units || seen[t.which][t.id]++)
                return 1;
            if (t.m0 < 0 || t.m0 >= p.M || t.m0 % pl.BM || t.n0 < 0 || t.n0 >= p.N || t.n0 % kBN || t.nk < 1)
                return 2;
            // a unit's place: its tile, and where the part before it ends
            const int tiles = p.mt * p.nt, s = t.id / tiles;
            if (t.k0 != (int)((int64_t)s * p.nk / p.split) || t.k0 + t.nk != (int)((int64_t)(s + 1) * p.nk / p.split))
                return 3;
        }
        // the list has no holes: nothing comes after its end
        for (int j = i; j < i + 3; ++j)
            if (unit_at<CG>(a, c, j, t))
                return 4;
        longest = i > longest ? i : longest;
    }
    for (int w = 0; w < 2; ++w) {
        for (int n : seen[w])
            if (n != 1)
                return 5;
        // all tiles of a part of K are other ones
        const Prod &p = a.p[w];
        if (!p.units)
            continue;
        if (p.units != p.mt * p.nt * p.split)
            return 6;
        at[w].assign(p.mt * p.nt * p.split, 0);
    }
    for (int c = 0; c < pl.C; ++c)
        for (int i = 0; unit_at<CG>(a, c, i, t); ++i) {
            const Prod &p = a.p[t.which];
            const int tile = t.m0 / pl.BM * p.nt + t.n0 / kBN, s = t.id / (p.mt * p.nt);
            if (at[t.which][s * p.mt * p.nt + tile]++)
                return 7;
        }
    const int32_t out[] = {CG, a.p[0].a_mn, a.p[0].units, a.p[1].units, a.p[0].split, a.p[1].split,
                           a.each, a.hi, a.b_hi, a.b_lo, longest};
    for (int i = 0; i < 11; ++i)
        info[i] = out[i];
    return 0;
}

extern "C" int deal(int64_t T, int64_t H, int64_t N, int backward, int dx, int dW, int32_t *info)
{
    Plan p;
    choose_tiles(T, H, N, backward, dx, dW, &p);
    return p.CG == 1 ? walk<1>(p, info) : walk<2>(p, info);
}
"""
NAMES = ("pairs", "dW_first", "units", "units2", "split", "split2", "each", "hi", "b_hi", "b_lo", "longest")


@pytest.fixture(scope="module")
def deal(tmp_path_factory):
    d = tmp_path_factory.mktemp("turns")
    (d / "walk.cpp").write_text(WALK)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", f"-I{_build.CSRC}", str(d / "walk.cpp"), "-o",
                    str(d / "walk.so")], check=True)
    fn = C.CDLL(str(d / "walk.so")).deal
    fn.argtypes = [C.c_int64] * 3 + [C.c_int] * 3 + [C.c_void_p]

    def call(T, H, N, backward=True, dx=True, dW=True):
        info = (C.c_int32 * 11)()
        rc = fn(T, H, N, backward, dx, dW, info)
        assert rc == 0, (rc, T, H, N, backward, dx, dW)
        d = dict(zip(NAMES, info))
        d["pairs"] = d["pairs"] == 2
        return d

    return call


def log_int(r, lo, hi):
    return int(round(lo * (hi / lo) ** r.random()))


def test_every_unit_is_dealt_once(deal):
    r = random.Random(0)
    kinds = set()
    for _ in range(4000):
        T, H, N = log_int(r, 1, 20000), log_int(r, 1, 20000), log_int(r, 1, 200000)
        if T * N * H > 1 << 41:
            continue
        for dx, dW in ((True, True), (True, False), (False, True)):
            d = deal(T, H, N, True, dx, dW)
            if dx and dW:
                kinds.add((d["pairs"], d["dW_first"], d["each"] > 0, d["hi"] > 0, d["b_hi"] > 0, d["b_lo"] > d["b_hi"]))
        deal(T, H, N, False)
    # with one unit at least of the first product in each cluster, and one more in
    # some of them, both kinds of cluster have turns of the second product
    for pairs in (False, True):
        assert (pairs, 1, True, True, True, True) in kinds and (pairs, 0, True, True, True, True) in kinds, pairs


# Sizes of the GPU test of the dealing (test_gpu_blocks8_long.py), each of which takes
# another path: CTAs or pairs, dW or dx first, split along K or not, and each cluster
# with units of the first product and some with one more
def path(pairs, dW_first, each, hi, b_hi, b_lo, split, split2):
    return dict(pairs=pairs, dW_first=dW_first, each=each, hi=hi, b_hi=b_hi, b_lo=b_lo, split=split, split2=split2)


PATHS = [
    (8192, 4096, 4096, path(True, 1, 3, 28, 5, 8, 1, 1)),
    (6000, 1024, 8000, path(True, 1, 1, 52, 1, 2, 1, 1)),
    (1, 8036, 16922, path(False, 0, 1, 8, 10, 29, 5, 1)),
    (1, 263, 18167, path(False, 1, 1, 132, 1, 1, 1, 48)),
    (514, 8275, 1554, path(False, 0, 1, 13, 1, 3, 1, 1)),
    (569, 8479, 794, path(False, 1, 1, 86, 1, 2, 1, 1)),
    (864, 1352, 6130, path(False, 1, 1, 136, 1, 2, 1, 4)),
    (8102, 2678, 317, path(False, 1, 1, 13, 1, 5, 5, 1)),
    (609, 8587, 1165, path(True, 0, 1, 26, 1, 3, 1, 1)),
    (135, 6676, 3999, path(True, 0, 1, 5, 2, 6, 3, 1)),
    (694, 8772, 524, path(True, 1, 1, 29, 1, 2, 1, 1)),
    (998, 339, 18651, path(True, 1, 1, 70, 1, 2, 1, 10)),
    (4004, 6909, 149, path(True, 1, 1, 5, 2, 6, 3, 1)),
    (5965, 528, 2276, path(True, 1, 1, 5, 1, 1, 3, 1)),
]


@pytest.mark.parametrize("T,H,N,want", PATHS)
def test_paths_of_sizes(deal, T, H, N, want):
    d = deal(T, H, N)
    assert {k: d[k] for k in want} == want, d
