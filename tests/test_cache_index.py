"""Index arithmetic of the paged cache (csrc/cache_index.h), compiled as plain C++: which row a slot is, what
happens to device integers out of range, and that the runs which the tiles are cut into cover each tile once."""
import ctypes
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SRC = r'''
#include "cache_index.h"
using namespace sage2;
extern "C" {
int c_slot_inside(int s, int sh, int mp) { return slot_inside(s, sh, mp); }
int c_page_inside(int p, int n) { return page_inside(p, n); }
long long c_row_of(int p, int H, int h, int sh, int s) { return row_of(p, H, h, sh, s); }
int c_seq_fits(int l, int n, int T, int cap) { return seq_fits(l, n, T, cap); }
void c_seq_clamped(int l, int n, int T, int cap, int* o) { SeqLen s = seq_clamped(l, n, T, cap); o[0] = s.len; o[1] = s.n; }
int c_pair_tiles(int l, int n, int tile) { SeqLen s{l, n}; return pair_tiles(s, tile); }
int c_run_blocks(long long t, int g, int least) { return run_blocks(t, g, least); }
long long c_run_start(long long t, int g, int c) { return run_start(t, g, c); }
int c_run_of(long long p, long long t, int g) { return run_of(p, t, g); }
}
'''


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("index")
    (d / "w.cpp").write_text(SRC)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I",
                           os.path.join(ROOT, "quantized_attention_04_b200", "csrc"), "-o", str(d / "w.so"),
                           str(d / "w.cpp")])
    l = ctypes.CDLL(str(d / "w.so"))
    L, I = ctypes.c_longlong, ctypes.c_int
    l.c_row_of.restype = l.c_run_start.restype = L
    l.c_run_blocks.argtypes = [L, I, I]
    l.c_run_start.argtypes = [L, I, I]
    l.c_run_of.argtypes = [L, L, I]
    return l


BAD = [-2 ** 31, -1, 0, 1, 15, 16, 17, 127, 128, 2 ** 31 - 1]


def test_slots_and_pages(lib):
    for shift in (4, 5, 6, 7):
        page = 1 << shift
        for mp in (1, 3, 100):
            for s in BAD + [mp * page - 1, mp * page]:
                assert bool(lib.c_slot_inside(s, shift, mp)) == (0 <= s < mp * page)
        for p, H, h, s in ((0, 1, 0, 0), (5, 8, 7, 3 * page + 9), (2 ** 24 - 1, 8, 7, page - 1)):
            assert lib.c_row_of(p, H, h, shift, s) == (p * H + h) * page + s % page
    for n in (1, 7, 2 ** 31 - 1):
        for p in BAD + [n - 1]:
            assert bool(lib.c_page_inside(p, n)) == (0 <= p < n)


def test_lengths_out_of_range_are_held_inside(lib):
    out = (ctypes.c_int * 2)()
    for cap in (16, 48, 2 ** 30):
        for T in (1, 5, 1024):
            for l in BAD + [cap, cap - 1, cap + 1, cap - T]:
                for n in BAD + [T, T + 1]:
                    fits = 0 <= n <= T and l >= 0 and l + n <= cap
                    assert bool(lib.c_seq_fits(l, n, T, cap)) == fits, (l, n, T, cap)
                    lib.c_seq_clamped(l, n, T, cap, out)
                    assert lib.c_seq_fits(out[0], out[1], T, cap)
                    if fits:
                        assert (out[0], out[1]) == (l, n)


def test_runs_cover_every_tile_once(lib):
    rng = random.Random(5)
    for _ in range(400):
        total = rng.choice([1, 2, 3, 147, 148, 149, rng.randint(1, 5000), rng.randint(1, 2 ** 40)])
        grid, least = rng.choice([1, 148, 296, 444, 592]), rng.choice([1, 2])
        g = lib.c_run_blocks(total, grid, least)
        assert 1 <= g <= grid and (g == grid or (g - 1) * least < total)
        starts = [lib.c_run_start(total, g, c) for c in range(g + 1)]
        assert starts[0] == 0 and starts[-1] == total
        sizes = [b - a for a, b in zip(starts, starts[1:])]
        assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1
        for c in rng.sample(range(g), min(g, 20)):
            assert lib.c_run_of(starts[c], total, g) == c == lib.c_run_of(starts[c + 1] - 1, total, g)


def test_pairs_of_sequences_with_nothing_asked(lib):
    assert lib.c_pair_tiles(1000, 0, 64) == 0
    assert [lib.c_pair_tiles(l, 1, 64) for l in (0, 62, 63, 64, 127)] == [1, 1, 1, 2, 2]
