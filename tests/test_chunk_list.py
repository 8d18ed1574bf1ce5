"""The chunk attention's work list, compiled for the host: closed-form units
against counting, and the CTAs' ranges covering every (sequence, KV head,
item, tile) once, with the same sharing seen by every CTA of a cut item."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COST = 8  # units of an item's start and end
SRC = r"""
#include "sv_chunk_list.h"
using namespace sv::chunk;
extern "C" long long c_floor_sum(uint32_t n, uint32_t a, uint32_t c) { return floor_sum(n, a, c); }
extern "C" int c_items(int tpt, int window, int L, int n) { return seq_of({tpt, window, 1 << 29, 1 << 29}, L, 5, 5 + n).items; }
extern "C" int c_tiles(int tpt, int window, int L, int n, int i) {
    const Shape p{tpt, window, 1 << 29, 1 << 29};
    return item_tiles(p, seq_of(p, L, 5, 5 + n), i);
}
extern "C" long long c_before(int tpt, int window, int L, int n, int i) {
    const Shape p{tpt, window, 1 << 29, 1 << 29};
    return units_before(p, seq_of(p, L, 5, 5 + n), i);
}
extern "C" int c_valid(int L, int r0, int r1, int rows, int smax) { return seq_of({32, 0, rows, smax}, L, r0, r1).n; }
extern "C" int c_ctas(long long U, long long items, int most, int grid) { return ctas_for(U, items, most, grid); }
extern "C" int c_bound(int tpt, int window, int most) { return units_bound({tpt, window, 1 << 29, 1 << 29}, most); }
extern "C" int c_whole(long long U, long long items, int most, int n, int grid) { return whole_items(U, items, most, n, grid); }
extern "C" void c_cut(long long ui, int n, int w, long long U, int nctas, int cta, int *out) {
    const Cut c = cut_item(ui, n, w, cta_begin(U, nctas, cta), cta_begin(U, nctas, cta + 1));
    out[0] = c.a; out[1] = c.z;
    out[2] = cta_of(U, nctas, tile_unit(ui, w, 0));
    out[3] = cta_of(U, nctas, tile_unit(ui, w, n - 1)) - out[2] + 1;
}
"""


@pytest.fixture(scope="module")
def C(tmp_path_factory):
    d = tmp_path_factory.mktemp("chunk_list")
    (d / "shim.cpp").write_text(SRC)
    inc = os.path.join(ROOT, "speculative_decoding_verification_81_gb300", "csrc")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                           "-fno-sanitize-recover", "-static-libubsan", f"-I{inc}", str(d / "shim.cpp"),
                           "-o", str(d / "shim.so")])
    L = ctypes.CDLL(str(d / "shim.so"))
    L.c_floor_sum.argtypes = [ctypes.c_uint32] * 3
    L.c_floor_sum.restype = L.c_before.restype = ctypes.c_longlong
    L.c_cut.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int,
                        ctypes.c_int, ctypes.c_void_p]
    L.c_whole.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int]
    L.c_ctas.argtypes = [ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_int]
    return L


def tiles(tpt, window, L, n, i):
    t0, t1 = i * 2 * tpt, min((i + 1) * 2 * tpt, n)
    lo = max(0, L + t0 - window + 1) if window else 0
    return (L + t1 - 1) // 128 - lo // 128 + 1


def weight(tpt, n, i):
    return 3 if n - i * 2 * tpt > tpt else 2  # two Q tiles or one


def test_floor_sum(C):
    rng = np.random.default_rng(1)
    for _ in range(500):
        n, a, c = (int(rng.integers(lo, hi)) for lo, hi in ((0, 300), (0, 600), (0, 5000)))
        assert C.c_floor_sum(n, a, c) == sum((a * i + c) // 128 for i in range(n)), (n, a, c)
    for n, a, c in ((1 << 22, 256, (1 << 30) - 1), (1 << 22, 254, (1 << 30) - 1), (1 << 22, 250, 12345)):
        assert C.c_floor_sum(n, a, c) == sum((a * i + c) // 128 for i in range(n))  # the largest lengths
    # items of two tokens up to the longest sequence: in closed form, i // 64 for c = 0
    n = 1 << 29
    q, r = divmod(n, 64)
    assert C.c_floor_sum(n, 2, 0) == 64 * q * (q - 1) // 2 + q * r
    # slope 127: floor(127 i / 128) = i - ceil(i / 128)
    assert C.c_floor_sum(n, 127, 0) == n * (n - 1) // 2 - _ceil_sum(n)


def _ceil_sum(n):
    """Sum of ceil(i / 128) for i < n."""
    q, r = divmod(n - 1, 128)
    return 128 * q * (q + 1) // 2 + (q + 1) * r


def test_units_closed_form(C):
    rng = np.random.default_rng(2)
    for _ in range(300):
        tpt = int(rng.choice([1, 2, 9, 18, 32, 42, 64, 128]))
        window = int(rng.choice([0, 1, 7, 128, 129, 1000, 1 << 29]))
        L, n = int(rng.integers(0, 3000)), int(rng.integers(1, 1500))
        items = C.c_items(tpt, window, L, n)
        assert items == -(-n // (2 * tpt))
        total = 0
        for i in range(items):
            assert C.c_before(tpt, window, L, n, i) == total, (tpt, window, L, n, i)
            assert C.c_tiles(tpt, window, L, n, i) == tiles(tpt, window, L, n, i)
            total += COST + weight(tpt, n, i) * tiles(tpt, window, L, n, i)
        assert C.c_before(tpt, window, L, n, items) == total


def test_refused_lengths_have_no_rows(C):
    assert C.c_valid(10, 0, 5, 5, 15) == 5
    assert C.c_valid(10, 0, 5, 4, 15) == 0    # rows past num_rows
    assert C.c_valid(10, 0, 5, 5, 14) == 0    # slots past the table
    assert C.c_valid(-1, 0, 5, 5, 15) == 0
    assert C.c_valid(0, 5, 4, 9, 15) == 0     # descending
    assert C.c_valid(0, -1, 4, 9, 15) == 0
    assert C.c_valid(2 ** 31 - 1, 0, 5, 5, 2 ** 30) == 0
    assert C.c_valid(0, -2 ** 31, 2 ** 31 - 1, 5, 15) == 0
    assert C.c_valid(3, 2, 2, 5, 15) == 0     # no rows


@pytest.mark.parametrize("sms", [152, 7, 3])
def test_ranges_cover_every_tile_once(C, sms):
    rng = np.random.default_rng(3)
    out = (ctypes.c_int * 4)()
    for _ in range(25):
        tpt = int(rng.choice([1, 18, 32, 128]))
        window = int(rng.choice([0, 0, 200]))
        hkv = int(rng.integers(1, 5))
        seqs = [(int(rng.integers(0, 1200)), int(rng.choice([1, 1, int(rng.integers(1, 400))])))
                for _ in range(int(rng.integers(1, 9)))]
        items = [(tiles(tpt, window, L, n, i), weight(tpt, n, i)) for L, n in seqs for _ in range(hkv)
                 for i in range(-(-n // (2 * tpt)))]
        U = sum(COST + n * w for n, w in items)
        nctas = C.c_ctas(U, len(items), max(COST + n * w for n, w in items), sms)
        assert 1 <= nctas <= sms and (nctas == 1 or U // nctas >= 8)
        ui, slots = 0, set()
        for n, w in items:
            parts = []
            for cta in range(nctas):
                C.c_cut(ui, n, w, U, nctas, cta, ctypes.addressof(out))
                a, z, first, nc = out
                if a < z:
                    parts.append((cta, a, z, first, nc))
            assert [p[1] for p in parts] == [0] + [p[2] for p in parts[:-1]] and parts[-1][2] == n
            for k, (cta, a, z, first, nc) in enumerate(parts):
                assert (first, nc) == (parts[0][0], len(parts)) and cta == first + k
                if nc > 1:  # a CTA's partial slots are its own: the item it begins, or the one it continues
                    assert (cta, k == 0) not in slots
                    slots.add((cta, k == 0))
            ui += COST + n * w


def test_few_items_kept_whole(C):
    """With every item as long as the largest, the CTAs' ranges hold an item each, uncut."""
    rng = np.random.default_rng(8)
    taken = 0
    for _ in range(300):
        items, grid = int(rng.integers(1, 200)), 152
        n = [int(x) for x in rng.integers(1, rng.integers(2, 20), items)]
        w = [int(x) for x in rng.integers(2, 4, items)]
        units = [a * b + COST for a, b in zip(n, w)]
        U, most = sum(units), max(units)
        whole = C.c_whole(U, items, most, C.c_ctas(U, items, most, grid), grid)
        if items > grid or len(set(units)) == 1:
            assert not whole
        if not whole:
            continue
        taken += 1
        out = (ctypes.c_int * 4)()
        for i in range(items):
            C.c_cut(i * most, n[i], w[i], items * most, items, i, out)
            assert list(out) == [0, n[i], i, 1]
    assert taken > 50


def test_no_item_exceeds_the_bound(C):
    """The largest of a sequence's last two items, and the bound with a window, against every item."""
    rng = np.random.default_rng(9)
    for k in range(400):
        tpt, window = int(rng.choice([1, 2, 4, 16, 32, 128])), int(rng.choice([0, 0, 1, 2, 92, 128, 129, 1000]))
        L, n = int(rng.integers(0, 1500)), int(rng.integers(1, 600))
        items = C.c_items(tpt, window, L, n)
        units = [tiles(tpt, window, L, n, i) * weight(tpt, n, i) + COST for i in range(items)]
        assert max(units) <= C.c_bound(tpt, window, max(units[-2:])), (tpt, window, L, n)
