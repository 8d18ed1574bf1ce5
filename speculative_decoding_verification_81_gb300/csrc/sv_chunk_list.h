// sv_chunk_list.h -- the work list of the chunk attention as arithmetic on
// host or device: items of a sequence, their units, and the cut of the list
// into the CTAs' ranges.
//
// An item is up to 2 tpt consecutive rows of one sequence and one KV head (one
// or two Q tiles); its units are kItemCost and, for each 128-slot K/V tile that
// its rows see, kOne or kTwo: a tile of two Q tiles takes about 1.6 times as
// long as one of one, whose loads set its pace, and an item's start and end
// about as long as two to three tiles (48 tokens beside 2 chunks: 112 us at 1
// to 2 and 4, 106 us at these).
// The list runs over sequences, then KV heads, then items; CTA c of nctas
// takes units floor(U c / nctas) .. floor(U (c + 1) / nctas) - 1 of the U.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SV_HD __host__ __device__ __forceinline__
// out of line on the device: the walking warp's instructions share the
// instruction caches with the loops that set the pace
#define SV_HD_CALL __host__ __device__ __noinline__ static
#else
#define SV_HD inline
#define SV_HD_CALL inline
#endif

namespace sv {
namespace chunk {

constexpr int kTileSlots = 128;
constexpr int kOne = 2, kTwo = 3;  // units of a K/V tile for an item of one and of two Q tiles
constexpr int kItemCost = 8;       // units of an item's start and end

// Sum of floor((a i + c) / 128) for i = 0 .. n - 1: the quotients' whole parts in
// closed form, the rest by exchanging the roles of slope and modulus, as
// Euclid's algorithm does: the published floor sum, lattice points below a
// line (Graham, Knuth and Patashnik, Concrete Mathematics, section 3.5, has
// the sum).  The first round divides by shifts and, with slopes
// that are powers of two, is the last but one; the others divide in 32 bits
// where they can.
SV_HD long long floor_sum(uint32_t n, uint32_t a, uint32_t c) {
    static_assert(kTileSlots == 128, "the shifts");
    if (n == 0) return 0;
    long long s = (long long)n * (n - 1) / 2 * (a >> 7) + (long long)n * (c >> 7);
    unsigned long long y = (unsigned long long)(a & 127) * n + (c & 127);
    n = (uint32_t)(y >> 7);
    c = (uint32_t)y & 127;
    uint32_t m = a & 127;
    a = 128;
    while (n > 0) {  // (m > 0: with m = 0 the sum above is all of it)
        s += (long long)n * (n - 1) / 2 * (a / m);
        a %= m;
        s += (long long)n * (c / m);
        c %= m;
        y = (unsigned long long)a * n + c;
        if (y < m) break;
        if (y >> 32) {
            n = (uint32_t)(y / m);
            c = (uint32_t)(y % m);
        } else {
            n = (uint32_t)y / m;
            c = (uint32_t)y - n * m;
        }
        const uint32_t t = m;
        m = a;
        a = t;
    }
    return s;
}

struct Shape {
    int tpt;     // tokens of a Q tile
    int window;  // slots a row sees at most, 0: all
    int num_rows, S_max;
};

struct Seq {
    int L, n;   // filled slots, new rows (0: none, or refused)
    int row0;   // its first row
    int items;  // items per KV head
};

// The lengths of a sequence whose rows are r0 .. r1 - 1 after L slots.
SV_HD bool lengths_ok(const Shape &p, int L, int r0, int r1) {
    return L >= 0 && r0 >= 0 && r1 >= r0 && r1 <= p.num_rows && (long long)L + r1 - r0 <= p.S_max;
}

SV_HD Seq seq_of(const Shape &p, int L, int r0, int r1) {
    Seq s;
    s.L = L;
    s.row0 = r0;
    s.n = lengths_ok(p, L, r0, r1) ? r1 - r0 : 0;
    s.items = s.n == 0 ? 0 : (s.n - 1) / (2 * p.tpt) + 1;
    return s;
}

// The first tile that the row at position pos sees.
SV_HD int first_tile(const Shape &p, int pos) {
    return p.window > 0 && pos >= p.window ? (pos - p.window + 1) / kTileSlots : 0;
}

// K/V tiles of item i.
SV_HD int item_tiles(const Shape &p, const Seq &s, int i) {
    const int t0 = i * 2 * p.tpt, t1 = s.n - t0 < 2 * p.tpt ? s.n : t0 + 2 * p.tpt;
    return (s.L + t1 + kTileSlots - 1) / kTileSlots - first_tile(p, s.L + t0);
}

// Units of a K/V tile of item i.
SV_HD int item_weight(const Shape &p, const Seq &s, int i) { return s.n - i * 2 * p.tpt > p.tpt ? kTwo : kOne; }

// Units of item i.
SV_HD int item_units(const Shape &p, const Seq &s, int i) {
    return item_tiles(p, s, i) * item_weight(p, s, i) + kItemCost;
}

// Units of items 0 .. i - 1 of one KV head.
SV_HD_CALL long long units_before(const Shape &p, const Seq &s, int i) {
    if (i <= 0) return 0;
    long long u = 0, tiles = 0;
    if (i == s.items) u = item_units(p, s, --i);  // the last item may be short
    if (i > 0) {
        const uint32_t tok = 2 * p.tpt;
        tiles = floor_sum(i, tok, s.L + tok + kTileSlots - 1);
        if (p.window > 0) {
            // first tiles: floor((L + k tok - window + 1) / 128), from the first k at which that is >= 0
            const long long c = (long long)s.L - p.window + 1;
            const long long k0 = c >= 0 ? 0 : (-c + tok - 1) / tok;
            if (k0 < i) tiles -= floor_sum((uint32_t)(i - k0), tok, (uint32_t)(c + k0 * tok));
        }
    }
    return u + kTwo * tiles + (long long)i * kItemCost;
}

// a / b of a >= 0, b > 0.  Numbers below 2^22, as a short call's are, divide in
// floats: the quotient is off by less than one (two roundings of at most 2^-22
// of it), which the remainder's sign puts right; about a fifth of the time.
SV_HD long long quot(long long a, long long b) {
    if (((unsigned long long)a | (unsigned long long)b) >> 22) return a / b;
    const int x = (int)a, y = (int)b;
#ifdef __CUDA_ARCH__
    int q = (int)__fdividef((float)x, (float)y);
#else
    int q = (int)((float)x / (float)y);
#endif
    const int r = x - q * y;
    q += r < 0 ? -1 : r >= y ? 1 : 0;
    return q;
}

SV_HD long long cta_begin(long long U, int nctas, int c) { return quot(U * c, nctas); }

// The CTA whose range holds unit u.
SV_HD int cta_of(long long U, int nctas, long long u) { return (int)quot((u + 1) * nctas - 1, U); }

// CTAs that take part, of `grid`: each at least kMinUnits units; and where the
// items are few and all alike (their number `items`, the largest and so each
// of `most` units), a multiple of their number, so that ranges end where
// items do.
constexpr int kMinUnits = 8;

SV_HD int ctas_for(long long U, long long items, int most, int grid) {
    const long long want = U / kMinUnits > 0 ? U / kMinUnits : 1;
    int n = want < grid ? (int)want : grid;
    if (items > 0 && items <= n && items * most == U && most < (1 << 20)) {
        const int k = (int)items, parts = n / k;  // CTAs an item
        // a cut item costs its merge, about as long as four tiles
        const int even = (most + parts - 1) / parts + (parts > 1 ? 4 * kOne : 0), flat = (k * most + n - 1) / n + 4 * kOne;
        if (even <= flat) n = k * parts;
    }
    return n;
}

// Units that no item exceeds, of which `most` is the largest of the sequences'
// last two each: without a window those see the most slots; with one, an item
// anywhere may lie across a tile's end, and its tiles' number is bounded by
// the slots that its rows see.
SV_HD int units_bound(const Shape &p, int most) {
    if (p.window == 0 || p.window >= (1 << 20)) return most;
    const int b = kItemCost + kTwo * ((p.window + 2 * p.tpt - 3 + kTileSlots) / kTileSlots + 1);
    return most > b ? most : b;
}

// Whether few items, not all alike, had better stay whole, a CTA each: every
// item is then given `most` units, which none exceeds, so that the ranges of
// `items` CTAs end where items do.  Ranges of n CTAs that end anywhere give
// most CTAs parts of two items, whose starts and ends and merges they pay (7
// prompts of 223 to 446, 12 query over 4 KV heads: 24.4 us, whole 17.5).
SV_HD bool whole_items(long long U, long long items, int most, int n, int grid) {
    // the largest item against a share, an item's cost and a merge (about four tiles)
    return items > 0 && items <= grid && items * most != U && (long long)(most - kItemCost - 4 * kOne) * n <= U;
}

// What of an item of n tiles of w units each, its units starting at ui, falls
// into a CTA's units u0 .. u1 - 1: tiles a .. z - 1 (none if a >= z; a tile is
// the CTA's that has its first unit).  A cut item is shared by the CTAs of
// its first and last tile's first units and all between them (a range is no
// shorter than w, so that each of them has a tile).
struct Cut {
    int a, z;
};

SV_HD long long tile_unit(long long ui, int w, int tile) { return ui + kItemCost + (long long)w * tile; }

// Tiles of an item (n of w units) whose first unit is before unit d of its tiles'.
SV_HD int tiles_before(long long d, int n, int w) {
    if (d <= 0) return 0;
    if (d >= (long long)w * n) return n;
    const int x = (int)d + w - 1;
    return w == kOne ? x / kOne : x / kTwo;
}

SV_HD Cut cut_item(long long ui, int n, int w, long long u0, long long u1) {
    const long long t = ui + kItemCost;  // the first unit of the first tile
    Cut c;
    c.a = tiles_before(u0 - t, n, w);
    c.z = tiles_before(u1 - t, n, w);
    return c;
}

}  // namespace chunk
}  // namespace sv
