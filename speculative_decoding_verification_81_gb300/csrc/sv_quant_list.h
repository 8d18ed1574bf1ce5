// sv_quant_list.h -- the work list of the attention over pages held in 4 bits,
// form for few rows, as arithmetic on host or device.
//
// An item is up to `tok` consecutive rows of one sequence and one KV head (all the
// heads that share it); its units are kRowsItemCost and one for each 128-slot tile that
// its rows see (a tile is a unit of 16 slots for each of a CTA's eight warps).  The
// list runs over sequences, then KV heads, then items, and is cut as the
// other form's is (sv_chunk_list.h): CTA c of nctas takes units floor(U c / nctas)
// .. floor(U (c + 1) / nctas) - 1 of the U.
#pragma once

#include "sv_chunk_list.h"

namespace sv {
namespace chunk {

constexpr int kRowsItemCost = 2;  // an item's start, its warps' meeting and its stores, in tiles
// Units of a CTA at least.  Measured, us, with 1, 2, 3 and 8 (32 query over 8 KV heads of 128): one token after 511
// slots 10.1, 10.8, 12.1, 16.1, after 2047 11.8, 11.6, 13.0, 20.4, after 8191 16.4, 15.4, 15.4, 21.6; 8 single tokens
// after 511 11.4, 11.5, 12.9, 19.2; chains of 4 for 4 requests after 2047 17.4, 17.4, 18.3, 28.1.
constexpr int kRowsMinUnits = 2;

struct RowsShape {
    int tok;     // rows of an item
    int window;  // slots a row sees at most, 0: all
    int num_rows, S_max;
};

struct RowsSeq {
    int L, n;   // filled slots, new rows (0: none, or refused)
    int row0;   // its first row
    int items;  // of one KV head
};

SV_HD RowsSeq rows_seq(const RowsShape &p, int L, int r0, int r1) {
    const Shape s{1, p.window, p.num_rows, p.S_max};
    RowsSeq q;
    q.L = L;
    q.row0 = r0;
    q.n = lengths_ok(s, L, r0, r1) ? r1 - r0 : 0;
    q.items = q.n == 0 ? 0 : (q.n - 1) / p.tok + 1;
    return q;
}

// The first tile that the row at position pos sees.
SV_HD int rows_first_tile(const RowsShape &p, int pos) {
    return p.window > 0 && pos >= p.window ? (pos - p.window + 1) / kTileSlots : 0;
}

// K/V tiles of item i.
SV_HD int rows_tiles(const RowsShape &p, const RowsSeq &s, int i) {
    const int t0 = i * p.tok, t1 = s.n - t0 < p.tok ? s.n : t0 + p.tok;
    return (s.L + t1 + kTileSlots - 1) / kTileSlots - rows_first_tile(p, s.L + t0);
}

// Units of items 0 .. i - 1 of one KV head.
SV_HD_CALL long long rows_units_before(const RowsShape &p, const RowsSeq &s, int i) {
    if (i <= 0) return 0;
    long long u = (long long)i * kRowsItemCost;
    if (i == s.items) u += rows_tiles(p, s, --i);  // the last item may be short
    if (i > 0) {
        const uint32_t tok = p.tok;
        u += floor_sum(i, tok, s.L + tok + kTileSlots - 1);
        if (p.window > 0) {
            // first tiles: floor((L + k tok - window + 1) / 128), from the first k at which that is >= 0
            const long long c = (long long)s.L - p.window + 1;
            const long long k0 = c >= 0 ? 0 : (-c + tok - 1) / tok;
            if (k0 < i) u -= floor_sum((uint32_t)(i - k0), tok, (uint32_t)(c + k0 * tok));
        }
    }
    return u;
}

// CTAs that take part, of `grid`.
SV_HD int rows_ctas(long long U, int grid) {
    const long long want = U / kRowsMinUnits > 0 ? U / kRowsMinUnits : 1;
    return want < grid ? (int)want : grid;
}

}  // namespace chunk
}  // namespace sv
