// sv_quant_walk.cuh -- the items that a CTA takes of the work list of the
// attention over pages held in 4 bits (sv_quant_list.h).
#pragma once

#include "sv_device.cuh"
#include "sv_quant_rows.h"

namespace sv {
namespace chunk {

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct RowsItem {
    int b, h;          // sequence (-1: no more), KV head
    int row0, ntok;    // first row, tokens
    int pos0;          // position of the first token
    int seq_row0;      // the sequence's first row
    int kt0, n;        // first K/V tile and number of tiles of this run
    int c_first, nc, ci;  // CTAs that share the item's tiles, this one's number among them
};

// The items of this CTA's units, one after another: in shared memory, where one thread goes on from item to item
// (a copy a lane does not fit the registers and went to the stack).
struct RowsWalk {
    long long U, u0, u1, ui;  // ui: first unit of item (b, h, i)
    int nctas, b, h, i;
    RowsSeq seq;
    bool loaded;
};

__device__ __forceinline__ RowsSeq load_seq(const RowsParams &p, int b) {
    return rows_seq(p.rows, p.prefix_lens[b], p.row_starts[b], p.row_starts[b + 1]);
}

__device__ __forceinline__ void next_item(const RowsParams &p, RowsWalk &w, RowsItem &it) {
    it.b = -1;
    while (w.b < p.B && w.ui < w.u1) {
        if (!w.loaded) {
            w.seq = load_seq(p, w.b);
            w.loaded = true;
            w.h = w.i = 0;
        }
        if (w.seq.items == 0 || w.h == p.Hkv) {
            ++w.b;
            w.loaded = false;
            continue;
        }
        const RowsSeq s = w.seq;
        const int i = w.i, h = w.h, n = rows_tiles(p.rows, s, i);
        const long long first = w.ui + kRowsItemCost;  // unit of the first tile
        w.ui = first + n;
        if (++w.i == s.items) w.i = 0, ++w.h;
        const int a = w.u0 > first ? (int)min(w.u0 - first, (long long)n) : 0;
        const int z = w.u1 > first ? (int)min(w.u1 - first, (long long)n) : 0;
        if (a >= z) continue;
        it.b = w.b;
        it.h = h;
        it.row0 = s.row0 + i * p.rows.tok;
        it.ntok = min(p.rows.tok, s.n - i * p.rows.tok);
        it.pos0 = s.L + i * p.rows.tok;
        it.seq_row0 = s.row0;
        it.kt0 = rows_first_tile(p.rows, it.pos0) + a;
        it.n = z - a;
        it.c_first = blockIdx.x;
        it.nc = 1;
        if (it.n < n) {
            it.c_first = cta_of(w.U, w.nctas, first);
            it.nc = cta_of(w.U, w.nctas, first + n - 1) - it.c_first + 1;
        }
        it.ci = (int)blockIdx.x - it.c_first;
        return;
    }
}

// Whether sequence sb has lengths that are none, a page id out of range among those its rows see, or
// parents that are no tree; by a whole warp.
static __device__ __noinline__ bool bad_sequence(const RowsParams &p, int sb, int lane) {
    const int L = p.prefix_lens[sb], first = p.row_starts[sb], end = p.row_starts[sb + 1];
    const RowsSeq s = rows_seq(p.rows, L, first, end);
    bool bad = !lengths_ok(Shape{1, p.rows.window, p.rows.num_rows, p.rows.S_max}, L, first, end);
    if (s.n > 0) {
        const int lo = p.rows.window > 0 ? max(0, L - p.rows.window + 1) : 0;
        const int32_t *trow = p.block_table + (size_t)sb * p.max_pages;
#pragma unroll 1
        for (int j = lo / p.page_size + lane; j <= (L + s.n - 1) / p.page_size; j += 32) {
            const int pg = trow[j];
            if (pg < 0 || pg >= p.num_pages) bad = true;
        }
        if (p.parents) {
            bad = bad || s.n > kTreeNodes;
#pragma unroll 1
            for (int i = lane; i < min(s.n, kTreeNodes); i += 32) {
                const int par = p.parents[first + i];
                if (i == 0 ? par != -1 : par < 0 || par >= i) bad = true;
            }
        }
    }
    return __any_sync(0xffffffffu, bad);
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ long long scan_units(long long x, int lane) {
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}

// This CTA's share of the list and the place where it begins, to `w`, by its kT threads together; warp 0 may
// use it at once.  Up to 32 sequences warp 0 sums alone, a lane a sequence (one token: 4200 cycles, so 2800);
// above, each thread sums a few (`before`, kT of them: the units before each thread's; warp_units, kT / 32).
template <int kT>
__device__ __forceinline__ void plan_walk(const RowsParams &p, long long *warp_units, long long *before, int tid, RowsWalk &w) {
    const int lane = tid & 31, warp = tid >> 5;
    const bool one = p.B <= 32;
    long long U = 0, ui = 0;
    int b = p.B, per = 1;
    RowsSeq s{};
    long long head = 0, x = 0;  // of a lane's sequence: units of a KV head; units up to and with it
    if (one) {
        if (warp > 0) return;
        if (lane < p.B) s = load_seq(p, lane);
        head = rows_units_before(p.rows, s, s.items);
        x = scan_units(head * p.Hkv, lane);
        U = __shfl_sync(0xffffffffu, x, 31);
    } else {
        per = (p.B + kT - 1) / kT;
        const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
        long long mine = 0;
#pragma unroll 1
        for (int k = b0; k < b1; ++k) {
            const RowsSeq q = load_seq(p, k);
            mine += rows_units_before(p.rows, q, q.items) * p.Hkv;
        }
        const long long sum = scan_units(mine, lane);
        if (lane == 31) warp_units[warp] = sum;
        __syncthreads();
        long long base = 0;
#pragma unroll 1
        for (int i = 0; i < kT / 32; ++i) {
            if (i < warp) base += warp_units[i];
            U += warp_units[i];
        }
        before[tid] = base + sum - mine;
        __syncthreads();
        if (warp > 0) return;
    }
    const int nctas = rows_ctas(U, gridDim.x);
    const bool has = U > 0 && (int)blockIdx.x < nctas;
    const long long u0 = has ? cta_begin(U, nctas, blockIdx.x) : 0, u1 = has ? cta_begin(U, nctas, blockIdx.x + 1) : 0;
    int h = 0, first = 0;
    if (has) {
        if (one) {  // the sequence that holds unit u0
            b = __ffs(__ballot_sync(0xffffffffu, u0 < x)) - 1;
            ui = __shfl_sync(0xffffffffu, x - head * p.Hkv, b);
            head = __shfl_sync(0xffffffffu, head, b);
            s.L = __shfl_sync(0xffffffffu, s.L, b);
            s.n = __shfl_sync(0xffffffffu, s.n, b);
            s.row0 = __shfl_sync(0xffffffffu, s.row0, b);
            s.items = __shfl_sync(0xffffffffu, s.items, b);
        } else {  // the last thread with at most u0 units before its sequences, then the sequence
            int at = 0;
#pragma unroll 1
            for (int i = lane; i < kT; i += 32) at += before[i] <= u0;
            at = __reduce_add_sync(0xffffffffu, at) - 1;
            ui = before[at];
#pragma unroll 1
            for (b = at * per; b < p.B; ++b) {
                s = load_seq(p, b);
                head = rows_units_before(p.rows, s, s.items);
                if (ui + head * p.Hkv > u0) break;
                ui += head * p.Hkv;
            }
        }
        h = (int)quot(u0 - ui, head);
        const long long v = u0 - ui - h * head;
        // the last item whose first unit is at most v: 32 candidates at a time
        int span = s.items;
        long long at_item = 0;
#pragma unroll 1
        while (span > 1) {
            const int step = (span + 31) / 32, c = first + lane * step;
            const bool in = lane * step < span;
            const long long u = in ? rows_units_before(p.rows, s, c) : 0;
            const int hit = 31 - __clz(__ballot_sync(0xffffffffu, in && u <= v));  // (lane 0 always)
            at_item = __shfl_sync(0xffffffffu, u, hit);
            first += hit * step;
            span = min(step, span - hit * step);
        }
        ui += h * head + at_item;
    }
    if (lane == 0) {
        w.U = U;
        w.u0 = u0;
        w.u1 = u1;
        w.ui = ui;
        w.nctas = nctas;
        w.b = b;
        w.h = h;
        w.i = first;
        w.seq = s;
        w.loaded = true;
    }
    __syncwarp();
}

}  // namespace chunk
}  // namespace sv
