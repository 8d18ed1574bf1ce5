// sv_chunk_tc.cu -- attention of chunks of new tokens over a paged KV cache
// (prompt chunks of any length, mixed with single tokens) on the
// 5th-generation tensor cores.
//
// Source: the paged KV of "Chapitre 9", section "Ce que prépare le Chapitre
// 9"; "Chapitre 9" §9.1 (the prefix's K/V is reused, the new positions attend
// to it and causally to each other in one pass).
//
// Row i of sequence b sits at position p = L_b + i and sees the slots
// max(0, p - window + 1) .. p.  An item is a run of consecutive rows of one
// sequence and one KV head: the G = Hq/Hkv heads of a token share K/V, so a
// Q tile holds tpt = 128 / G tokens (128 MMA rows), and an item one or two
// tiles.  For each 128-slot tile of K/V an item runs one step a Q tile:
//     S = Q K^T (128 x 128, f32 in tensor memory)
//     P = 2^(scale * log2 e * S - m), written over S as bf16
//     O += P V (f32 in tensor memory)
// with a running row maximum m that moves only when it grows by more than
// 2^8 (O is then rescaled) and the row sums of the f32 P.
//
// Two streams of steps alternate, so that the tensor core works on one
// stream's products while the softmax warps of the other turn S into P: the
// steps of a CTA are one list, step g belongs to stream g & 1 (its own S/P
// and O columns and its own four softmax warps).  An item of two Q tiles puts
// a tile on each stream and both read every K/V tile; an item of one Q tile
// (single tokens, short chunks) gives the streams its K/V tiles in turn, and
// their (O, m, sum) are merged at the end.
//
// The work list is every (sequence, KV head, item, K/V tile).  A persistent
// grid takes equal contiguous ranges of it, weighed by what tiles and items take
// (sv_chunk_list.h), so the load is even whatever the lengths;
// an item cut by a range's end leaves partials in the workspace, merged by the
// warp that arrives last, in index order.
//
// Warps: 0-3 and 4-7 softmax of streams 0 and 1 (one thread a row); 8 and 11
// load K and V tiles by TMA through the page table; 9 issues the products; 10
// walks the work list, publishes the items, loads Q and at the end checks the
// page table and writes seq_status.  Every wait is bounded.
//
// What bounds it (32 query over 8 KV heads of 128, one GB300): long chunks the
// tensor core and the power cap -- 4096 rows after 28672 slots 1.19 ms (1.73
// PFLOP/s) after a pause, 1.31-1.38 ms back to back; large batches of single
// tokens HBM -- 128 after 4096 slots 316-321 us, 6.8 TB/s.  In between, a step's chain: S product, softmax of one row a thread
// (about 1400 cycles a tile), PV product; and for short items the instructions
// themselves: the roles' code is fetched through one instruction cache, and
// every shortening of it (loops kept rolled, rare parts out of line) gained
// several per cent.  Tried without gain: P released in two halves; the softmax
// in two or four rounds of columns read twice from tensor memory; with D = 64,
// P in columns of its own so that the next S is made during the softmax;
// products of 64 rows for few rows; the two streams finishing items in turn.
#include "sv_chunk.cuh"

namespace sv {
namespace chunk {

// ---------------------------------------------------------------- small pieces

__device__ __forceinline__ uint32_t sw128(int row, int c) {
    return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4));
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll 1
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}

// A sequence's items and units, of one KV head.
struct Units {
    int items, most;  // most: units of its largest item
    long long per_head;
};

__device__ __forceinline__ Units units_of(const Params &p, int L, int r0, int r1) {
    const Seq s = seq_of(p.shape, L, r0, r1);
    Units u{s.items, 0, 0};
    if (s.items == 1) {
        u.most = item_units(p.shape, s, 0);
        u.per_head = u.most;
    } else if (s.items > 1) {
        // (the last item sees the most slots; a window may leave the one before it a tile more)
        u.most = max(item_units(p.shape, s, s.items - 1), item_units(p.shape, s, s.items - 2));
        u.per_head = units_before(p.shape, s, s.items);
    }
    return u;
}

// Wait for the phase of `bar` with the given parity, by a whole warp with one
// verdict for its lanes; false after kWaitCycles.  The first probe may suspend
// and nearly always suffices; the counting is out of line, so that the loops
// around the waits stay short.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        if (__all_sync(0xffffffffu, ok != 0)) return true;
        if (__any_sync(0xffffffffu, clock64() - t0 > kWaitCycles)) return false;
    }
}
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || wait_long(smem_u32(bar), parity);
}

// 1 in one lane of the (converged) warp, 0 in the others.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// A value that is the same in every lane, as one the compiler knows to be.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// The commit of tc::, run by a whole warp and issued by its lane with leader = 1.
__device__ __forceinline__ void commit(uint32_t leader, uint64_t *bar) {
    if (leader) tc::commit(bar);
}

// Stream s's S = Q K^T, from the descriptors of its Q tile and the K tile; by a
// whole warp, issued by its lane with leader = 1 (as the next).
template <int D>
__device__ __forceinline__ void s_products(uint32_t leader, uint32_t tbase, uint32_t s, uint64_t dq, uint64_t dk) {
    constexpr uint32_t idesc = tc::idesc_bf16(kRows, kBK, false);
    if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t o = (uint64_t)((kk >> 2) * (kBox >> 4) + (kk & 3) * 2);
            tc::mma_bf16(tbase + kColS + s * kBK, dq + o, dk + o, idesc, kk > 0 ? 1u : 0u);
        }
    }
}
// Stream s's O += P V (O = P V where accumulate is 0); V rows 16kk.. start
// 2048 bytes apart (descriptor units of 16 bytes).
template <int D>
__device__ __forceinline__ void pv_products(uint32_t leader, uint32_t tbase, uint32_t s, uint64_t dv,
                                            uint32_t accumulate) {
    constexpr uint32_t idesc = tc::idesc_bf16(kRows, D, true);
    if (leader) {
#pragma unroll
        for (int kk = 0; kk < kBK / 16; ++kk)
            tc::mma_bf16_ts(tbase + kColO + s * 128, tbase + kColS + s * kBK + kk * 8,
                            dv + (uint64_t)(kk * (2048 >> 4)), idesc, kk > 0 ? 1u : accumulate);
    }
}

// 16 bytes from 8 floats.
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// 32 bytes of a row: in one store where the output is 32-byte aligned, a whole
// sector each lane (two stores of 16 bytes cost the load/store unit twice the
// time with a row a lane; exchanging pieces between lanes first, so that a
// store covers 64 bytes of 8 rows, costs more instructions than it saves).
__device__ __forceinline__ void store32(uint16_t *to, const uint32_t (&x)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(x[0]), "r"(x[1]),
                     "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(to)[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4 *>(to)[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
}

// This warp's O rows (D columns at TMEM address o) times a.
template <int D>
__device__ __noinline__ void rescale_o(uint32_t o, float a) {
#pragma unroll
    for (int h = 0; h < D / 32; ++h) {
        uint32_t ov[32];
        tc::tmem_ld32(o + 32 * h, ov);
        tc::wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * a);
        tc::tmem_st32(o + 32 * h, ov);
    }
    tc::wait_st();
}

// V rows [z0, z1) of a tile zeroed by the 128 threads of a stream, visible to
// the tensor core: slots that no row sees may hold anything, and 0 * NaN
// would reach every row.
template <int D>
__device__ __noinline__ void zero_v_rows(uint8_t *st, int z0, int z1, int t) {
    constexpr int kW = D / 8;  // 16-byte words of a row
    for (int i = t; i < (z1 - z0) * kW; i += 128) {
        const int row = z0 + i / kW, c = i % kW;
        *reinterpret_cast<uint4 *>(st + (c >> 3) * kBox + sw128(row, c & 7)) = make_uint4(0u, 0u, 0u, 0u);
    }
}

// A split item's rows of one warp: partial O (chunk-major, so that a warp's
// lanes, one row each, use consecutive 16 bytes) and (m, sum).
template <int D>
__device__ __forceinline__ float4 *part_o(const Params &p, int cta, int slot, int qt) {
    return reinterpret_cast<float4 *>(p.part_o) + ((size_t)(cta * 2 + slot) * 2 + qt) * (D / 4) * kRows;
}
__device__ __forceinline__ float2 *part_ml(const Params &p, int cta, int slot, int qt) {
    return reinterpret_cast<float2 *>(p.part_ml) + ((size_t)(cta * 2 + slot) * 2 + qt) * kRows;
}

// The nc partials of this warp's rows (row0 .. row0 + nv - 1 of Q tile qt)
// merged in index order and written out, for few rows: a lane takes 8 columns
// of a row and passes over the parts once, eight in flight, with a running
// maximum (a single token spread over many CTAs has many; a round of loads
// takes about a microsecond).  Out of line, since a call runs it once or
// twice.  out_off and lse_off: lane r's row in `out` and `lse`.
template <int D>
__device__ __noinline__ void merge_few(const float4 *part_o, const float2 *part_ml, uint16_t *out, float *lse,
                                       int nc, int nv, int lane, long long out_off, long long lse_off) {
    // from part to part: the first is in its CTA's slot 1, the others in their CTAs' slot 0
    constexpr size_t kO = (size_t)2 * (D / 4) * kRows, kMl = 2 * kRows;  // a slot (two Q tiles)
    constexpr int kParts = 8;
    const int total = nv * (D / 8);
#pragma unroll 1
    for (int idx0 = 0; idx0 < total; idx0 += 32) {
        const int idx = min(idx0 + lane, total - 1), c8 = idx / nv, r = idx - c8 * nv;
        float acc[8] = {}, M = kNegInf, l = 0.f;
#pragma unroll 1
        for (int i0 = 0; i0 < nc; i0 += kParts) {
            float2 ml[kParts];
            float4 x[kParts], y[kParts];
#pragma unroll
            for (int u = 0; u < kParts; ++u) {
                const int i = min(i0 + u, nc - 1), slot = 2 * i + (i == 0 ? 1 : 0);
                ml[u] = __ldcg(part_ml + slot * kMl + r);
                x[u] = __ldcg(part_o + slot * kO + (size_t)(2 * c8) * kRows + r);
                y[u] = __ldcg(part_o + slot * kO + (size_t)(2 * c8 + 1) * kRows + r);
            }
#pragma unroll
            for (int u = 0; u < kParts; ++u) {
                // (a part without a visible slot, its sum 0, weighs nothing; one whose scores are
                // NaN has a maximum of -inf too, and its sum, NaN, goes on)
                if (i0 + u >= nc || ml[u].y == 0.f) continue;
                const float Mn = fmaxf(M, ml[u].x);
                const float f = M == kNegInf ? 0.f : ex2_approx(M - Mn), w = ex2_approx(ml[u].x - Mn);
                M = Mn;
                l = l * f + ml[u].y * w;
                const float o[8] = {x[u].x, x[u].y, x[u].z, x[u].w, y[u].x, y[u].y, y[u].z, y[u].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = __fmaf_rn(o[e], w, acc[e] * f);
            }
        }
        const long long off = __shfl_sync(0xffffffffu, out_off, r);
        const long long loff = __shfl_sync(0xffffffffu, lse_off, r);
        const float inv = 1.f / l;  // (a row sees its own slot: l is 0 or NaN where its scores are not finite)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= inv;
        if (idx0 + lane < total) {
            *reinterpret_cast<uint4 *>(out + off + 8 * c8) = pack8(acc);
            if (lse && c8 == 0) lse[loff] = M * kLn2 + logf(l);
        }
    }
}

// The same for many rows (nv of 16 or more): a lane takes its row, 32 columns
// and two parts at a time.
template <int D>
__device__ __noinline__ void merge_rows(const float4 *part_o, const float2 *part_ml, uint16_t *out, float *lse, int nc,
                                        int nv, int lane, bool wide) {
    constexpr size_t kO = (size_t)2 * (D / 4) * kRows, kMl = 2 * kRows;
    if (lane >= nv) return;
#pragma unroll 1
    for (int h = 0; h < D / 32; ++h) {
        float acc[32] = {}, M = kNegInf, l = 0.f;
#pragma unroll 1
        for (int i0 = 0; i0 < nc; i0 += 2) {
            float2 ml[2];
            float4 o[2][8];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int i = min(i0 + u, nc - 1), slot = 2 * i + (i == 0 ? 1 : 0);
                ml[u] = __ldcg(part_ml + slot * kMl + lane);
#pragma unroll
                for (int c = 0; c < 8; ++c) o[u][c] = __ldcg(part_o + slot * kO + (size_t)(8 * h + c) * kRows + lane);
            }
            // (a part without a visible slot weighs nothing; M stays at -inf before the first that has
            // one; a sum of NaN goes on whatever its weight)
            if (i0 + 1 >= nc) ml[1] = make_float2(kNegInf, 0.f);
            const float Mn = fmaxf(M, fmaxf(ml[0].x, ml[1].x));
            const float base = Mn == kNegInf ? 0.f : Mn;
            const float f = ex2_approx(M - base), w0 = ex2_approx(ml[0].x - base), w1 = ex2_approx(ml[1].x - base);
            M = Mn;
            l = l * f + ml[0].y * w0 + ml[1].y * w1;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float a[4] = {o[0][c].x, o[0][c].y, o[0][c].z, o[0][c].w};
                const float b[4] = {o[1][c].x, o[1][c].y, o[1][c].z, o[1][c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[4 * c + e] = __fmaf_rn(b[e], w1, __fmaf_rn(a[e], w0, acc[4 * c + e] * f));
            }
        }
        const float inv = 1.f / l;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = pack_bf16x2(acc[16 * c + 2 * i] * inv, acc[16 * c + 2 * i + 1] * inv);
            store32(out + 32 * h + 16 * c, x, wide);
        }
        if (lse && h == 0) *lse = M * kLn2 + logf(l);
    }
}

// ---------------------------------------------------------------- the kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap tmk,
                           const __grid_constant__ CUtensorMap tmv,
                           const __grid_constant__ CUtensorMap tmq,
                           const __grid_constant__ CUtensorMap tmq1, const Params p) {
    constexpr int kStages = kStagesOf<D>;
    constexpr int kTile = kTileBytes<D>;
    constexpr int kHalves = D / 64;
    extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle's atoms are 1024 bytes)
    const uint32_t base_u32 = smem_u32(smem);
    uint8_t *qbuf = smem + kStages * kTile;
    const uint32_t q_u32 = base_u32 + kStages * kTile;
    Shared *sh = reinterpret_cast<Shared *>(qbuf + 2 * kTile);

    // (the warp's number as the compiler knows to be the same in all its lanes)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], 1);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->o_full[i], 1);
            mbar_init(&sh->o_empty[i], 4);
            mbar_init(&sh->x_full[i], 4);
        }
#pragma unroll 1
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh->item_full[i], 1);
            mbar_init(&sh->item_empty[i], 11);  // softmax warps, loaders, issuer
        }
        mbar_init(&sh->fin, 1);
        sh->abort_flag = 0;
        fence_mbar_init();
    }
    if (tid == 32 * 8) {
        prefetch_tensormap(&tmk);
        prefetch_tensormap(&tmv);
        prefetch_tensormap(&tmq);
        prefetch_tensormap(&tmq1);
    }
    if (warp == 9) tc::tmem_alloc(&sh->tmem, kCols);

    griddep_wait();
    griddep_launch_dependents();
    if ((base_u32 & 1023u) != 0) {  // (never seen: nothing else takes shared memory here)
        if (p.seq_status)
#pragma unroll 1
            for (int b = tid; b < p.B; b += kThreads) p.seq_status[b] = SV_ERR_CUDA;
        if (tid == 0) {
            const unsigned long long call = begin_call(p.call);
            for (int i = 0; i < kCtaCounters; ++i) p.counters[counters_of(call + 1, gridDim.x, blockIdx.x) + i] = 0;
        }
        __syncthreads();
        if (warp == 9) tc::tmem_dealloc(sh->tmem, kCols);
        return;
    }

    // up to 32 sequences: the walking warp's lengths, on their way while the CTA meets, and the
    // call's number (lane 0; wanted for the first cut item and at the end)
    int pre = 0, r0 = 0, r1 = 0;
    unsigned long long call = 0;
    if (warp == 10 && lane == 0) call = begin_call(p.call);
    if (warp == 10 && p.B <= 32 && lane < p.B) {
        pre = p.prefix_lens[lane];
        r0 = p.row_starts[lane];
        r1 = p.row_starts[lane + 1];
    }
    tc::fence_before();  // (the barriers and the tensor memory's address)
    __syncthreads();
    tc::fence_after();
    // ---- many sequences: the units before each thread's share of them, for the
    // walking warp (up to kWarpPlanB sequences it sums alone), in the still idle Q tiles
    long long *before = reinterpret_cast<long long *>(qbuf);
    const int per = (p.B + kThreads - 1) / kThreads;
    if (p.B > kWarpPlanB) {
        const int b1 = min((tid + 1) * per, p.B);
        long long mine = 0;
        int items = 0, most = 0;
#pragma unroll 1
        for (int b = tid * per; b < b1; ++b) {
            const Units u = units_of(p, p.prefix_lens[b], p.row_starts[b], p.row_starts[b + 1]);
            mine += u.per_head * p.Hkv;
            items += u.items * p.Hkv;
            most = max(most, u.most);
        }
        const long long x = warp_scan(mine, lane);
        items = __reduce_add_sync(0xffffffffu, items);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 31) {
            sh->warp_units[warp] = x;
            sh->warp_items[warp] = items;
            sh->warp_most[warp] = most;
        }
        __syncthreads();
        long long base = 0;
#pragma unroll 1
        for (int w = 0; w < warp; ++w) base += sh->warp_units[w];
        before[tid] = base + x - mine;
        tc::fence_proxy_async_smem();  // (a TMA copy writes there next)
        __syncthreads();
    }
    const uint32_t tbase = sh->tmem;
    volatile int *abort_flag = &sh->abort_flag;
    auto fail = [&] { *abort_flag = 1; };  // (reported at the end, for the whole call)

    if (warp < 8) {
        // ===================== softmax: stream s, one thread a row
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int s = warp >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;  // the row in its Q tile
        const int t = r / p.G, g = r - t * p.G;
        const int t_lo = (quarter * 32) / p.G, t_hi = (quarter * 32 + 31) / p.G;  // the warp's tokens
        const uint32_t tl = tbase + ((uint32_t)(quarter * 32) << 16);
        const uint32_t sbuf = tl + kColS + s * kBK;
        const float sc = p.scale_log2;
        const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
        uint32_t s_ph = 0, o_ph = 0, x_ph = 0;
        uint32_t gstep = 0;       // steps of the CTA before this item
        uint32_t ring = 0;        // K/V ring position of the item's first tile
        bool ok = true;
#pragma unroll 1
        for (uint32_t k = 0;; ++k) {
            const int slot = k % kItems;
            if (!warp_wait_bounded(&sh->item_full[slot], (k / kItems) & 1)) {
                fail();
                break;
            }
            const Item it = sh->items[slot];
            if (it.b < 0) break;
            const bool two = it.ntok > p.shape.tpt;
            const int a = (s ^ (int)gstep) & 1;         // this stream's first step of the item
            const int qt = two ? a : 0;                 // its Q tile
            const int ntok = min(p.shape.tpt, it.ntok - qt * p.shape.tpt);
            const int pos0 = it.pos0 + qt * p.shape.tpt;      // position of the tile's first token
            const int rows = ntok * p.G;                // valid rows of the tile
            const bool active = quarter * 32 < rows;    // the warp has valid rows
            const int pos = pos0 + t;                   // this row's position
            const int see_hi = pos + 1, see_lo = p.shape.window > 0 ? pos - p.shape.window + 1 : 0;
            // tiles all of whose slots every row of the warp sees
            const int w_hi = pos0 + t_lo + 1;
            const int w_lo = p.shape.window > 0 ? pos0 + min(t_hi, ntok - 1) - p.shape.window + 1 : 0;
            const int item_lo = p.shape.window > 0 ? max(0, it.pos0 - p.shape.window + 1) : 0;
            const int item_hi = it.pos0 + it.ntok;
            float m = kNegInf, l = 0.f;
            const int first = two ? 0 : a, stride = two ? 1 : 2;
            const uint32_t o_cols = tl + kColO + s * 128;
#pragma unroll 1
            for (int j = first; j < it.n; j += stride) {
                const int kb = (it.kt0 + j) * kBK;
                // (one probe and a vote nearly always suffice; the slow part in line, since a call
                // here costs the kernel its registers)
                ok = __all_sync(0xffffffffu, mbar_try_wait(&sh->s_full[s], s_ph)) ||
                     warp_wait_bounded(&sh->s_full[s], s_ph);
                if (!ok) break;
                s_ph ^= 1;
                tc::fence_after();
                if (active) {
                    float sv[kBK];
                    {
                        uint32_t ra[32], rb[32], rc[32], rd[32];
                        tc::tmem_ld32(sbuf, ra);
                        tc::tmem_ld32(sbuf + 32, rb);
                        tc::tmem_ld32(sbuf + 64, rc);
                        tc::tmem_ld32(sbuf + 96, rd);
                        tc::wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            sv[i] = __uint_as_float(ra[i]);
                            sv[32 + i] = __uint_as_float(rb[i]);
                            sv[64 + i] = __uint_as_float(rc[i]);
                            sv[96 + i] = __uint_as_float(rd[i]);
                        }
                    }
                    if (kb + kBK > w_hi || kb < w_lo) {
                        // bit i of word i / 32: slot kb + i is at least see_lo and below see_hi
                        const int hi = see_hi - kb, lo = see_lo - kb;
#pragma unroll
                        for (int w = 0; w < kBK / 32; ++w) {
                            const int h = hi - 32 * w, o = lo - 32 * w;
                            const uint32_t below = h >= 32 ? ~0u : h <= 0 ? 0u : (1u << h) - 1u;
                            const uint32_t under = o >= 32 ? ~0u : o <= 0 ? 0u : (1u << o) - 1u;
                            const uint32_t sees = below & ~under;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((sees >> i) & 1u)) sv[32 * w + i] = kNegInf;
                        }
                    }
                    float mq[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                    for (int i = 0; i < kBK; i += 8) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) mq[e] = fmaxf(fmaxf(mq[e], sv[i + e]), sv[i + 4 + e]);
                    }
                    const float c = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * sc;
                    const bool up = c > m + kRescaleThreshold;
                    const bool any_up = __any_sync(0xffffffffu, up);
                    const float f = up ? ex2_approx(m - c) : 1.f;
                    if (up) {
                        m = c;
                        l *= f;
                    }
                    const float nb = m == kNegInf ? 0.f : -m;
                    const float2 nb2 = make_float2(nb, nb), sc2 = make_float2(sc, sc);
                    float2 ls0 = make_float2(0.f, 0.f), ls1 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pk[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float2 x = __ffma2_rn(make_float2(sv[64 * h + 2 * i], sv[64 * h + 2 * i + 1]), sc2, nb2);
                            const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                            if (i & 1) ls1 = __fadd2_rn(ls1, e);
                            else ls0 = __fadd2_rn(ls0, e);
                            pk[i] = pack_bf16x2(e.x, e.y);
                        }
                        tc::tmem_st32(sbuf + 32 * h, pk);
                    }
                    l += (ls0.x + ls0.y) + (ls1.x + ls1.y);
                    // (the wait for S covers this stream's earlier PV products: issued before it)
                    if (any_up && j != first) rescale_o<D>(o_cols, f);
                    tc::wait_st();
                }
                if (kb + kBK > item_hi || kb < item_lo) {
                    const uint32_t pv = ring + 2 * j + 1;
                    if (!(ok = warp_wait_bounded(&sh->full[pv % kStages], (pv / kStages) & 1))) break;
                    uint8_t *st = smem + (pv % kStages) * kTile;
                    if (kb + kBK > item_hi) zero_v_rows<D>(st, max(0, item_hi - kb), kBK, tid & 127);
                    if (kb < item_lo) zero_v_rows<D>(st, 0, min(kBK, item_lo - kb), tid & 127);
                    tc::fence_proxy_async_smem();
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[s]);
            }
            if (!ok) {
                fail();
                break;
            }
            const int steps = two ? it.n : (it.n - a + 1) / 2;
            if (steps > 0) {  // the stream's last PV product of the item
                if (!(ok = warp_wait_bounded(&sh->o_full[s], o_ph))) {
                    fail();
                    break;
                }
                o_ph ^= 1;
                tc::fence_after();
            }
            const bool pair = !two && it.n > 1;  // one Q tile, shared: its first stream finishes it
            if (!two && a == 1) {
                if (steps > 0) {
                    sh->xml[s][r] = make_float2(m, l);
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->x_full[s]);
                }
            } else {
                float m2 = kNegInf, l2 = 0.f;
                if (pair) {
                    if (!(ok = warp_wait_bounded(&sh->x_full[s ^ 1], x_ph))) {
                        fail();
                        break;
                    }
                    x_ph ^= 1;
                    tc::fence_after();
                    m2 = sh->xml[s ^ 1][r].x;
                    l2 = sh->xml[s ^ 1][r].y;
                }
                const bool valid = r < rows;
                const long long row = (long long)it.row0 + qt * p.shape.tpt + t;
                const long long head = (long long)it.h * p.G + g;
                const long long out_off = (row * p.Hq + head) * D, lse_off = row * p.Hq + head;
                const float M = fmaxf(m, m2);
                const float w1 = m == kNegInf ? 0.f : ex2_approx(m - M);
                const float w2 = m2 == kNegInf ? 0.f : ex2_approx(m2 - M);
                const float lt = l * w1 + l2 * w2;
                const bool whole = it.nc == 1;
                const float inv = whole ? 1.f / lt : 1.f;  // (lt: 0 or NaN only where the row's scores are not finite)
                const float f1 = w1 * inv, f2 = w2 * inv;
                const int pslot = it.ci == 0 ? 1 : 0;
                if (active) {
                    if (valid && whole && p.lse) p.lse[lse_off] = M * kLn2 + logf(lt);
                    if (valid && !whole)
                        __stcg(part_ml(p, blockIdx.x, pslot, qt) + r, make_float2(M, lt));
#pragma unroll 1
                    for (int h = 0; h < D / 32; ++h) {  // (short code: most of its time is instruction fetch)
                        uint32_t ov[32];
                        __syncwarp();
                        tc::tmem_ld32(o_cols + 32 * h, ov);
                        tc::wait_ld();
                        float acc[32];
                        // (a share that no row of its tiles sees has O = 0 and f = 0)
#pragma unroll
                        for (int i = 0; i < 32; ++i) acc[i] = __uint_as_float(ov[i]) * f1;
                        if (pair) {
                            tc::tmem_ld32(tl + kColO + (s ^ 1) * 128 + 32 * h, ov);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) acc[i] = __fmaf_rn(__uint_as_float(ov[i]), f2, acc[i]);
                        }
                        if (whole) {
                            if (!valid) continue;
                            uint16_t *to = p.out + out_off + 32 * h;
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                uint32_t x[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) x[i] = pack_bf16x2(acc[16 * c + 2 * i], acc[16 * c + 2 * i + 1]);
                                store32(to + 16 * c, x, wide);
                            }
                        } else if (valid) {
                            float4 *po = part_o<D>(p, blockIdx.x, pslot, qt) + r;
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                __stcg(po + (size_t)(8 * h + c) * kRows,
                                       make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]));
                        }
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) {  // O may start over
                    mbar_arrive(&sh->o_empty[s]);
                    if (pair) mbar_arrive(&sh->o_empty[s ^ 1]);
                }
                if (!whole && active) {
                    int *ctr = p.counters + it.counters + qt * 4 + quarter;
                    int last = 0;
                    if (lane == 0) {  // (its release covers the warp's partials, written before the barrier above)
                        int before_me;
                        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before_me) : "l"(ctr) : "memory");
                        last = before_me == it.nc - 1;
                    }
                    __syncwarp();
                    if (__shfl_sync(0xffffffffu, last, 0)) {
                        const float4 *po = part_o<D>(p, it.c_first, 0, qt) + quarter * 32;
                        const float2 *pm = part_ml(p, it.c_first, 0, qt) + quarter * 32;
                        const int nv = min(32, rows - quarter * 32);
                        // (not through a pointer to either: with an indirect call in it
                        // the kernel is built without its register split)
                        if (nv >= 16) merge_rows<D>(po, pm, p.out + out_off, p.lse ? p.lse + lse_off : nullptr, it.nc, nv, lane, wide);
                        else merge_few<D>(po, pm, p.out, p.lse, it.nc, nv, lane, out_off, lse_off);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
            gstep += two ? 2 * it.n : it.n;
            ring += 2 * it.n;
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
        if (warp == 8 || warp == 11) {
            // ===================== K tiles (warp 8: the even ring positions) and V tiles
            // (warp 11: the odd ones): lane (half, page of the tile)
            const int kv = warp == 11;
            const CUtensorMap *map = kv ? &tmv : &tmk;
            const int ps = p.page_size;
            const int sub = ps < kBK ? ps : kBK;          // rows of a box
            const int npg = kBK / sub;                    // boxes a tile and half
            const int tpp = ps < kBK ? 1 : ps / kBK;      // tiles a page (of 128 slots or more)
            const int pg_l = lane & 15, half = lane >> 4;
            const bool lane_on = pg_l < npg && half < kHalves;
            const uint64_t once = l2_policy_evict_first();
            uint32_t pos = kv;
            bool ok = true;
#pragma unroll 1
            for (uint32_t k = 0; ok; ++k) {
                const int slot = k % kItems;
                if (!wait(&sh->item_full[slot], (k / kItems) & 1)) {
                    fail();
                    break;
                }
                const Item it = sh->items[slot];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
                if (it.b < 0) break;
                const int lo = p.shape.window > 0 ? max(0, it.pos0 - p.shape.window + 1) : 0, hi = it.pos0 + it.ntok;
                const int32_t *trow = p.block_table + (size_t)it.b * p.max_pages;
                // row of this lane's box of tile j in the caches; kNone: no slot of it is seen.  A page id
                // out of range (reported by the check) reads zeros.
                auto box_row = [&](int j) -> int {
                    const int tile = it.kt0 + j, s0 = tile * kBK + pg_l * sub;
                    if (!lane_on || s0 >= hi || s0 + sub <= lo) return kNone;
                    const int page = tpp == 1 ? tile * npg + pg_l : tile / tpp;
                    const int pg = trow[page];
                    if (pg < 0 || pg >= p.num_pages) return -kBK;
                    return (pg * p.Hkv + it.h) * ps + (tpp == 1 ? 0 : (tile - page * tpp) * kBK);
                };
                int y = box_row(0);
#pragma unroll 1
                for (int j = 0; j < it.n && ok; ++j) {
                    const int y_next = j + 1 < it.n ? box_row(j + 1) : kNone;
                    const int boxes = __popc(__ballot_sync(0xffffffffu, y != kNone));
                    const int st = pos % kStages;
                    if (!wait(&sh->empty[st], ((pos / kStages) & 1) ^ 1)) {
                        fail();
                        ok = false;
                        break;
                    }
                    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&sh->full[st], (uint32_t)(boxes * sub * 128));
                    __syncwarp();  // the expected bytes are set before any box lands
                    if (y != kNone) {
                        uint8_t *dst = smem + st * kTile + half * kBox + pg_l * sub * 128;
                        if (it.single) tma_load_2d_hint(dst, map, half * 64, y, &sh->full[st], once);
                        else tma_load_2d(dst, map, half * 64, y, &sh->full[st]);
                    }
                    pos += 2;
                    y = y_next;
                }
            }
            // every copy issued must land before the CTA may exit: the products have
            // waited for all of them, unless a wait gave up
            if (__shfl_sync(0xffffffffu, *abort_flag, 0))
#pragma unroll 1
                for (uint32_t q = pos > kStages ? pos - kStages : kv; q < pos; ++q)
                    if ((q & 1) == (uint32_t)kv) wait(&sh->full[q % kStages], (q / kStages) & 1);
        } else if (warp == 9) {
            // ===================== the products, in step order.  The whole warp runs the
            // loop with values that are the same in every lane (the item's by a
            // warp-wide maximum, the waits' by a vote), and one elected lane
            // issues: a loop that only lane 0 ran made the compiler move
            // every operand of every product to the uniform registers anew, and the
            // issue, ~88 cycles a product against the tensor core's 64, set the pace
            // (a chunk of 4096 rows after 28672 slots: 1924 us).
            const uint32_t leader = elect_one();
            const uint64_t desc_k = tc::smem_desc(base_u32, 16, 1024), desc_v = tc::smem_desc(base_u32, kBox, 1024);
            const uint64_t desc_q = tc::smem_desc(q_u32, 16, 1024);
            // a step whose PV product is still to be issued: its V tile's stage, and flags
            constexpr uint32_t kLive = 16, kPhase = 32, kFirst = 64, kLast = 128, kFrees = 256;
            uint32_t before2 = 0, before1 = 0;  // steps g - 2 and g - 1
            uint32_t p_ph = 0, o_ph = 3;        // a bit a stream
            uint32_t g = 0, qpos = 0;
            uint32_t st = 0, st_ph = 0;         // ring stage of the K tile at hand
            bool ok = true;
            auto issue_pv = [&](uint32_t s, uint32_t q) -> bool {
                if (!wait(&sh->p_full[s], (p_ph >> s) & 1)) return false;
                p_ph ^= 1u << s;
                if (!wait(&sh->full[q & 15], q & kPhase ? 1 : 0)) return false;
                if (q & kFirst) {
                    if (!wait(&sh->o_empty[s], (o_ph >> s) & 1)) return false;
                    o_ph ^= 1u << s;
                }
                const uint32_t vs = q & 15;
                tc::fence_after();
                pv_products<D>(leader, tbase, s, desc_v + (uint64_t)(vs * (kTile >> 4)), q & kFirst ? 0u : 1u);
                if (q & kFrees) commit(leader, &sh->empty[vs]);
                if (q & kLast) commit(leader, &sh->o_full[s]);
                return true;
            };
#pragma unroll 1
            for (uint32_t k = 0; ok; ++k) {
                const int slot = k % kItems;
                if (!(ok = wait(&sh->item_full[slot], (k / kItems) & 1))) break;
                const int b = uniform(sh->items[slot].b), n = uniform(sh->items[slot].n);
                const bool two = uniform(sh->items[slot].ntok) > p.shape.tpt;
                if (b >= 0) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
                }
                // (the end of the list: two steps without an S, for the last products)
                const int steps = b < 0 ? 2 : two ? 2 * n : n;
#pragma unroll 1
                for (int i = 0; i < steps; ++i, ++g) {
                    if (two && i == 4 && b >= 0) {  // (n > 2)
                        // An item of two Q tiles from its third K/V tile on: both
                        // streams' steps of a tile, without the generic step's
                        // bookkeeping (its instructions, fetched anew each time beside
                        // the softmax warps' code, held the products up).
                        const uint32_t sa = g & 1, sb = sa ^ 1;
                        uint32_t vs = before1 & 15, v_ph = before1 & kPhase ? 1 : 0;  // V of the tile before
                        const uint64_t qa = desc_q + (uint64_t)((qpos & 1) * (kTile >> 4));
                        const uint64_t qb = desc_q + (uint64_t)(((qpos & 1) ^ 1) * (kTile >> 4));
#pragma unroll 1
                        for (int j = 2; j < n; ++j) {
                            const uint64_t dk = desc_k + (uint64_t)(st * (kTile >> 4));
                            const uint64_t dv = desc_v + (uint64_t)(vs * (kTile >> 4));
                            if (!(ok = wait(&sh->full[st], st_ph))) break;
                            if (!(ok = wait(&sh->full[vs], v_ph))) break;
                            if (!(ok = wait(&sh->p_full[sa], (p_ph >> sa) & 1))) break;
                            tc::fence_after();
                            pv_products<D>(leader, tbase, sa, dv, 1u);
                            s_products<D>(leader, tbase, sa, qa, dk);
                            commit(leader, &sh->s_full[sa]);
                            if (!(ok = wait(&sh->p_full[sb], (p_ph >> sb) & 1))) break;
                            tc::fence_after();
                            pv_products<D>(leader, tbase, sb, dv, 1u);
                            commit(leader, &sh->empty[vs]);
                            s_products<D>(leader, tbase, sb, qb, dk);
                            commit(leader, &sh->s_full[sb]);
                            commit(leader, &sh->empty[st]);
                            p_ph ^= 3u;
                            vs = st + 1 == kStages ? 0 : st + 1;
                            v_ph = st + 1 == kStages ? st_ph ^ 1 : st_ph;
                            st = vs + 1 == kStages ? 0 : vs + 1;
                            st_ph = vs + 1 == kStages ? v_ph ^ 1 : v_ph;
                        }
                        if (!ok) break;
                        commit(leader, &sh->q_empty[0]);
                        commit(leader, &sh->q_empty[1]);
                        before2 = vs | kLive | (v_ph ? kPhase : 0u) | kLast;
                        before1 = vs | kLive | (v_ph ? kPhase : 0u) | kLast | kFrees;
                        g += steps - 4;
                        break;
                    }
                    const uint32_t s = g & 1;
                    const bool second = two && (i & 1);  // of an item of two Q tiles: the second tile's step
                    const uint32_t qp = qpos + (second ? 1 : 0);
                    if (before2 && !(ok = issue_pv(s, before2))) break;
                    before2 = before1;
                    before1 = 0;
                    if (b < 0) continue;
                    if (i == 0 || (two && i == 1)) ok = wait(&sh->q_full[qp & 1], (qp >> 1) & 1);
                    if (ok && !second) ok = wait(&sh->full[st], st_ph);
                    if (!ok) break;
                    tc::fence_after();
                    const uint64_t dk = desc_k + (uint64_t)(st * (kTile >> 4));
                    const uint64_t dq = desc_q + (uint64_t)((qp & 1) * (kTile >> 4));
                    s_products<D>(leader, tbase, s, dq, dk);
                    commit(leader, &sh->s_full[s]);
                    const bool frees = !two || second;  // the tile's last reader
                    if (frees) commit(leader, &sh->empty[st]);
                    const bool last_tile = i >= steps - (two ? 2 : 1);
                    if (last_tile) commit(leader, &sh->q_empty[qp & 1]);
                    const uint32_t vs = st + 1 == kStages ? 0 : st + 1;
                    const uint32_t v_ph = st + 1 == kStages ? st_ph ^ 1 : st_ph;
                    before1 = vs | kLive | (v_ph ? kPhase : 0u) | (i < 2 ? kFirst : 0u) |
                              (i >= steps - 2 ? kLast : 0u) | (frees ? kFrees : 0u);
                    if (frees) {  // on to the next tile: K and V took a stage each
                        st = vs + 1 == kStages ? 0 : vs + 1;
                        st_ph = vs + 1 == kStages ? v_ph ^ 1 : v_ph;
                    }
                }
                if (b < 0) break;
                qpos += two ? 2 : 1;
            }
            if (!ok && lane == 0) fail();
            // every product issued is complete before the tensor memory is given back
            commit(leader, &sh->fin);
            wait(&sh->fin, 0);
        } else if (warp == 10) {
            // ===================== the work list: items of this CTA's units, and their Q tiles
            long long U, u0, u1, ub;  // ub: first unit of sequence b
            int nctas, b;
            Units un{0, 0, 0};        // lane: units of sequence cached + lane (pre, r0, r1: its lengths)
            int cached = -1;
            auto load = [&](int first) {
                cached = first;
                un = Units{0, 0, 0};
                if (first + lane < p.B) {
                    pre = p.prefix_lens[first + lane];
                    r0 = p.row_starts[first + lane];
                    r1 = p.row_starts[first + lane + 1];
                    un = units_of(p, pre, r0, r1);
                }
            };
            long long items = 0, x = 0, mine = 0;
            int most = 0, some = 0;   // some: items of this lane's sequences, of one KV head
            const int few = (p.B + 31) / 32;
            if (p.B > kWarpPlanB) {
                U = 0;
#pragma unroll 1
                for (int w = 0; w < kThreads / 32; ++w) {
                    U += sh->warp_units[w];
                    items += sh->warp_items[w];
                    most = max(most, sh->warp_most[w]);
                }
            } else {
                if (p.B <= 32) {
                    cached = 0;
                    un = units_of(p, pre, r0, r1);  // (no rows past the last sequence)
                    mine = un.per_head * p.Hkv;
                    some = un.items;
                    most = un.most;
                } else {  // a lane sums a few consecutive sequences (their lengths share cache lines)
#pragma unroll 1
                    for (int i = lane * few; i < min((lane + 1) * few, p.B); ++i) {
                        const Units v = units_of(p, p.prefix_lens[i], p.row_starts[i], p.row_starts[i + 1]);
                        mine += v.per_head * p.Hkv;
                        some += v.items;
                        most = max(most, v.most);
                    }
                }
                x = warp_scan(mine, lane);
                U = __shfl_sync(0xffffffffu, x, 31);
                items = (long long)__reduce_add_sync(0xffffffffu, some) * p.Hkv;
                most = __reduce_max_sync(0xffffffffu, most);
            }
            nctas = ctas_for(U, items, most, gridDim.x);
            // few items kept whole: units of each (0: its own)
            const int bound = units_bound(p.shape, most);
            const int each = p.B <= kWarpPlanB && p.shape.window < (1 << 20) &&
                                     whole_items(U, items, bound, nctas, gridDim.x)
                                 ? bound
                                 : 0;
            if (each > 0) {
                nctas = (int)items;
                U = items * each;
                mine = (long long)some * p.Hkv * each;
                x = warp_scan(mine, lane);
            }
            const bool has = U > 0 && (int)blockIdx.x < nctas;
            {
                const long long edge = cta_begin(U, nctas, blockIdx.x + (lane & 1));  // (both ends at once)
                u0 = __shfl_sync(0xffffffffu, edge, 0);
                u1 = __shfl_sync(0xffffffffu, edge, 1);
            }
            if (!has) {
                b = p.B;
                ub = 0;
            } else if (p.B > kWarpPlanB) {  // the last thread with at most u0 units before its sequences
                int below = 0;
#pragma unroll 1
                for (int i = lane; i < kThreads; i += 32) below += before[i] <= u0;
                const int at = __reduce_add_sync(0xffffffffu, below) - 1;
                b = at * per;
                ub = before[at];
                __syncwarp();
            } else {
                const int at = __ffs(__ballot_sync(0xffffffffu, u0 < x)) - 1;  // (x only grows)
                ub = __shfl_sync(0xffffffffu, x - mine, at);
                b = at * few;
            }
            uint32_t k = 0, qpos = 0;
            bool ok = true;
#pragma unroll 1
            while (ok && b < p.B && ub < u1) {
                if (cached < 0 || b >= cached + 32) load(b);
                const Seq sq = seq_of(p.shape, __shfl_sync(0xffffffffu, pre, b - cached),
                                      __shfl_sync(0xffffffffu, r0, b - cached), __shfl_sync(0xffffffffu, r1, b - cached));
                long long per_head = __shfl_sync(0xffffffffu, un.per_head, b - cached);
                if (each > 0) per_head = (long long)sq.items * each;
                if (ub + per_head * p.Hkv <= u0 || sq.items == 0) {
                    ub += per_head * p.Hkv;
                    ++b;
                    continue;
                }
                int h = 0, i = 0;
                long long ui = ub;  // first unit of item (h, i)
                if (u0 > ub) {      // the range starts inside this sequence
                    h = (int)quot(u0 - ub, per_head);
                    const long long v = (u0 - ub) - (long long)h * per_head;
                    ui = ub + (long long)h * per_head;
                    // the last item whose first unit is at most v: 32 candidates at a time
                    int span = sq.items;
                    long long at = 0;
#pragma unroll 1
                    while (span > 1) {
                        const int step = (span + 31) / 32;
                        const bool in = lane * step < span;
                        const long long u = !in ? 0 : each > 0 ? (long long)(i + lane * step) * each
                                                               : units_before(p.shape, sq, i + lane * step);
                        const int hit = 31 - __clz(__ballot_sync(0xffffffffu, in && u <= v));  // (lane 0 always)
                        at = __shfl_sync(0xffffffffu, u, hit);
                        i += hit * step;
                        span = min(step, span - hit * step);
                    }
                    ui += at;
                }
#pragma unroll 1
                for (; ok && h < p.Hkv && ui < u1; ++h, i = 0)
#pragma unroll 1
                    for (; ok && i < sq.items && ui < u1; ++i) {
                        const int n = item_tiles(p.shape, sq, i);
                        const int w = item_weight(p.shape, sq, i);
                        const Cut c = cut_item(ui, n, w, u0, u1);
                        const long long own = ui;
                        ui += each > 0 ? each : n * w + kItemCost;
                        if (c.a >= c.z) continue;  // only its cost falls into the range
                        Item it;
                        it.b = b;
                        it.h = h;
                        it.row0 = sq.row0 + i * 2 * p.shape.tpt;
                        it.ntok = min(2 * p.shape.tpt, sq.n - i * 2 * p.shape.tpt);
                        it.pos0 = sq.L + i * 2 * p.shape.tpt;
                        it.kt0 = first_tile(p.shape, it.pos0) + c.a;
                        it.n = c.z - c.a;
                        it.single = sq.items == 1;
                        it.c_first = blockIdx.x;
                        it.nc = 1;
                        it.counters = 0;
                        if (it.n < n) {  // the CTAs of its first and its last tile
                            const int cta = cta_of(U, nctas, tile_unit(own, w, lane & 1 ? n - 1 : 0));
                            it.c_first = __shfl_sync(0xffffffffu, cta, 0);
                            it.nc = __shfl_sync(0xffffffffu, cta, 1) - it.c_first + 1;
                            it.counters = counters_of(call, gridDim.x, it.c_first);  // (lane 0's, which publishes it)
                        }
                        it.ci = blockIdx.x - it.c_first;
                        const int slot = k % kItems;
                        if (!wait(&sh->item_empty[slot], ((k / kItems) & 1) ^ 1) ||
                            __shfl_sync(0xffffffffu, *abort_flag, 0)) {
                            ok = false;
                            break;
                        }
                        if (lane == 0) {
                            sh->items[slot] = it;
                            mbar_arrive(&sh->item_full[slot]);
                        }
                        ++k;
                        const int tiles = it.ntok > p.shape.tpt ? 2 : 1;
#pragma unroll 1
                        for (int q = 0; q < tiles; ++q, ++qpos) {
                            const int qb = qpos & 1;
                            if (!wait(&sh->q_empty[qb], ((qpos >> 1) & 1) ^ 1)) {
                                ok = false;
                                break;
                            }
                            if (lane == 0) {
                                // a single token needs one token's box, the rest of the tile may hold anything
                                const bool one = it.ntok - q * p.shape.tpt == 1;
                                const CUtensorMap *map = one ? &tmq1 : &tmq;
                                uint8_t *qd = qbuf + qb * kTile;
                                mbar_arrive_expect_tx(&sh->q_full[qb],
                                                      (uint32_t)(kHalves * 128 * p.G * (one ? 1 : p.shape.tpt)));
#pragma unroll 1
                                for (int hf = 0; hf < kHalves; ++hf)
                                    tma_load_3d(qd + hf * kBox, map, hf * 64, h * p.G, it.row0 + q * p.shape.tpt,
                                                &sh->q_full[qb]);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    }
                ub += per_head * p.Hkv;
                ++b;
            }
            if (!ok) fail();
            // the end of the list
            const int slot = k % kItems;
            if (wait(&sh->item_empty[slot], ((k / kItems) & 1) ^ 1) && lane == 0) {
                sh->items[slot].b = -1;
                mbar_arrive(&sh->item_full[slot]);
            }
            // seq_status: lengths, and the ids of the pages that rows see
#pragma unroll 1
            for (int sb = p.seq_status ? (int)blockIdx.x : p.B; sb < p.B; sb += gridDim.x) {
                const int L = p.prefix_lens[sb], first = p.row_starts[sb], end = p.row_starts[sb + 1];
                const Seq s = seq_of(p.shape, L, first, end);
                bool bad = !lengths_ok(p.shape, L, first, end);
                if (s.n > 0) {
                    const int lo = p.shape.window > 0 ? max(0, L - p.shape.window + 1) : 0;
                    const int32_t *trow = p.block_table + (size_t)sb * p.max_pages;
#pragma unroll 1
                    for (int j = lo / p.page_size + lane; j <= (L + s.n - 1) / p.page_size; j += 32) {
                        const int pg = trow[j];
                        if (pg < 0 || pg >= p.num_pages) bad = true;
                    }
                }
                bad = __any_sync(0xffffffffu, bad);
                if (lane == 0) p.seq_status[sb] = bad ? SV_ERR_BAD_INPUT : SV_OK;
            }
            if (lane == 0 && p.seq_status && (int)blockIdx.x < p.B && gave_up(p.call))
#pragma unroll 1
                for (int sb = blockIdx.x; sb < p.B; sb += gridDim.x) p.seq_status[sb] = SV_ERR_TIMEOUT;
            // the next call's counters
            call = __shfl_sync(0xffffffffu, call, 0);
            if (lane < kCtaCounters) p.counters[counters_of(call + 1, gridDim.x, blockIdx.x) + lane] = 0;
#pragma unroll 1
            for (uint32_t q = qpos > 2 ? qpos - 2 : 0; q < qpos; ++q)
                wait(&sh->q_full[q & 1], (q >> 1) & 1);
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 9) {
        tc::fence_after();
        tc::tmem_dealloc(tbase, kCols);
    }
    if (tid == 0 && *abort_flag) give_up(p.call, p.seq_status, p.B);
}

const void *kernel_fn(int D) {
    return D == 128 ? reinterpret_cast<const void *>(&chunk_attention_kernel<128>)
                    : reinterpret_cast<const void *>(&chunk_attention_kernel<64>);
}

static_assert((kStagesOf<128> + 2) * kTileBytes<128> + sizeof(Shared) <= 227 * 1024, "shared memory");

int smem_bytes(int D) { return (D == 128 ? (kStagesOf<128> + 2) * kTileBytes<128> : (kStagesOf<64> + 2) * kTileBytes<64>) + (int)sizeof(Shared); }

}  // namespace chunk
}  // namespace sv
