// sv_chunk_tc.cuh -- the chunk attention on the 5th-generation tensor cores, as
// a template of the cache's form: bf16 pages (sv_chunk_tc.cu, which says how it
// works) or pages held in 4 bits (sv_quant_tc.cu, which says what differs).
#pragma once

#include "sv_attn_common.cuh"
#include "sv_chunk.cuh"
#include "sv_quant.cuh"

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
static __device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity) {
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
template <int D, bool kF16>
__device__ __forceinline__ void pv_products(uint32_t leader, uint32_t tbase, uint32_t s, uint64_t dv,
                                            uint32_t accumulate) {
    constexpr uint32_t idesc = tc::idesc_bf16(kRows, D, true) & (kF16 ? ~(1u << 7 | 1u << 10) : ~0u);  // (0: f16)
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

// Two floats to f16 (nearest even), lo in the low half, and back.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
    float2 y;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}" : "=f"(y.x), "=f"(y.y) : "r"(x));
    return y;
}

// 16 columns of tensor memory a warp.
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
// Waits for the loads of r; what uses it stays behind.
__device__ __forceinline__ void ld_done(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// This warp's P in the first n columns from TMEM address s on (n a multiple of 16) times a.
__device__ __noinline__ inline void rescale_p(uint32_t s, int n, float a) {
    tc::wait_st();
#pragma unroll 1
    for (int i = 0; i < n; i += 16) {
        uint32_t pv[32];
        tc::tmem_ld32(s + i, pv);  // (of which half is used; a row has room behind it)
        tc::wait_ld();
        uint32_t y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float2 x = unpack_f16x2(pv[j]);
            y[j] = pack_f16x2(x.x * a, x.y * a);
        }
        tmem_st16(s + i, y);
    }
}

// Of the slots at .. at + 31 a bit for each from lo on and below hi.
__device__ __forceinline__ uint32_t visible(int at, int lo, int hi) {
    const int h = hi - at, o = lo - at;
    const uint32_t below = h >= 32 ? ~0u : h <= 0 ? 0u : (1u << h) - 1u;
    const uint32_t under = o >= 32 ? ~0u : o <= 0 ? 0u : (1u << o) - 1u;
    return below & ~under;
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

// ---------------------------------------------------------------- tiles held in 4 bits

// The slots' steps and middles, behind the tiles as they lie in the pages: [K's and V's places][slot pairs].
template <int D>
__device__ __forceinline__ uint8_t *raw_slots(uint8_t *raw) {
    return raw + kRawStages<D> * kRawTile<D>;
}

// Sum of a row of a Q tile.
template <int D>
__device__ __forceinline__ float row_sum(const uint8_t *tile, int r) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 x = *reinterpret_cast<const uint4 *>(tile + (c >> 3) * kBox + sw128(r, c & 7));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = __fadd2_rn(sum, make_float2(bf16_lo(w[i]), bf16_hi(w[i])));
    }
    return sum.x + sum.y;
}

// The tiles as they lie in the pages: K's (kv = 0: the even ring positions) or V's
// by a warp, its lane a page of the tile; each one copy of codes and one of
// parameters.
template <int D, class P, class S>
__device__ __forceinline__ void load_quant(const P &p, S *sh, uint8_t *raw, int kv, int lane) {
    constexpr int kRow = D / 2, kStages = kRawStages<D>, kTile = kRawTile<D>;
    volatile int *abort_flag = &sh->abort_flag;
    auto fail = [&] { *abort_flag = 1; };
    const uint8_t *codes = kv ? p.v_codes : p.k_codes;
    const uint32_t *params = kv ? p.v_params : p.k_params;
    const int ps = p.page_size;
    const int sub = ps < kBK ? ps : kBK;      // slots of a copy
    const int npg = kBK / sub;                // copies a tile
    const int tpp = ps < kBK ? 1 : ps / kBK;  // tiles a page (of 128 slots or more)
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
        // cache row of the first slot of this lane's copy of tile j; -1: no slot of it is seen.  In the place of
        // a page id out of range (reported by the check, its rows unspecified) page 0 is read.
        auto first_row = [&](int j) -> int {
            const int tile = it.kt0 + j, s0 = tile * kBK + lane * sub;
            if (lane >= npg || s0 >= hi || s0 + sub <= lo) return -1;
            const int page = tpp == 1 ? tile * npg + lane : tile / tpp;
            int pg = trow[page];
            if (pg < 0 || pg >= p.num_pages) pg = 0;
            return (pg * p.Hkv + it.h) * ps + (tpp == 1 ? 0 : (tile - page * tpp) * kBK);
        };
        int y = first_row(0);
#pragma unroll 1
        for (int j = 0; j < it.n; ++j) {
            const int y_next = j + 1 < it.n ? first_row(j + 1) : -1;
            const int copies = __popc(__ballot_sync(0xffffffffu, y >= 0));
            const int st = pos % kStages;
            if (!wait(&sh->raw_empty[st], ((pos / kStages) & 1) ^ 1)) {
                fail();
                ok = false;
                break;
            }
            if (__shfl_sync(0xffffffffu, *abort_flag, 0)) {
                ok = false;
                break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&sh->raw_full[st], (uint32_t)(copies * sub * (kRow + 4)));
            __syncwarp();  // the expected bytes are set before any copy lands
            if (y >= 0) {
                uint8_t *to = raw + st * kTile;
                bulk_load(to + lane * sub * kRow, codes + (size_t)y * kRow, (uint32_t)(sub * kRow), &sh->raw_full[st]);
                bulk_load(to + kBK * kRow + lane * sub * 4, params + y, (uint32_t)(sub * 4), &sh->raw_full[st]);
            }
            pos += 2;
            y = y_next;
        }
    }
    // every copy issued must land before the CTA may exit
    if (__shfl_sync(0xffffffffu, *abort_flag, 0))
#pragma unroll 1
        for (uint32_t q = pos > kStages ? pos - kStages : kv; q < pos; ++q)
            if ((q & 1) == (uint32_t)kv) wait(&sh->raw_full[q % kStages], (q / kStages) & 1);
}

// The tiles as the products read them: a thread a slot.  K's codes less 8 are exact in
// bf16; their step and middle (minimum + 8 steps), times the scale, lie beside the tile
// in f32.  V's values go to f16 times 2^-e, where a warp's 32 slots share e: their
// largest is below 2^15, and above 2^-28 of it steps are exact, middles and values rounded
// by at most 2^-11 of themselves each.  A slot
// that no row of the item sees has zeros, and so has one whose row of V is not finite: a
// weight of 0 would bring it to every row of the tile.  Its NaN goes into the score instead,
// which is masked where the slot is hidden.
template <int D, class P, class S>
__device__ __forceinline__ void expand_quant(const P &p, S *sh, uint8_t *smem, uint8_t *raw, int w, int lane) {
    constexpr int kRow = D / 2, kPieces = D / 32, kStages = kStagesOf<D, true>, kRaw = kRawStages<D>;
    volatile int *abort_flag = &sh->abort_flag;
    auto fail = [&] { *abort_flag = 1; };
    const int r = 32 * w + lane;  // the slot in its tile
    const uint8_t *const raw_at = raw + r * kRow, *const par_at = raw + kBK * kRow + r * 4;
    float *slots = reinterpret_cast<float *>(raw_slots<D>(raw));
    uint32_t pos = 0;
    bool ok = true;
#pragma unroll 1
    for (uint32_t k = 0; ok; ++k) {
        const int slot = k % kItems;
        if (!wait(&sh->item_full[slot], (k / kItems) & 1)) {
            fail();
            break;
        }
        const Item &item = sh->items[slot];
        const int b = item.b, n = item.n, pos0 = item.pos0, ntok = item.ntok, kt0 = item.kt0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->item_empty[slot]);
        if (b < 0) break;
        const int lo = p.shape.window > 0 ? max(0, pos0 - p.shape.window + 1) : 0, hi = pos0 + ntok;
#pragma unroll 1
        for (int j = 0; j < 2 * n; ++j, ++pos) {  // K, then V of each tile
            const uint32_t rs = pos % kRaw, st = pos % kStages;
            if (!(ok = wait(&sh->raw_full[rs], (pos / kRaw) & 1))) break;
            const int at = (kt0 + (j >> 1)) * kBK + r;
            const bool seen = at >= lo && at < hi;
            // (rows two and two read their pieces in turn from another one on, so that eight lanes of
            // an access, to the codes or to the tile, meet eight bank groups)
            uint4 c[kPieces];
            uint32_t par = 0;
#pragma unroll
            for (int i = 0; i < kPieces; ++i) c[i] = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
            if (seen) {
                par = *reinterpret_cast<const uint32_t *>(par_at + rs * kRawTile<D>);
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int piece = (i + (r >> (D == 128 ? 1 : 2))) & (kPieces - 1);
                    c[i] = *reinterpret_cast<const uint4 *>(raw_at + rs * kRawTile<D> + piece * 16);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->raw_empty[rs]);
            if (!(ok = wait(&sh->empty[st], ((pos / kStages) & 1) ^ 1))) break;
            if (__shfl_sync(0xffffffffu, *abort_flag, 0)) {
                ok = false;
                break;
            }
            const uint32_t tile = pos >> 1;
            float step = bf16_lo(par), mid = __fmaf_rn(8.f, step, bf16_hi(par));
            uint8_t *const to = smem + r * 128 + st * kTileBytes<D>;
            auto store = [&](auto &&values) {
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int piece = (i + (r >> (D == 128 ? 1 : 2))) & (kPieces - 1);
                    const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
                    uint8_t *const at = to + (piece >> 1) * kBox;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint4 v = values(words[q]);
                        const uint32_t chunk = (uint32_t)((piece & 1) * 4 + q) ^ (uint32_t)(r & 7);
                        *reinterpret_cast<uint4 *>(at + chunk * 16) = v;
                    }
                }
            };
            if (pos & 1) {
                uint32_t mine = __float_as_uint(__fmaf_rn(8.f, fabsf(step), fabsf(mid))) >> 23;
                if (mine == 255u) {  // (the softmax reads K's middle once V's tile is there too)
                    slots[tile % kKSlots<D> * (kSlotBytes / 4) + (r >> 1) * 4 + (r & 1) + 2] = __uint_as_float(0x7fc00000u);
                    step = mid = 0.f;
                    mine = 0;
                }
                const uint32_t most = max(__reduce_max_sync(0xffffffffu, mine), (uint32_t)(126 + 15 + kLeastV));
                const float down = __uint_as_float((127u + 15u + 126u - most) << 23);
                const uint32_t step2 = pack_f16x2(step * down, step * down), mid2 = pack_f16x2(mid * down, mid * down);
                if (lane == 0) {  // e and 2^-e
                    const int e = (int)most - 126 - 15;
                    reinterpret_cast<float2 *>(slots + kKSlots<D> * (kSlotBytes / 4))[tile % kVSlots<D> * 4 + w] =
                        make_float2((float)e, __uint_as_float((uint32_t)(127 - e) << 23));
                }
                store([&](uint32_t x) { return quant::scaled_f16(x, step2, mid2); });  // (not seen: 0 of both)
            } else {
                float *to = slots + tile % kKSlots<D> * (kSlotBytes / 4) + (r >> 1) * 4 + (r & 1);
                to[0] = step * p.scale_log2;  // (of two slots the steps, then the middles)
                to[2] = mid * p.scale_log2;
                store([&](uint32_t x) { return quant::expand(x); });
            }
            tc::fence_proxy_async_smem();  // (the tensor core reads them next)
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->full[st]);
        }
    }
    if (!ok) fail();
}

// ---------------------------------------------------------------- the kernel

template <int D, bool kQuant>
__global__ void __launch_bounds__(kThreadsOf<kQuant>, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap tmk,
                           const __grid_constant__ CUtensorMap tmv,
                           const __grid_constant__ CUtensorMap tmq,
                           const __grid_constant__ CUtensorMap tmq1, const ParamsOf<kQuant> p) {
    constexpr int kStages = kStagesOf<D, kQuant>;
    constexpr int kThreads = kThreadsOf<kQuant>;
    constexpr int kTile = kTileBytes<D>;
    constexpr int kHalves = D / 64;
    constexpr int kKS = kKSlots<D>, kVS = kVSlots<D>;
    extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle's atoms are 1024 bytes)
    const uint32_t base_u32 = smem_u32(smem);
    uint8_t *qbuf = smem + kStages * kTile;
    const uint32_t q_u32 = base_u32 + kStages * kTile;
    uint8_t *raw = qbuf + 2 * kTile;  // the tiles as they lie in the pages, where those are in 4 bits
    SharedOf<kQuant> *sh = reinterpret_cast<SharedOf<kQuant> *>(raw + kRawBytes<D, kQuant>);

    // (the warp's number as the compiler knows to be the same in all its lanes)
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->full[i], kQuant ? kExpandWarps : 1);
            mbar_init(&sh->empty[i], 1);
        }
        if constexpr (kQuant) {
#pragma unroll 1
            for (int i = 0; i < kRawStages<D>; ++i) {
                mbar_init(&sh->raw_full[i], 1);
                mbar_init(&sh->raw_empty[i], kExpandWarps);
            }
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], kQuant ? 1 + 8 : 1);  // (in 4 bits the softmax warps read Q too)
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->o_full[i], 1);
            mbar_init(&sh->o_empty[i], 4);
            mbar_init(&sh->x_full[i], 4);
        }
#pragma unroll 1
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh->item_full[i], 1);
            mbar_init(&sh->item_empty[i], kQuant ? 11 + kExpandWarps : 11);  // softmax warps, loaders, issuer
        }
        mbar_init(&sh->fin, 1);
        sh->abort_flag = 0;
        fence_mbar_init();
    }
    if (tid == 32 * 8) {
        if constexpr (!kQuant) {
            prefetch_tensormap(&tmk);
            prefetch_tensormap(&tmv);
        }
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
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegsOf<kQuant>));
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
        uint32_t qpos = 0;        // Q tiles before this item
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
            int w_hi = pos0 + t_lo + 1;
            const int w_lo = p.shape.window > 0 ? pos0 + min(t_hi, ntok - 1) - p.shape.window + 1 : 0;
            const int item_lo = p.shape.window > 0 ? max(0, it.pos0 - p.shape.window + 1) : 0;
            const int item_hi = it.pos0 + it.ntok;
            // a tree: which of the sequence's own rows this one sees, and the slot of the first of them
            unsigned long long above = 0;
            int own0 = 0;
            bool tree = false;
            if constexpr (kQuant) {
                if (p.parents) {
                    tree = true;
                    const int node0 = it.row0 - it.seq_row0, node = node0 + qt * p.shape.tpt + t;
                    const int nodes = min(node0 + it.ntok, kTreeNodes);  // (parents come before their children)
                    const int32_t *par = p.parents + it.seq_row0;
                    const int lo = lane < nodes ? par[lane] : -1, hi = lane + 32 < nodes ? par[lane + 32] : -1;
                    above = ancestors_warp(false, lo, hi, node, node < nodes);
                    own0 = w_hi = it.pos0 - node0;
                }
            }
            float m = kNegInf, l = 0.f;
            float qs = 0.f;  // in 4 bits: the sum of the row of Q
            if constexpr (kQuant) {
                const uint32_t qp = qpos + qt;
                ok = warp_wait_bounded(&sh->q_full[qp & 1], (qp >> 1) & 1);
                if (!ok) {
                    fail();
                    break;
                }
                if (active) qs = row_sum<D>(qbuf + (qp & 1) * kTile, r);
                __syncwarp();
                // (eight arrivals a tile, of the warps that waited for it alone: where two tiles are on the streams each
                // warp's is two.  One for a tile that the warp has not waited for could complete the phase before)
                if (lane == 0) {
                    mbar_arrive(&sh->q_empty[qp & 1]);
                    if (two) mbar_arrive(&sh->q_empty[qp & 1]);
                }
                qpos += two ? 2 : 1;
            }
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
                if (kQuant && active) {
                    // a warp of V's slots at a time (all of a row's scores beside what the codes need do not
                    // fit a thread's registers), the next ones' S on its way
                    const uint32_t pv = ring + 2 * j + 1;
                    ok = warp_wait_bounded(&sh->full[pv % kStages], (pv / kStages) & 1);  // (V's exponents, and its NaN)
                    if (!ok) break;
                    const uint8_t *slots = raw_slots<D>(raw);
                    const float4 *ks = reinterpret_cast<const float4 *>(slots + (pv >> 1) % kKS * kSlotBytes);
                    const float2 *es = reinterpret_cast<const float2 *>(slots + kKS * kSlotBytes) + (pv >> 1) % kVS * 4;
                    const float2 qs2 = make_float2(qs, qs);
                    const bool masked = kb + kBK > w_hi || kb < w_lo;
                    uint32_t ra[32];
                    float2 sv[16];
                    tc::tmem_ld32(sbuf, ra);
                    // (two of the four in line: with all of them and the next part's scores beside a part's weights a
                    // prompt's 539 us become 534, but the chains' 87 become 110)
#pragma unroll 2
                    for (int h = 0; h < 4; ++h) {
                        // step * (q . (codes - 8)) + middle * sum(q), scaled
                        ld_done(ra);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float4 k4 = ks[16 * h + i];
                            sv[i] = __ffma2_rn(make_float2(__uint_as_float(ra[2 * i]), __uint_as_float(ra[2 * i + 1])),
                                               make_float2(k4.x, k4.y), __fmul2_rn(make_float2(k4.z, k4.w), qs2));
                        }
                        if (h < 3) tc::tmem_ld32(sbuf + 32 * (h + 1), ra);
                        if (masked) {
                            const int at = kb + 32 * h;
                            uint32_t sees = visible(at, see_lo, see_hi);
                            if (tree) {  // all of the slots before own0, and of those from it on the path's
                                const int x = at - own0;
                                sees = x <= -32 ? ~0u
                                     : x < 0    ? ((1u << -x) - 1u) | (uint32_t)(above << -x)
                                     : x < 64   ? (uint32_t)(above >> x)
                                                : 0u;
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                if (!((sees >> (2 * i)) & 1u)) sv[i].x = kNegInf;
                                if (!((sees >> (2 * i + 1)) & 1u)) sv[i].y = kNegInf;
                            }
                        }
                        // the exponent of these slots' V joins the score
                        const float2 e2 = es[h];
                        float mq[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                        for (int i = 0; i < 16; ++i) mq[i & 3] = fmaxf(fmaxf(mq[i & 3], sv[i].x), sv[i].y);
                        // (m: kTop below the maximum that it was set to)
                        const float c = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) + (e2.x - kTop);
                        const bool up = c > m + kRescaleThreshold;
                        if (__any_sync(0xffffffffu, up)) {
                            const float f = up ? ex2_approx(m - c) : 1.f;
                            if (up) {
                                m = c;
                                l *= f;
                            }
                            if (h < 3) ld_done(ra);
                            // (the wait for S covers this stream's earlier PV products: issued before it)
                            if (j != first) rescale_o<D>(o_cols, f);
                            if (h > 0) rescale_p(sbuf, 16 * h, f);
                        }
                        const float nb = (m == kNegInf ? 0.f : -m) + e2.x;
                        const float2 nb2 = make_float2(nb, nb);
                        float2 ls = make_float2(0.f, 0.f);
                        uint32_t pk[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 x = __fadd2_rn(sv[i], nb2);
                            const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                            ls = __fadd2_rn(ls, e);
                            pk[i] = pack_f16x2(e.x, e.y);
                        }
                        l = __fmaf_rn(ls.x + ls.y, e2.y, l);
                        tmem_st16(sbuf + 16 * h, pk);
                    }
                    tc::wait_st();
                } else if (active) {
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
                if (!kQuant && (kb + kBK > item_hi || kb < item_lo)) {  // (in 4 bits: zeroed as they are expanded)
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegsOf<kQuant>));
        if (kQuant && warp != 9 && warp != 10) {
            if constexpr (kQuant) {
                if (warp >= 12) expand_quant<D>(p, sh, smem, raw, warp - 12, lane);
                else load_quant<D>(p, sh, raw, warp == 11, lane);
            }
        } else if (warp == 8 || warp == 11) {
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
                pv_products<D, kQuant>(leader, tbase, s, desc_v + (uint64_t)(vs * (kTile >> 4)), q & kFirst ? 0u : 1u);
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
                            pv_products<D, kQuant>(leader, tbase, sa, dv, 1u);
                            s_products<D>(leader, tbase, sa, qa, dk);
                            commit(leader, &sh->s_full[sa]);
                            if (!(ok = wait(&sh->p_full[sb], (p_ph >> sb) & 1))) break;
                            tc::fence_after();
                            pv_products<D, kQuant>(leader, tbase, sb, dv, 1u);
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
                        it.seq_row0 = sq.row0;
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
                    if constexpr (kQuant) {
                        if (p.parents) {
                            bad = bad || s.n > kTreeNodes;
#pragma unroll 1
                            for (int i = lane; i < min(s.n, kTreeNodes); i += 32) {
                                const int par = p.parents[first + i];
                                if (i == 0 ? par != -1 : par < 0 || par >= i) bad = true;
                            }
                        }
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

}  // namespace chunk
}  // namespace sv
