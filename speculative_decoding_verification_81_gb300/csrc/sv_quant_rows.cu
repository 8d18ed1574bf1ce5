// sv_quant_rows.cu -- attention over pages held in 4 bits, form for few rows a
// sequence: single tokens and short chains.
//
// An item is the rows of some tokens of one sequence and the heads of them that
// share K/V: up to 8 NT columns, NT = 1 or 2.  Each of the CTA's eight warps takes 16
// slots of every 128-slot tile and goes on by itself to the item's end:
//     S = codes Q^T             (16 slots x 8 NT columns; codes less 8, exact in bf16)
//     s = step_k S + middle_k sum(q), scaled to log2 units
//     P = 2^(s - u) step_v, rounded to f16; l += 2^(s - u); z += 2^(s - u) middle_v
//     O^T += codes^T P          (D dims x 8 NT columns; codes less 8, exact in f16)
// and out = (O + z) / l, where the warps, then the CTAs that share an item, are
// brought to one u.  A column's u moves only when some P would pass 2^15, to where the
// largest is 2^7: f16 then rounds P by at most 2^-11 of itself down to 2^-21 of the
// largest, and the steps and middles never meet a matrix product, so that nothing
// of the cache is rounded.
//
// Why the warp's own products of 16 x 8 (mma.sync; 1024 multiply-adds a clock and SM
// measured, a quarter of tcgen05's): the codes become operands in the registers that
// they are loaded to, eleven instructions for eight of them, where tensor memory's
// products want them written to shared memory as 16-bit tiles first, four times the
// pages' bytes, and read from there for a column count that is mostly padding; and a
// slot's step and middle are a lane's own, where a thread a row needs each of them
// from shared memory.
//
// Every lane copies its 16 bytes of a unit four units ahead (cp.async): with a bulk
// copy for each of a page's four parts 32 single tokens took 51 us instead of 44.
//
// What bounds it (32 query over 8 KV heads of 128): the instructions, some 320 a unit
// of which the integer pipe has half (52% busy, 2.1 of 4 issue slots taken), and the
// barriers where an item's warps meet -- 32 single tokens after 2048-4096 slots 43 us,
// 0.36 of the measured bandwidth, 64 after 4096 94 us, 0.45.  One token after 2047
// slots is 11.6 us: in cycles, the list 2800, the page table 1800, the pages and two
// tiles 3800, the warps' meeting 1600, the joining of 72 CTAs' shares 2300, and the
// launch, one after another.  S in sums of their own, so that no product
// waits for another: no gain.
#include <mutex>

#include "sv_attn_common.cuh"
#include "sv_chunk.cuh"
#include "sv_quant.cuh"
#include "sv_quant_walk.cuh"

namespace sv {
namespace chunk {

namespace {

constexpr int kRW = 8, kRT = 32 * kRW;  // warps, threads
constexpr int kU = 16;                  // slots of a unit

// K codes, V codes, K's and V's parameters of a unit.
template <int D>
constexpr int kUnitRaw = kU * (D + 8);
constexpr int kCtasAnSm = 2;
template <int D>
constexpr int kRowsDepth = D == 128 ? 4 : 8;  // units of a warp on their way
template <int D>
constexpr int kMeetBytes = kRW * 8 * D * 4;

template <int D, int NT>
struct RowsShared {
    uint8_t ring[kRW][kRowsDepth<D>][kUnitRaw<D>];
    float4 meet[kMeetBytes<D> / 16];
    uint8_t q[2][8 * NT * D * 2];
    float qs[8 * NT];
    float u[kRW][8 * NT];
    float2 ml[kRW][8 * NT];
    unsigned long long above[2][kTreeNodes];
    RowsWalk walk;       // warp 0's
    RowsItem items[2];   // the item at hand and the next
    long long warp_units[kRW];
    long long before[kRT];
    uint8_t tok[2][8 * NT];
    int last;
};

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 x;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a) : "memory");
    return x;
}
__device__ __forceinline__ uint32_t lds4(uint32_t a) {
    uint32_t x;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(a) : "memory");
    return x;
}

// 16 bytes to shared memory without a register, zeros where `on` is false.
__device__ __forceinline__ void copy16(uint32_t to, const void *from, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>  // of a thread's groups of copies, the last kLeft may still be on their way
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// D (16 x 8, f32) += A (16 x 16) B (16 x 8): with g = lane / 4 and t = lane % 4, a0..a3 hold A at
// rows g, g + 8, g, g + 8 and columns 2t, 2t + 1 (the last two 8 further), b0, b1 B at rows 2t,
// 2t + 1 and 8 further, column g, d[0..3] D at (g, 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1).
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16 bits, lane (g, t) with row g, columns 2t and 2t + 1.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// Two floats to f16 (nearest even), lo in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Place of 16-byte piece `piece` of column c's row of Q, of D / 8: lane t reads pieces
// (D / 32) t .. of it, and eight lanes (two columns, t = 0 .. 3) then meet eight bank groups.
template <int D>
__device__ __forceinline__ uint32_t q_piece(int c, int piece) {
    const int x = D == 128 ? (piece >> 3 & 1) ^ (c & 1) << 1 : c & 1;
    return (uint32_t)(c * (D * 2) + ((piece ^ x) << 4));
}

// Row r of a unit's S is slot r ^ (r >> 1 & 1): the slots of rows 2t and 2t + 1, whose V codes lane
// t reads, then start in the other 64 bytes for every other t.
__device__ __forceinline__ int slot_of(int r) { return r ^ (r >> 1 & 1); }

}  // namespace

template <int D, int NT>
__global__ void __launch_bounds__(kRT, kCtasAnSm) quant_rows_kernel(const RowsParams p) {
    constexpr int kDepth = kRowsDepth<D>;
    constexpr int kRow = D / 2;   // bytes of a row's codes
    constexpr int kW = D / 32;    // words of a K row a lane: words kW t + j
    constexpr int kX = D / 16;    // blocks of 16 dims of O^T
    extern __shared__ __align__(16) uint8_t dynamic[];
    using Sh = RowsShared<D, NT>;
    Sh &sh = *reinterpret_cast<Sh *>(dynamic);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, g = lane >> 2, t = lane & 3;
    griddep_wait();
    griddep_launch_dependents();
    unsigned long long call = 0;
    if (tid == 0) call = begin_call(p.call);

    auto look_ahead = [&](int to) {  // the next item (by one warp)
        if (lane == 0) next_item(p, sh.walk, sh.items[to]);
        __syncwarp();
    };
    plan_walk<kRT>(p, sh.warp_units, sh.before, tid, sh.walk);
    if (tid == 0) sh.items[1].b = 0;

    const uint32_t ring_at = smem_u32(sh.ring[warp][0]);
    uint32_t got = 0;  // units used

    // of the item at hand, or of the one whose copies are begun: this warp's tiles i0 .. i1 - 1, the
    // next to ask for, and, a lane a tile from `base` on, the cache rows of the unit's halves
    int i0 = 0, i1 = 0, ask = 0, base = 0, y0 = -1, y1 = -1;
    auto load_rows = [&](const RowsItem &x) {
        const int slot = (x.kt0 + base + lane) * kTileSlots + warp * kU;
        const int lo = p.rows.window > 0 ? max(0, x.pos0 - p.rows.window + 1) : 0, hi = x.pos0 + x.ntok;
        const int32_t *trow = p.block_table + (size_t)x.b * p.max_pages;
        auto row = [&](int s) -> int {  // (a page id out of range is reported; page 0 is read in its place)
            int pg = trow[s / p.page_size];
            if (pg < 0 || pg >= p.num_pages) pg = 0;
            return (pg * p.Hkv + x.h) * p.page_size + s % p.page_size;
        };
        y0 = y1 = -1;
        if (base + lane < i1) {
            if (p.page_size > 8) {
                y0 = row(slot);
                y1 = y0 + 8;
            } else {
                if (slot + 8 > lo && slot < hi) y0 = row(slot);
                if (slot + 16 > lo && slot + 8 < hi) y1 = row(slot + 8);
            }
        }
    };
    auto fetch = [&](const RowsItem &x, uint32_t unit) {  // the unit of tile `ask`: one group of copies, empty past the end
        if (ask < i1) {
            if (ask - base == 32) {
                base = ask;
                load_rows(x);
            }
            const int a0 = __shfl_sync(0xffffffffu, y0, ask - base), a1 = __shfl_sync(0xffffffffu, y1, ask - base);
            const uint32_t to = ring_at + unit % kDepth * kUnitRaw<D> + lane * 16;
            if constexpr (D == 128) {
                copy16(to, p.k_codes + (size_t)max(a0, 0) * kRow + lane * 16, a0 >= 0);
                copy16(to + 512, p.k_codes + (size_t)max(a1, 0) * kRow + lane * 16, a1 >= 0);
                copy16(to + 1024, p.v_codes + (size_t)max(a0, 0) * kRow + lane * 16, a0 >= 0);
                copy16(to + 1536, p.v_codes + (size_t)max(a1, 0) * kRow + lane * 16, a1 >= 0);
            } else {
                const int a = lane < 16 ? a0 : a1;
                copy16(to, p.k_codes + (size_t)max(a, 0) * kRow + (lane & 15) * 16, a >= 0);
                copy16(to + 512, p.v_codes + (size_t)max(a, 0) * kRow + (lane & 15) * 16, a >= 0);
            }
            if (lane < 8) {
                const int a = lane & 2 ? a1 : a0;
                copy16(to + 2 * kU * kRow, (lane < 4 ? p.k_params : p.v_params) + max(a, 0) + (lane & 1) * 4, a >= 0);
            }
            ++ask;
        }
        copies_end();
    };
    auto begin = [&](const RowsItem &x, int buf) {  // its first copies, and its queries
        const int lo = p.rows.window > 0 ? max(0, x.pos0 - p.rows.window + 1) : 0, hi = x.pos0 + x.ntok;
        const int s0 = x.kt0 * kTileSlots + warp * kU;  // (the slots seen end, or begin, within a tile)
        i0 = s0 + kU <= lo ? 1 : 0;
        i1 = s0 < hi ? min(x.n, (hi - s0 - 1) / kTileSlots + 1) : 0;
        ask = base = i0;
        load_rows(x);
        const int cols = x.ntok * p.G, head0 = x.h * p.G;
        const uint32_t q_at = smem_u32(sh.q[buf]);
        for (int i = tid; i < 8 * NT * (D / 8); i += kRT) {
            const int c = i / (D / 8), piece = i % (D / 8), tk = c / p.G, hd = c - tk * p.G;
            const bool on = c < cols;
            const uint16_t *from = p.q + (size_t)(x.row0 + (on ? tk : 0)) * p.q_stride + (size_t)(head0 + (on ? hd : 0)) * D + piece * 8;
            copy16(q_at + q_piece<D>(c, piece), from, on);
            if (piece == 0) sh.tok[buf][c] = (uint8_t)min(tk, x.ntok - 1);
        }
        copies_end();
#pragma unroll 1
        for (int i = 0; i < kDepth; ++i) fetch(x, got + i);
        if (p.parents && warp < 2) {  // a token's set of nodes above it, of those up to the item's last
            const int node0 = x.row0 - x.seq_row0, nodes = min(node0 + x.ntok, kTreeNodes);
            const int32_t *par = p.parents + x.seq_row0;
            const int a = lane < nodes ? par[lane] : -1, b = lane + 32 < nodes ? par[lane + 32] : -1;
            const int tk = tid, node = node0 + tk;
            const unsigned long long set = ancestors_warp(false, a, b, node, tk < x.ntok && node < nodes);
            sh.above[buf][tk] = set;
        }
    };
    // (item k is items[k & 1]; the first look ahead is of item 0, the loop's of the one after)
    if (warp == 0) look_ahead(0);
    __syncthreads();
    if (sh.items[0].b >= 0) begin(sh.items[0], 0);

    // ---- seq_status, while the first copies are on their way
    const int own = p.seq_status ? (int)blockIdx.x * kRW + warp : p.B;
#pragma unroll 1
    for (int sb = own; sb < p.B; sb += (int)gridDim.x * kRW) {
        const bool bad = bad_sequence(p, sb, lane);
        if (lane == 0) p.seq_status[sb] = bad ? SV_ERR_BAD_INPUT : SV_OK;
    }

#pragma unroll 1
    for (int qb = 0;; qb ^= 1) {
        const RowsItem it = sh.items[qb];
        if (it.b < 0) break;
        const int cols = it.ntok * p.G, nt = (cols + 7) / 8;
        const int lo = p.rows.window > 0 ? max(0, it.pos0 - p.rows.window + 1) : 0, hi = it.pos0 + it.ntok;
        const int own0 = it.pos0 - (it.row0 - it.seq_row0);  // slot of the sequence's first new row
        // below: every row sees the slots; from all_lo on too
        const int all_hi = p.parents ? own0 : it.pos0 + 1;
        const int all_lo = p.rows.window > 0 ? it.pos0 + it.ntok - p.rows.window : 0;
        copies_wait<kDepth>();
        for (int i = lane; i < 8 * NT; i += 32) sh.u[warp][i] = kUnset;
        __syncthreads();
        const uint32_t q_at = smem_u32(sh.q[qb]), u_at = smem_u32(sh.u[warp]), qs_at = smem_u32(sh.qs);
        float o[kX][NT][4], l[NT][2], z[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            l[n][0] = l[n][1] = z[n][0] = z[n][1] = 0.f;
#pragma unroll
            for (int x = 0; x < kX; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][n][e] = 0.f;
        }
        // the columns' sums of Q, by products with ones; each warp a block of columns
        if (warp < NT) {
            float s[4] = {0.f, 0.f, 0.f, 0.f};
            const uint32_t one = 0x3f803f80u;
#pragma unroll
            for (int j = 0; j < kW; ++j) {
                const uint4 b = lds16(q_at + q_piece<D>(8 * warp + g, kW * t + j));
                mma_bf16(s, one, one, one, one, b.x, b.y);
                mma_bf16(s, one, one, one, one, b.z, b.w);
            }
            if (g == 0) {
                sh.qs[8 * warp + 2 * t] = s[0];
                sh.qs[8 * warp + 2 * t + 1] = s[1];
            }
        }
        __syncthreads();
        if (warp == 0) look_ahead(qb ^ 1);
#pragma unroll 1
        for (int i = i0; i < i1; ++i) {
            const uint32_t st = got % kDepth;
            copies_wait<kDepth - 1>();
            __syncwarp();
            const uint32_t at = ring_at + st * kUnitRaw<D>;
            const int slot0 = (it.kt0 + i) * kTileSlots + warp * kU;
            // ---- S
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            {
                uint32_t k0[kW], k1[kW];
                const uint32_t ka = at + slot_of(g) * kRow + t * (4 * kW);
                if constexpr (kW == 4) {
                    const uint4 a = lds16(ka), b = lds16(ka + 8 * kRow);
                    k0[0] = a.x, k0[1] = a.y, k0[2] = a.z, k0[3] = a.w;
                    k1[0] = b.x, k1[1] = b.y, k1[2] = b.z, k1[3] = b.w;
                } else {
                    const uint2 a = lds8(ka), b = lds8(ka + 8 * kRow);
                    k0[0] = a.x, k0[1] = a.y;
                    k1[0] = b.x, k1[1] = b.y;
                }
#pragma unroll
                for (int j = 0; j < kW; ++j) {
                    const uint4 a = quant::expand(k0[j]), b = quant::expand(k1[j]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint4 q = lds16(q_at + q_piece<D>(8 * n + g, kW * t + j));
                        mma_bf16(s[n], a.x, b.x, a.y, b.y, q.x, q.y);
                        mma_bf16(s[n], a.z, b.z, a.w, b.w, q.z, q.w);
                    }
                }
            }
            // ---- steps and middles of the lane's two slots (rows g and g + 8 of S)
            const int slot = slot0 + slot_of(g);
            float ks[2], km[2], vs[2], vm[2], bound[2];
            const bool inside = slot0 >= lo && slot0 + kU <= hi;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t pa = at + 2 * kU * kRow + (slot_of(g) + 8 * r) * 4;
                const uint32_t kp = lds4(pa);
                uint32_t vp = lds4(pa + kU * 4);
                if (!inside && (slot + 8 * r < lo || slot + 8 * r >= hi)) vp = 0;  // (it may hold anything; K's is hidden)
                ks[r] = bf16_lo(kp) * p.scale_log2;
                km[r] = __fmaf_rn(8.f, bf16_lo(kp), bf16_hi(kp)) * p.scale_log2;
                vs[r] = bf16_lo(vp);
                vm[r] = __fmaf_rn(8.f, vs[r], bf16_hi(vp));
                // (a step that is nothing beside the middle counts as 2^-24 of it: what the weight meets is no larger)
                bound[r] = kRoom - fmaxf(lg2_approx(fmaxf(fabsf(vs[r]), fabsf(vm[r]) * 0x1p-24f)), kLeast);
            }
            const bool masked = slot0 + kU > all_hi || slot0 < all_lo;
            bool over = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint2 q2 = lds8(qs_at + (8 * n + 2 * t) * 4), u2 = lds8(u_at + (8 * n + 2 * t) * 4);
                const float qs[2] = {__uint_as_float(q2.x), __uint_as_float(q2.y)};
                const float u[2] = {__uint_as_float(u2.x), __uint_as_float(u2.y)};
#pragma unroll
                for (int e = 0; e < 4; ++e) s[n][e] = __fmaf_rn(s[n][e], ks[e >> 1], km[e >> 1] * qs[e & 1]);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int tk = sh.tok[qb][8 * n + 2 * t + c], pos = it.pos0 + tk;
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int x = slot + 8 * r;
                            bool sees = x <= pos && (p.rows.window == 0 || x > pos - p.rows.window);
                            if (p.parents) sees = x < own0 || (x - own0 < kTreeNodes && (sh.above[qb][tk] >> (x - own0) & 1));
                            if (!sees) s[n][2 * r + c] = kNegInf;
                            else if (!(fabsf(vm[r]) < __builtin_huge_valf())) s[n][2 * r + c] = __uint_as_float(0x7fc00000u);
                        }
                    }
                    // (a row of V that is not finite is in the scores of the columns that see it now: a weight of 0 would
                    // bring it to the others)
                    if (n == NT - 1) {
#pragma unroll
                        for (int r = 0; r < 2; ++r)
                            if (!(fabsf(vm[r]) < __builtin_huge_valf())) vs[r] = vm[r] = 0.f;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) over = over || s[n][e] - u[e & 1] > bound[e >> 1];
            }
            if (__any_sync(0xffffffffu, over)) {  // some column's u moves up, so that its largest P is 2^kTop
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint2 u2 = lds8(u_at + (8 * n + 2 * t) * 4);
                    float u[2] = {__uint_as_float(u2.x), __uint_as_float(u2.y)}, f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float a = fmaxf(s[n][c] + (kRoom - bound[0]), s[n][2 + c] + (kRoom - bound[1]));
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
                        const bool up = a > u[c] + kRoom;
                        a -= kTop;
                        f[c] = up ? ex2_approx(u[c] - a) : 1.f;
                        if (up) u[c] = a;
                        l[n][c] *= f[c];
                        z[n][c] *= f[c];
                    }
#pragma unroll
                    for (int x = 0; x < kX; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[x][n][e] *= f[e & 1];
                    if (g == 0) *reinterpret_cast<float2 *>(&sh.u[warp][8 * n + 2 * t]) = make_float2(u[0], u[1]);
                }
                __syncwarp();
            }
            // ---- P
            uint32_t p0[NT], p1[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                p0[n] = p1[n] = 0;
                const uint2 u2 = lds8(u_at + (8 * n + 2 * t) * 4);
                const float u[2] = {__uint_as_float(u2.x), __uint_as_float(u2.y)};
                float e[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = ex2_approx(s[n][k] - u[k & 1]);
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    l[n][c] += e[c] + e[2 + c];
                    z[n][c] = __fmaf_rn(e[c], vm[0], __fmaf_rn(e[2 + c], vm[1], z[n][c]));
                }
                p0[n] = transposed(pack_f16x2(e[0] * vs[0], e[1] * vs[0]));
                p1[n] = transposed(pack_f16x2(e[2] * vs[1], e[3] * vs[1]));
            }
            // ---- O^T: a byte of each of four slots' words is two dims' operand
            {
                const uint32_t va = at + kU * kRow + g * (kX), s0 = slot_of(2 * t), s1 = slot_of(2 * t + 1);
                uint32_t w[4][kX / 4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const uint32_t from = va + ((y & 1 ? s1 : s0) + (y >> 1) * 8) * kRow;
                    if constexpr (kX == 8) {
                        const uint2 a = lds8(from);
                        w[y][0] = a.x, w[y][1] = a.y;
                    } else {
                        w[y][0] = lds4(from);
                    }
                }
#pragma unroll
                for (int x = 0; x < kX; ++x) {
                    const int b = x & 3;
                    const uint32_t sel = b | b << 4 | (4 + b) << 8 | (4 + b) << 12;
                    const uint32_t c0 = __byte_perm(w[0][x >> 2], w[1][x >> 2], sel), c1 = __byte_perm(w[2][x >> 2], w[3][x >> 2], sel);
                    const uint32_t a0 = quant::centred_f16(c0), a1 = quant::centred_f16(c0 >> 4);
                    const uint32_t a2 = quant::centred_f16(c1), a3 = quant::centred_f16(c1 >> 4);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_f16(o[x][n], a0, a1, a2, a3, p0[n], p1[n]);
                    }
                }
            }
            __syncwarp();
            fetch(sh.items[qb], got + kDepth);
            ++got;
        }
        // ---- the warps' sums
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (n >= nt) break;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], off);
                    z[n][c] += __shfl_xor_sync(0xffffffffu, z[n][c], off);
                }
                if (g == 0) sh.ml[warp][8 * n + 2 * t + c] = make_float2(sh.u[warp][8 * n + 2 * t + c], l[n][c]);
            }
        }
        const RowsItem cur = sh.items[qb];
        const bool whole = cur.nc == 1;
        const int part = (int)blockIdx.x * 2 + (cur.ci == 0 ? 1 : 0);
        // where column c's row goes; -1: it is padding
        auto out_row = [&](int c) -> long long {
            const int tk = c / p.G;
            return c < cols ? (long long)(cur.row0 + tk) * p.Hq + cur.h * p.G + c - tk * p.G : -1;
        };
#pragma unroll
        for (int n = 0; n < NT; ++n) {  // a block of 8 columns
            if (n >= nt) break;
#pragma unroll
            for (int x = 0; x < kX; ++x)
                sh.meet[(warp * kX + x) * 32 + lane] =
                    make_float4(o[x][n][0] + z[n][0], o[x][n][1] + z[n][1], o[x][n][2] + z[n][0], o[x][n][3] + z[n][1]);
            __syncthreads();
            if (n == 0 && sh.items[qb ^ 1].b >= 0) begin(sh.items[qb ^ 1], qb ^ 1);  // (its copies run while the sums meet)
            // a task: eight dims of two columns
            for (int i = tid; i < kX / 4 * 32; i += kRT) {
                const int ln = i & 31, w4 = i >> 5;
                const int c0 = 8 * n + 2 * (ln & 3);
                float M[2] = {kUnset, kUnset}, sum[2] = {0.f, 0.f}, f[2][kRW], acc[2][8] = {};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int w = 0; w < kRW; ++w) M[c] = fmaxf(M[c], sh.ml[w][c0 + c].x);
#pragma unroll
                    for (int w = 0; w < kRW; ++w) {
                        const float2 y = sh.ml[w][c0 + c];
                        f[c][w] = ex2_approx(y.x - M[c]);
                        sum[c] = __fmaf_rn(y.y, f[c][w], sum[c]);
                    }
                }
#pragma unroll
                for (int w = 0; w < kRW; ++w)
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        constexpr int kDim[4][2] = {{0, 2}, {4, 6}, {1, 3}, {5, 7}};
                        const float4 v = sh.meet[(w * kX + 4 * w4 + b) * 32 + ln];
                        acc[0][kDim[b][0]] = __fmaf_rn(v.x, f[0][w], acc[0][kDim[b][0]]);
                        acc[1][kDim[b][0]] = __fmaf_rn(v.y, f[1][w], acc[1][kDim[b][0]]);
                        acc[0][kDim[b][1]] = __fmaf_rn(v.z, f[0][w], acc[0][kDim[b][1]]);
                        acc[1][kDim[b][1]] = __fmaf_rn(v.w, f[1][w], acc[1][kDim[b][1]]);
                    }
                const int dim = (ln >> 2) * (D / 8) + 8 * w4;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    if (whole) {
                        const long long row = out_row(c0 + c);
                        if (row < 0) continue;
                        const float inv = 1.f / sum[c];
                        *reinterpret_cast<uint4 *>(p.out + row * D + dim) =
                            make_uint4(pack_bf16x2(acc[c][0] * inv, acc[c][1] * inv), pack_bf16x2(acc[c][2] * inv, acc[c][3] * inv),
                                       pack_bf16x2(acc[c][4] * inv, acc[c][5] * inv), pack_bf16x2(acc[c][6] * inv, acc[c][7] * inv));
                        if (p.lse && dim == 0) p.lse[row] = M[c] * kLn2 + logf(sum[c]);
                    } else {
                        float4 *to = reinterpret_cast<float4 *>(p.part_o + ((size_t)part * kRowsCols + c0 + c) * D + dim);
                        __stcg(to, make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]));
                        __stcg(to + 1, make_float4(acc[c][4], acc[c][5], acc[c][6], acc[c][7]));
                        if (dim == 0) __stcg(reinterpret_cast<float2 *>(p.part_ml) + (size_t)part * kRowsCols + c0 + c, make_float2(M[c], sum[c]));
                    }
                }
            }
            __syncthreads();
        }
        if (whole) continue;
        // ---- an item shared by CTAs: the one that arrives last adds the shares up, in their order
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            int *ctr = p.counters + rows_counter(call, cur.c_first);
            int before_me;
            asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before_me) : "l"(ctr) : "memory");
            sh.last = before_me == cur.nc - 1;
        }
        __syncthreads();
        if (!sh.last) continue;
        __threadfence();
        for (int i = tid; i < cols * (D / 8); i += kRT) {
            const int c = i / (D / 8), dim = i % (D / 8) * 8;
            const long long row = out_row(c);
            if (row < 0) continue;
            float acc[8] = {}, M = kUnset, sum = 0.f;
            constexpr int kAhead = 4;
#pragma unroll 1
            for (int k0 = 0; k0 < cur.nc; k0 += kAhead) {
                float2 ml[kAhead];
                float4 a[kAhead], b[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int j = min(k0 + k, cur.nc - 1);
                    const size_t from = (size_t)(2 * (cur.c_first + j) + (j == 0 ? 1 : 0)) * kRowsCols + c;
                    ml[k] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml) + from);
                    a[k] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + from * D + dim));
                    b[k] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + from * D + dim) + 1);
                }
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    if (k0 + k >= cur.nc) continue;
                    const float Mn = fmaxf(M, ml[k].x), f = ex2_approx(M - Mn), w = ex2_approx(ml[k].x - Mn);
                    M = Mn;
                    sum = sum * f + ml[k].y * w;
                    const float v[8] = {a[k].x, a[k].y, a[k].z, a[k].w, b[k].x, b[k].y, b[k].z, b[k].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = __fmaf_rn(v[e], w, acc[e] * f);
                }
            }
            const float inv = 1.f / sum;
            *reinterpret_cast<uint4 *>(p.out + row * D + dim) =
                make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                           pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
            if (p.lse && dim == 0) p.lse[row] = M * kLn2 + logf(sum);
        }
    }
    copies_wait<0>();
    if (tid == 0) {  // the next call's, whose grid may be another
        for (int c = blockIdx.x; c < kRowsMaxGrid; c += gridDim.x) p.counters[rows_counter(call + 1, c)] = 0;
    }
}

namespace {

struct Form {
    const void *fn;
    int cols, smem, ctas;
};

template <int D, int NT>
Form form() {
    return Form{reinterpret_cast<const void *>(&quant_rows_kernel<D, NT>), 8 * NT, (int)sizeof(RowsShared<D, NT>), kCtasAnSm};
}

constexpr int kForms = 2;
// By columns, the fewest first.
const Form &form_at(int D, int i) {
    static const Form f128[kForms] = {form<128, 1>(), form<128, 2>()};
    static const Form f64[kForms] = {form<64, 1>(), form<64, 2>()};
    return D == 128 ? f128[i] : f64[i];
}

// CTAs of a form that the current device holds at once, asked for once a device; 0 where it does not run.
int form_grid(int D, int i) {
    struct Entry {
        int dev, D, i, grid;
    };
    static std::mutex mu;
    static Entry cache[64];
    static int ncache = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int k = 0; k < ncache; ++k)
        if (cache[k].dev == dev && cache[k].D == D && cache[k].i == i) return cache[k].grid;
    const Form &f = form_at(D, i);
    int occ = 0;
    if (cudaFuncSetAttribute(f.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, f.smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, f.fn, kRT, f.smem) != cudaSuccess || occ < 1)
        return 0;
    const int grid = device_sm_count() * (occ < f.ctas ? occ : f.ctas);
    if (ncache < 64) cache[ncache++] = Entry{dev, D, i, grid};
    return grid;
}

}  // namespace

// Rows a sequence go by the call's mean: the lengths are on the device, and any form
// takes any rows.
static long long mean_columns(const ChunkArgs &a) { return ((long long)a.num_rows + a.B - 1) / a.B * (a.Hq / a.Hkv); }

int rows_form(const ChunkArgs &a) {
    const long long mean = mean_columns(a);
    if (mean > kRowsMost) return -1;
    int i = 0;
    while (i + 1 < kForms && form_at(a.D, i).cols < mean) ++i;
    return i;
}

sv_status launch_rows(const ChunkArgs &a, const QuantParams &c, int form, cudaStream_t st) {
    const Form &f = form_at(a.D, form);
    const int grid = form_grid(a.D, form);
    if (grid <= 0 || grid > kRowsMaxGrid) return SV_ERR_CUDA;
    RowsParams p{};
    static_cast<QuantParams &>(p) = c;
    p.q = static_cast<const uint16_t *>(a.q);
    p.q_stride = a.q_stride;
    p.rows = RowsShape{f.cols / p.G, c.shape.window, c.shape.num_rows, c.shape.S_max};  // (G is at most the mean's columns)
    void *args[] = {&p};
    return launch_pdl(f.fn, dim3((unsigned)grid), dim3(kRT), (size_t)f.smem, st, args) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace chunk
}  // namespace sv
