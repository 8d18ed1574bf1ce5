// sv_quant_tc.cu -- attention over pages held in 4 bits on the 5th-generation
// tensor cores: chains, draft trees and parts of prompts.
//
// An item is the rows of some tokens of one sequence and the heads of them that
// share K/V, N = 32, 48 or 64 columns; for each 128-slot tile of K/V
//     S = (1 + codes_k / 16) Q^T + r sum(q) - i u   (128 slots x N, f32 in tensor memory)
//     P = 2^(step S) 2^e, rounded to f16; l += 2^(step S)
//     O^T += (v 2^-e)^T P                           (D dims x N, f32 in tensor memory)
// and out = O / l.  step is 16 steps of the slot's K, scaled to log2 units, r what
// its minimum adds in such steps and i the step's inverse: a column's sum of q and
// its u enter the product as sixteen more dims, each number in three bf16 parts of
// which the six largest products are taken (2^-24 of the whole is left out), so that
// a score comes out of it but for one factor.  The codes are exact in bf16.  e is
// the exponent of a slot's largest value of V, so that f16 holds its values to 2^-12
// of themselves (below 2^-14 of the largest, to 2^-26 of that).  A column's u moves
// only when some P would pass 2^12.
//
// Why slots are the rows of S: a slot's step and exponent are then numbers of the
// thread that has the slot.  With queries as rows every thread would need all of a
// tile's from shared memory, which set the pace (a chunk of 2048 rows after 14336
// slots 640 us).
//
// The softmax groups, warps 0-3 and 4-7, take the tiles in turn, a thread a slot,
// each with its own u, l and O, so that one's exponentials run beside the other's
// loads; at an item's end the group of its first tile brings the two together, a
// thread a dim.  Warps 8-11 turn a tile's codes into operands, a thread a slot:
// K's to tensor memory, V's to shared memory.  12 loads codes, parameters and
// queries, 13 issues the products, 14 walks the work list (sv_quant_list.h), 15
// adds the sums of an item's queries to them.  An
// item cut by a CTA's range leaves its share in the workspace; the CTA that arrives
// last adds the shares up in their order.  Every wait is bounded; the warps of a
// softmax group agree on a wait that gave up before any of them leaves the group's
// barriers.
#include "sv_attn_common.cuh"
#include "sv_chunk.cuh"
#include "sv_quant.cuh"
#include "sv_quant_walk.cuh"

namespace sv {
namespace chunk {

namespace {

constexpr int kTT = 512;                       // threads
constexpr int kN = 64;                         // columns of an item at most
constexpr uint32_t kTCols = 512, kTColS = 0, kTColO = 128, kTColK = 256;  // one a group each, 64 columns apart
constexpr uint32_t kTColsK = 80;               // of K's operand: D / 2, and eight for the sixteen dims more

// 256 x 184 + 256 x 72 = 256 x 168 + 256 x 88 = 512 x 128
template <int kCh>
constexpr int kTRegsSoftmax = kCh == 4 ? 184 : 168;
template <int kCh>
constexpr int kTRegsOther = 256 - kTRegsSoftmax<kCh>;

template <int D>
constexpr int kVTile = kBK * D * 2;            // V's operand
constexpr int kPTile = kBK * kN * 2;
constexpr int kQBox = kN * 128;                // 64 columns of 64 dims
constexpr int kExt = kQBox;                    // the sixteen dims more, of two items' and two groups' columns
template <int D>
constexpr int kQTile = kQBox * (D / 64);
template <int D>
constexpr int kTRaw = kBK * (D + 8);           // a tile's codes and parameters
template <int D>
constexpr int kTRawStages = D == 128 ? 4 : 7;

struct TShared {
    uint64_t raw_full[8], raw_empty[8];
    uint64_t k_full[2], k_empty[2], v_full[2], pv_done[2];
    uint64_t s_full[2], s_empty[2], p_full[2];
    uint64_t q_full[2], q_empty[2], ext_full[2], o_full[2], o_empty[2], x_full;
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t fin;
    RowsItem items[kItems];
    float2 slots[4][kBK];              // a tile's slots: K's step, 2^e
    float u[2][kN];                    // a group's columns'
    float part[2][4][kN];              // a warp's maxima or sums
    float2 f[2][kN / 2], d[2][kN / 2]; // what a column's sums are to be multiplied by, what is to be added to its scores
    float2 other[kN];                  // the (u, l) of the group that does not finish the item
    float2 w[2][kN];                   // what the two groups' O are to be multiplied by
    unsigned long long above[2][kTreeNodes];
    long long warp_units[kTT / 32];
    long long before[kTT];
    unsigned long long call;
    uint8_t tok[kN];
    uint32_t tmem;
    int abort_flag, last[2];
};

template <int D>
constexpr int kTSmem = 2 * (kVTile<D> + kPTile + kQTile<D>) + kExt + kTRawStages<D> * kTRaw<D> + (int)sizeof(TShared);
static_assert(kTSmem<128> <= 227 * 1024 && kTSmem<64> <= 227 * 1024, "shared memory");

// Wait for the phase of `bar` with the given parity, by a whole warp with one verdict; a probe suspends
// the warp for some 150 cycles, so that this many take about a second.
constexpr int kProbes = 1 << 23;
__device__ __noinline__ bool twait_long(uint64_t *bar, uint32_t parity) {
    bool ok = false;
#pragma unroll 1
    for (int i = 0; i < kProbes && !ok; ++i) ok = mbar_try_wait(bar, parity);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool twait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || twait_long(bar, parity);
}
// The same without a call, for the softmax warps (a function that both parts call costs the kernel its
// register split).
__device__ __forceinline__ bool twait_here(uint64_t *bar, uint32_t parity) {
    bool ok = mbar_try_wait(bar, parity);
#pragma unroll 1
    for (int i = 0; i < kProbes && !ok; ++i) ok = mbar_try_wait(bar, parity);
    return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ uint32_t telect() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// Barrier of a softmax group's 128 threads; whether any of them says so.
__device__ __forceinline__ bool group_any(int group, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x), "r"(1 + group)
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void group_sync(int group) { named_bar_sync(1 + group, 128); }

// 16 columns of tensor memory as eight pairs.
__device__ __forceinline__ void tmem_ld16(uint32_t at, float2 *x) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const float2 *x) {
    uint32_t r[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[2 * i] = __float_as_uint(x[i].x), r[2 * i + 1] = __float_as_uint(x[i].y);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t at, const float2 (&x)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(at),
                 "r"(__float_as_uint(x[0].x)), "r"(__float_as_uint(x[0].y)), "r"(__float_as_uint(x[1].x)),
                 "r"(__float_as_uint(x[1].y)), "r"(__float_as_uint(x[2].x)), "r"(__float_as_uint(x[2].y)),
                 "r"(__float_as_uint(x[3].x)), "r"(__float_as_uint(x[3].y))
                 : "memory");
}

__device__ __forceinline__ uint32_t t_sw128(int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); }

__device__ __forceinline__ uint32_t t_pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// x as three bf16 parts, the halves of the words a sum of products needs: side A's (x1, x1, x2, x1, x3, x2)
// or side B's (x1, x2, x1, x3, x1, x2), two zeros behind them.
template <bool kA>
__device__ __forceinline__ uint4 parts3(float x) {
    const uint32_t a = pack_bf16x2(x, 0.f) & 0xffffu;
    const float y = x - __uint_as_float(a << 16);
    const uint32_t b = pack_bf16x2(y, 0.f) & 0xffffu;
    const uint32_t c = pack_bf16x2(y - __uint_as_float(b << 16), 0.f) & 0xffffu;
    return kA ? make_uint4(a | a << 16, b | a << 16, c | b << 16, 0u) : make_uint4(a | b << 16, a | c << 16, a | b << 16, 0u);
}

// The sums (or maxima) over the warp of 16 values a lane: lane c's and c + 16's is that of v[c].
template <bool kMax>
__device__ __forceinline__ float across(float (&v)[16], int lane) {
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < off; ++i) {
            const float keep = up ? v[i + off] : v[i], send = up ? v[i] : v[i + off];
            const float got = __shfl_xor_sync(0xffffffffu, send, off);
            v[i] = kMax ? fmaxf(keep, got) : keep + got;
        }
    }
    const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
    return kMax ? fmaxf(v[0], got) : v[0] + got;
}

}  // namespace

template <int D, int kCh>  // kCh chunks of 8 columns a softmax group
__global__ void __launch_bounds__(kTT, 1) quant_tc_kernel(const __grid_constant__ CUtensorMap tmq, const RowsParams p) {
    constexpr int kRow = D / 2, kRaw = kTRawStages<D>, N = 16 * kCh;
    extern __shared__ __align__(1024) uint8_t smem[];  // (the swizzle's atoms are 1024 bytes)
    uint8_t *const vbuf = smem, *const pbuf = vbuf + 2 * kVTile<D>, *const qbuf = pbuf + 2 * kPTile;
    uint8_t *const ext = qbuf + 2 * kQTile<D>, *const raw = ext + kExt;
    TShared *sh = reinterpret_cast<TShared *>(raw + kRaw * kTRaw<D>);
    const uint32_t base_u32 = smem_u32(smem);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(&sh->raw_full[i], 1);
            mbar_init(&sh->raw_empty[i], 4);
        }
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->k_full[i], 4);
            mbar_init(&sh->k_empty[i], 1);
            mbar_init(&sh->v_full[i], 4);
            mbar_init(&sh->pv_done[i], 1);
            mbar_init(&sh->s_full[i], 1);
            mbar_init(&sh->s_empty[i], 4);
            mbar_init(&sh->p_full[i], 4);
            mbar_init(&sh->q_full[i], 1);
            mbar_init(&sh->q_empty[i], 1 + 1);  // the products, the sums
            mbar_init(&sh->ext_full[i], 1);
            mbar_init(&sh->o_full[i], 1);
            mbar_init(&sh->o_empty[i], 4);
        }
#pragma unroll 1
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sh->item_full[i], 1);
            mbar_init(&sh->item_empty[i], 8 + 4 + 2 + 1);
        }
        mbar_init(&sh->x_full, 1);
        mbar_init(&sh->fin, 1);
        sh->abort_flag = 0;
        fence_mbar_init();
    }
    for (int i = tid; i < (2 * kQTile<D> + kExt) / 16; i += kTT) reinterpret_cast<uint4 *>(qbuf)[i] = make_uint4(0, 0, 0, 0);  // (columns past the items' stay zeros)
    tc::fence_proxy_async_smem();
    if (tid < kN) sh->tok[tid] = (uint8_t)(tid / p.Gs);
    if (tid == 32 * 12) prefetch_tensormap(&tmq);
    if (warp == 13) tc::tmem_alloc(&sh->tmem, kTCols);
    griddep_wait();
    griddep_launch_dependents();
    if (tid == 0) sh->call = begin_call(p.call);
    RowsWalk walk;
    tc::fence_before();
    plan_walk<kTT>(p, sh->warp_units, sh->before, tid, 14, walk);  // (two barriers of the CTA)
    tc::fence_after();
    const uint32_t tbase = sh->tmem;
    volatile int *abort_flag = &sh->abort_flag;
    auto fail = [&] { *abort_flag = 1; };
    const bool aligned = (base_u32 & 1023u) == 0;  // (always: nothing else takes shared memory here)

    if (warp < 8) {
        // ===================== softmax: a thread a slot, every second tile
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTRegsSoftmax<kCh>));
        const int group = warp >> 2, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t tl = tbase + ((uint32_t)(quarter * 32) << 16);
        const uint32_t s_at = tl + kTColS + group * kN, o_at = tl + kTColO + group * kN;
        uint8_t *const pto = pbuf + group * kPTile;
        uint32_t tile = 0, o_ph = 0, x_ph = 0;  // tiles of the CTA before this item
        bool bad = !aligned;
#pragma unroll 1
        for (uint32_t k = 0;; ++k) {
            const int slot_i = k % kItems;
            bad = bad || !twait_here(&sh->item_full[slot_i], (k / kItems) & 1);
            if (group_any(group, bad)) {
                bad = true;
                break;
            }
            const RowsItem it = sh->items[slot_i];
            if (it.b < 0) break;
            const int own0 = it.pos0 - (it.row0 - it.seq_row0);  // slot of the sequence's first new row
            const int all_hi = p.parents ? own0 : it.pos0 + 1;   // below, and from all_lo on, every row sees a slot
            const int all_lo = p.rows.window > 0 ? it.pos0 + it.ntok - p.rows.window : 0;
            if (r < N) sh->u[group][r] = kUnset;
            if (p.parents && quarter < 2) {  // a token's set of nodes above it, of those up to the item's last
                const int node0 = it.row0 - it.seq_row0, nodes = min(node0 + it.ntok, kTreeNodes);
                const int32_t *par = p.parents + it.seq_row0;
                const int a = lane < nodes ? par[lane] : -1, b = lane + 32 < nodes ? par[lane + 32] : -1;
                sh->above[group][r] = ancestors_warp(false, a, b, node0 + r, r < it.ntok && node0 + r < nodes);
            }
            group_sync(group);
            bool unset = true;  // some column has no u yet
            float2 l[N / 2];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) l[i] = make_float2(0.f, 0.f);
            const int j0 = (group ^ (int)tile) & 1;  // this group's first tile of the item
#pragma unroll 1
            for (int j = j0; j < it.n; j += 2) {
                const uint32_t g = tile + j, ph = (g >> 1) & 1;
                const int slot0 = (it.kt0 + j) * kBK, slot = slot0 + r;
                bad = bad || !twait_here(&sh->s_full[group], ph);
                tc::fence_after();
                const float2 par = sh->slots[g & 3][r];
                const float ks = par.x, w = par.y, e = (float)((int)(__float_as_uint(w) >> 23) - 127);  // w: 2^e
                const float2 ks2 = make_float2(ks, ks), w2 = make_float2(w, w);
                const bool masked = slot0 + kBK > all_hi || slot0 < all_lo;
                float2 x[N / 2];
#pragma unroll
                for (int ch = 0; ch < N / 16; ++ch) tmem_ld16(s_at + 16 * ch, x + 8 * ch);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < N / 2; ++i) x[i] = __fmul2_rn(x[i], ks2);
                if (masked) {
                    unsigned long long sees = ~0ull;  // a bit a column
                    if (p.parents) {
                        const int node = slot - own0;
                        if (node >= 0) {
                            sees = 0;
#pragma unroll 1
                            for (int c = 0; c < N; ++c) {
                                const int tk = min((int)sh->tok[c], it.ntok - 1);
                                if (node < kTreeNodes && (sh->above[group][tk] >> node & 1)) sees |= 1ull << c;
                            }
                        }
                    } else {  // tokens slot - pos0 .. slot - pos0 + window - 1
                        const long long from = (long long)(slot - it.pos0) * p.Gs;
                        const long long to = p.rows.window > 0 ? from + (long long)p.rows.window * p.Gs : 64;
                        const unsigned long long under = from >= 64 ? ~0ull : from <= 0 ? 0ull : (1ull << from) - 1ull;
                        const unsigned long long below = to >= 64 ? ~0ull : to <= 0 ? 0ull : (1ull << to) - 1ull;
                        sees = below & ~under;
                    }
                    const uint32_t half[2] = {(uint32_t)sees, (uint32_t)(sees >> 32)};
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        if (!(half[i >> 4] >> (2 * i & 31) & 1)) x[i].x = kNegInf;
                        if (!(half[i >> 4] >> ((2 * i & 31) + 1) & 1)) x[i].y = kNegInf;
                    }
                }
                float top[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                for (int i = 0; i < N / 2; ++i) top[i & 3] = fmaxf(fmaxf(top[i & 3], x[i].x), x[i].y);
                if (group_any(group, bad || unset || fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) + e > kRoom)) {
                    if (group_any(group, bad)) {
                        bad = true;
                        break;
                    }
                    // some column's u moves up to its largest P (the first tile's do)
                    const float2 *const us = reinterpret_cast<const float2 *>(sh->u[group]);
#pragma unroll
                    for (int h = 0; h < N / 16; ++h) {
                        float v[16];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 y = x[8 * h + i], u = us[8 * h + i];
                            v[2 * i] = y.x + (e + (u.x == kUnset ? 0.f : u.x));
                            v[2 * i + 1] = y.y + (e + (u.y == kUnset ? 0.f : u.y));
                        }
                        const float a = across<true>(v, lane);
                        if (lane < 16) sh->part[group][quarter][16 * h + lane] = a;
                    }
                    group_sync(group);
                    bool still = false;
                    if (r < N) {
                        const float a = fmaxf(fmaxf(sh->part[group][0][r], sh->part[group][1][r]),
                                              fmaxf(sh->part[group][2][r], sh->part[group][3][r]));
                        const float u = sh->u[group][r];
                        const bool none = u == kUnset, up = a > u + kRoom;
                        const float was = none ? 0.f : u, now = up ? a : was;
                        reinterpret_cast<float *>(sh->f[group])[r] = up ? ex2_approx(u - a) : 1.f;
                        reinterpret_cast<float *>(sh->d[group])[r] = was - now;
                        if (up) {
                            sh->u[group][r] = a;
                            // (behind the group's last S of the item the place may be the next item's but one)
                            if (j + 2 < it.n) *reinterpret_cast<uint4 *>(ext + t_sw128(r, ((k & 1) * 2 + group) * 2 + 1)) = parts3<false>(-a);
                        }
                        still = none && !up;
                    }
                    tc::fence_proxy_async_smem();  // (the next S reads u)
                    // (the products that added to O last)
                    if (j > j0) bad = !twait_here(&sh->pv_done[group], ph ^ 1);
                    if (group_any(group, bad)) {
                        bad = true;
                        break;
                    }
                    unset = group_any(group, still);
                    tc::fence_after();
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        l[i] = __fmul2_rn(l[i], sh->f[group][i]);
                        x[i] = __fadd2_rn(x[i], sh->d[group][i]);
                    }
                    if (j > j0) {
#pragma unroll 1
                        for (int ch = 0; ch < N / 16; ++ch) {
                            float2 o[8];
                            tmem_ld16(o_at + 16 * ch, o);
                            tc::wait_ld();
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] = __fmul2_rn(o[i], sh->f[group][8 * ch + i]);
                            tmem_st16(o_at + 16 * ch, o);
                        }
                        tc::wait_st();
                    }
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->s_empty[group]);
                bad = !twait_here(&sh->pv_done[group], ph ^ 1);  // (P's place; told at the next vote)
#pragma unroll
                for (int ch = 0; ch < N / 8; ++ch) {
                    uint32_t y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int n = 4 * ch + i;
                        const float2 z = make_float2(ex2_approx(x[n].x), ex2_approx(x[n].y));
                        l[n] = __fadd2_rn(l[n], z);
                        const float2 q = __fmul2_rn(z, w2);
                        y[i] = t_pack_f16x2(q.x, q.y);
                    }
                    *reinterpret_cast<uint4 *>(pto + r * 128 + ((ch ^ (r & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[group]);
            }
            // ---- the columns' sums over the slots
            const bool mine = j0 == 0, both = it.n > 1;  // whether this group finishes the item; whether the other has a share
            if (j0 < it.n) {
                bad = bad || !twait_here(&sh->o_full[group], o_ph);
                o_ph ^= 1;
            }
#pragma unroll
            for (int h = 0; h < N / 16; ++h) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[2 * i] = l[8 * h + i].x;
                    v[2 * i + 1] = l[8 * h + i].y;
                }
                const float a = across<false>(v, lane);
                if (lane < 16) sh->part[group][quarter][16 * h + lane] = a;
            }
            tile += it.n;
            if (group_any(group, bad)) {
                bad = true;
                break;
            }
            tc::fence_after();
            float lsum = 0.f, u = 0.f;
            if (r < N) {
                lsum = (sh->part[group][0][r] + sh->part[group][1][r]) + (sh->part[group][2][r] + sh->part[group][3][r]);
                u = sh->u[group][r];
            }
            if (!mine) {
                x_ph ^= both ? 1 : 0;
                if (both && r < N) sh->other[r] = make_float2(u, lsum);
                tc::fence_before();
                group_sync(group);
                if (both && r == 0) mbar_arrive(&sh->x_full);
                if (lane == 0) mbar_arrive(&sh->item_empty[slot_i]);
                continue;
            }
            if (both) {
                bad = !twait_here(&sh->x_full, x_ph);
                x_ph ^= 1;
                tc::fence_after();
            }
            const bool whole = it.nc == 1;
            const int part = (int)blockIdx.x * 2 + (it.ci == 0 ? 1 : 0), cols = it.ntok * p.Gs;
            const int hpart = it.h % p.parts * p.Gs, heads = min(p.Gs, p.G - hpart);
            const int head0 = it.h / p.parts * p.G + hpart;
            // where a column's row goes; -1: it is padding
            auto out_row = [&](int c) -> long long {
                const int tk = sh->tok[c], hd = c - tk * p.Gs;
                return c < cols && hd < heads ? (long long)(it.row0 + tk) * p.Hq + head0 + hd : -1;
            };
            if (r < N) {
                const float2 y = both ? sh->other[r] : make_float2(kUnset, 0.f);
                const float M = fmaxf(u, y.x), f0 = ex2_approx(u - M), f1 = ex2_approx(y.x - M);
                const float sum = lsum * f0 + y.y * f1, inv = whole ? 1.f / sum : 1.f;
                sh->w[group][r] = make_float2(f0 * inv, f1 * inv);
                const long long row = out_row(r);
                if (!whole) __stcg(reinterpret_cast<float2 *>(p.part_ml) + (size_t)part * kRowsCols + r, make_float2(M, sum));
                else if (p.lse && row >= 0) p.lse[row] = M * kLn2 + logf(sum);
            }
            if (group_any(group, bad)) {
                bad = true;
                break;
            }
            const uint32_t o2_at = tl + kTColO + (group ^ 1) * kN;
#pragma unroll 1
            for (int ch = 0; ch < N / 16; ++ch) {  // 16 columns of a dim
                float2 a[8], b[8];
                __syncwarp();
                tmem_ld16(o_at + 16 * ch, a);
                if (both) tmem_ld16(o2_at + 16 * ch, b);
                tc::wait_ld();
                if (r < D) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int c = 16 * ch + i;
                        const float2 f = sh->w[group][c];
                        float y = (i & 1 ? a[i >> 1].y : a[i >> 1].x) * f.x;
                        if (both) y = __fmaf_rn(i & 1 ? b[i >> 1].y : b[i >> 1].x, f.y, y);
                        if (whole) *reinterpret_cast<uint16_t *>(pto + (c * D + r) * 2) = (uint16_t)pack_bf16x2(y, 0.f);
                        else __stcg(p.part_o + ((size_t)part * kRowsCols + c) * D + r, y);
                    }
                }
            }
            tc::fence_before();
            if (!whole) __threadfence();
            group_sync(group);
            if (lane == 0) {  // O may start over
                mbar_arrive(&sh->o_empty[group]);
                if (both) mbar_arrive(&sh->o_empty[group ^ 1]);
                mbar_arrive(&sh->item_empty[slot_i]);
            }
            if (whole) {  // rows by 16 bytes, through the place of P
#pragma unroll 1
                for (int i = r; i < N * (D / 8); i += 128) {
                    const int c = i / (D / 8), piece = i % (D / 8);
                    const long long row = out_row(c);
                    if (row >= 0) *reinterpret_cast<uint4 *>(p.out + row * D + piece * 8) = *reinterpret_cast<const uint4 *>(pto + (c * D + piece * 8) * 2);
                }
                continue;  // (the next item's first vote comes before the next P)
            }
            // ---- an item shared by CTAs: the one that arrives last adds the shares up, in their order
            if (r == 0) {
                int *ctr = p.counters + rows_counter(sh->call, it.c_first);
                int before_me;
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(before_me) : "l"(ctr) : "memory");
                sh->last[group] = before_me == it.nc - 1;
            }
            group_sync(group);
            if (!sh->last[group]) continue;
            __threadfence();
#pragma unroll 1
            for (int i = r; i < N * (D / 8); i += 128) {
                const int c = i / (D / 8), dim = i % (D / 8) * 8;
                const long long row = out_row(c);
                if (row < 0) continue;
                float acc[8] = {}, M = kUnset, sum = 0.f;
                constexpr int kAhead = 4;
#pragma unroll 1
                for (int k0 = 0; k0 < it.nc; k0 += kAhead) {
                    float2 ml[kAhead];
                    float4 a[kAhead], b[kAhead];
#pragma unroll
                    for (int q = 0; q < kAhead; ++q) {
                        const int m = min(k0 + q, it.nc - 1);
                        const size_t from = (size_t)(2 * (it.c_first + m) + (m == 0 ? 1 : 0)) * kRowsCols + c;
                        ml[q] = __ldcg(reinterpret_cast<const float2 *>(p.part_ml) + from);
                        a[q] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + from * D + dim));
                        b[q] = __ldcg(reinterpret_cast<const float4 *>(p.part_o + from * D + dim) + 1);
                    }
#pragma unroll
                    for (int q = 0; q < kAhead; ++q) {
                        if (k0 + q >= it.nc) continue;
                        const float Mn = fmaxf(M, ml[q].x), f = ex2_approx(M - Mn), w = ex2_approx(ml[q].x - Mn);
                        M = Mn;
                        sum = sum * f + ml[q].y * w;
                        const float y[8] = {a[q].x, a[q].y, a[q].z, a[q].w, b[q].x, b[q].y, b[q].z, b[q].w};
#pragma unroll
                        for (int z = 0; z < 8; ++z) acc[z] = __fmaf_rn(y[z], w, acc[z] * f);
                    }
                }
                const float in = 1.f / sum;
                *reinterpret_cast<uint4 *>(p.out + row * D + dim) =
                    make_uint4(pack_bf16x2(acc[0] * in, acc[1] * in), pack_bf16x2(acc[2] * in, acc[3] * in),
                               pack_bf16x2(acc[4] * in, acc[5] * in), pack_bf16x2(acc[6] * in, acc[7] * in));
                if (p.lse && dim == 0) p.lse[row] = M * kLn2 + logf(sum);
            }
        }
        if (bad) fail();
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTRegsOther<kCh>));
        if (warp < 12) {
            // ===================== codes to operands: a thread a slot
            const int quarter = warp & 3, r = quarter * 32 + lane;
            const uint32_t k_at = tbase + ((uint32_t)(quarter * 32) << 16) + kTColK;
            uint32_t g = 0;
            bool ok = aligned;
#pragma unroll 1
            for (uint32_t k = 0; ok; ++k) {
                const int slot_i = k % kItems;
                if (!(ok = twait(&sh->item_full[slot_i], (k / kItems) & 1))) break;
                const int b = sh->items[slot_i].b, n = sh->items[slot_i].n, pos0 = sh->items[slot_i].pos0;
                const int ntok = sh->items[slot_i].ntok, kt0 = sh->items[slot_i].kt0;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->item_empty[slot_i]);
                if (b < 0) break;
                const int lo = p.rows.window > 0 ? max(0, pos0 - p.rows.window + 1) : 0, hi = pos0 + ntok;
#pragma unroll 1
                for (int j = 0; j < n; ++j, ++g) {
                    const uint32_t rs = g % kRaw, buf = g & 1, ph = (g >> 1) & 1;
                    if (!(ok = twait(&sh->raw_full[rs], (g / kRaw) & 1))) break;
                    const uint8_t *from = raw + rs * kTRaw<D>;
                    const int at = (kt0 + j) * kBK + r;
                    const bool seen = at >= lo && at < hi;  // (another slot may hold anything)
                    const uint32_t *par = reinterpret_cast<const uint32_t *>(from + 2 * kBK * kRow);
                    // pieces of 32 dims, in turn from another one on for rows two and two (four and four), so
                    // that eight lanes of an access meet eight bank groups
                    constexpr int kPieces = D / 32;
                    const int turn = r >> (D == 128 ? 1 : 2);
                    uint4 c[kPieces];
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        c[i] = *reinterpret_cast<const uint4 *>(from + r * kRow + ((i + turn) & (kPieces - 1)) * 16);
                    if (!(ok = twait(&sh->k_empty[buf], ph ^ 1))) break;
                    tc::fence_after();
                    // V's values times 2^-e, below 2
                    const uint32_t vpar = seen ? par[kBK + r] : 0u, kpar = seen ? par[r] : 0u;
                    const float vstep = bf16_lo(vpar), vmid = __fmaf_rn(8.f, vstep, bf16_hi(vpar));
                    const uint32_t most = __float_as_uint(__fmaf_rn(8.f, fabsf(vstep), fabsf(vmid))) >> 23;
                    const uint32_t e = min(max(most, (uint32_t)(127 + (int)kLeast)), 253u);  // the exponent, and 127
                    const float down = __uint_as_float((254u - e) << 23);
                    const uint32_t step2 = t_pack_f16x2(vstep * down, vstep * down), mid2 = t_pack_f16x2(vmid * down, vmid * down);
                    // K's score in units of 16 steps: 1 + code / 16, and a multiple of the sum of q.  Codes that say less
                    // than 2^-60 of the middle, or than 2^-100, are left out
                    const float k16 = 16.f * bf16_lo(kpar) * p.scale_log2;
                    const float kmid = __fmaf_rn(8.f, bf16_lo(kpar), bf16_hi(kpar)) * p.scale_log2;
                    const float least = fmaxf(0x1p-100f, fabsf(kmid) * 0x1p-60f);
                    const bool coded = fabsf(k16) >= least;
                    const float ks = coded ? k16 : fmaxf(0x1p-100f, fabsf(kmid)), inv = 1.f / ks;
                    const float rest = coded ? __fmaf_rn(kmid, inv, -1.5f) : kmid * inv;
                    sh->slots[g & 3][r] = make_float2(ks, __uint_as_float(e << 23));
                    // (a thread's row in order: the pieces put back by selects, a bit of the turn at a time)
                    if constexpr (kPieces == 4) {
                        const bool one = turn & 1, two = turn & 2;
                        uint4 y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) y[i] = one ? c[(i + 3) & 3] : c[i];
#pragma unroll
                        for (int i = 0; i < 4; ++i) c[i] = two ? y[(i + 2) & 3] : y[i];
                    } else {
                        const uint4 y = c[0];
                        c[0] = turn & 1 ? c[1] : y;
                        c[1] = turn & 1 ? y : c[1];
                    }
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {  // 32 dims, 16 columns of tensor memory at a time
                        const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
                        float2 x[8];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint4 y = quant::sixteenths(words[q]);
                            if (!coded) y = make_uint4(0, 0, 0, 0);
                            x[2 * q] = make_float2(__uint_as_float(y.x), __uint_as_float(y.y));
                            x[2 * q + 1] = make_float2(__uint_as_float(y.z), __uint_as_float(y.w));
                        }
                        tmem_st16(k_at + buf * kTColsK + i * 16, x);
                    }
                    {
                        const uint4 a = parts3<true>(rest), b = parts3<true>(inv);
                        const float2 x[4] = {make_float2(__uint_as_float(a.x), __uint_as_float(a.y)), make_float2(__uint_as_float(a.z), 0.f),
                                             make_float2(__uint_as_float(b.x), __uint_as_float(b.y)), make_float2(__uint_as_float(b.z), 0.f)};
                        tmem_st8(k_at + buf * kTColsK + D / 2, x);
                    }
                    // V's codes, on their way while K's are written
#pragma unroll
                    for (int i = 0; i < kPieces; ++i)
                        c[i] = *reinterpret_cast<const uint4 *>(from + kBK * kRow + r * kRow + ((i + turn) & (kPieces - 1)) * 16);
                    tc::wait_st();
                    tc::fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh->k_full[buf]);
                        mbar_arrive(&sh->raw_empty[rs]);
                    }
                    if (!(ok = twait(&sh->pv_done[buf], ph ^ 1))) break;
                    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) {
                        ok = false;
                        break;
                    }
                    uint8_t *const to = vbuf + buf * kVTile<D> + r * 128;
#pragma unroll
                    for (int i = 0; i < kPieces; ++i) {
                        const int piece = (i + turn) & (kPieces - 1);
                        const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(to + (piece >> 1) * kBox + ((((piece & 1) * 4 + q) ^ (r & 7)) << 4)) =
                                quant::scaled_f16(words[q], step2, mid2);
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->v_full[buf]);
                }
            }
            if (!ok) fail();
        } else if (warp == 12) {
            // ===================== codes and parameters of the tiles, a lane a page; the queries
            const int ps = p.page_size;
            const int sub = ps < kBK ? ps : kBK;      // slots of a copy
            const int npg = kBK / sub;                // copies a tile
            const int tpp = ps < kBK ? 1 : ps / kBK;  // tiles a page (of 128 slots or more)
            uint32_t g = 0, nq = 0;
            bool ok = aligned;
#pragma unroll 1
            for (uint32_t k = 0; ok; ++k) {
                const int slot_i = k % kItems;
                if (!(ok = twait(&sh->item_full[slot_i], (k / kItems) & 1))) break;
                const RowsItem it = sh->items[slot_i];
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->item_empty[slot_i]);
                if (it.b < 0) break;
                const int lo = p.rows.window > 0 ? max(0, it.pos0 - p.rows.window + 1) : 0, hi = it.pos0 + it.ntok;
                const int32_t *trow = p.block_table + (size_t)it.b * p.max_pages;
                // cache row of the first slot of this lane's copy of tile j; -1: no slot of it is seen.  In the place
                // of a page id out of range (reported by the check, its rows unspecified) page 0 is read.
                auto first_row = [&](int j) -> int {
                    const int t = it.kt0 + j, s0 = t * kBK + lane * sub;
                    if (lane >= npg || s0 >= hi || s0 + sub <= lo) return -1;
                    const int page = tpp == 1 ? t * npg + lane : t / tpp;
                    int pg = trow[page];
                    if (pg < 0 || pg >= p.num_pages) pg = 0;
                    return (pg * p.Hkv + it.h / p.parts) * ps + (tpp == 1 ? 0 : (t - page * tpp) * kBK);
                };
                int y = first_row(0);
                if (!(ok = twait(&sh->q_empty[k & 1], ((k >> 1) & 1) ^ 1))) break;
                if (lane == 0) {
                    uint8_t *qd = qbuf + (k & 1) * kQTile<D>;
                    mbar_arrive_expect_tx(&sh->q_full[k & 1], (uint32_t)(D * 2 * p.Gs * p.rows.tok));
#pragma unroll 1
                    for (int hf = 0; hf < D / 64; ++hf)
                        tma_load_3d(qd + hf * kQBox, &tmq, hf * 64, it.h / p.parts * p.G + it.h % p.parts * p.Gs, it.row0, &sh->q_full[k & 1]);
                }
                __syncwarp();
                ++nq;
#pragma unroll 1
                for (int j = 0; j < it.n; ++j, ++g) {
                    const int y_next = j + 1 < it.n ? first_row(j + 1) : -1;
                    const int copies = __popc(__ballot_sync(0xffffffffu, y >= 0));
                    const uint32_t rs = g % kRaw;
                    if (!(ok = twait(&sh->raw_empty[rs], ((g / kRaw) & 1) ^ 1))) break;
                    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) mbar_arrive_expect_tx(&sh->raw_full[rs], (uint32_t)(copies * sub * (D + 8)));
                    __syncwarp();  // the expected bytes are set before any copy lands
                    if (y >= 0) {
                        uint8_t *to = raw + rs * kTRaw<D>;
                        uint64_t *bar = &sh->raw_full[rs];
                        bulk_load(to + lane * sub * kRow, p.k_codes + (size_t)y * kRow, (uint32_t)(sub * kRow), bar);
                        bulk_load(to + kBK * kRow + lane * sub * kRow, p.v_codes + (size_t)y * kRow, (uint32_t)(sub * kRow), bar);
                        bulk_load(to + 2 * kBK * kRow + lane * sub * 4, p.k_params + y, (uint32_t)(sub * 4), bar);
                        bulk_load(to + 2 * kBK * kRow + kBK * 4 + lane * sub * 4, p.v_params + y, (uint32_t)(sub * 4), bar);
                    }
                    y = y_next;
                }
            }
            if (!ok) fail();
            // every copy issued must land before the CTA may exit
#pragma unroll 1
            for (uint32_t q = nq > 2 ? nq - 2 : 0; q < nq; ++q) twait(&sh->q_full[q & 1], (q >> 1) & 1);
            if (__shfl_sync(0xffffffffu, *abort_flag, 0))
#pragma unroll 1
                for (uint32_t q = g > kRaw ? g - kRaw : 0; q < g; ++q) twait(&sh->raw_full[q % kRaw], (q / kRaw) & 1);
        } else if (warp == 13) {
            // ===================== the products: S of a tile, then O of the tile before
            const uint32_t leader = telect();
            const uint64_t desc_v = tc::smem_desc(base_u32, kBox, 1024);
            const uint64_t desc_p = tc::smem_desc(base_u32 + 2 * kVTile<D>, kPTile, 1024);
            const uint64_t desc_q = tc::smem_desc(base_u32 + 2 * (kVTile<D> + kPTile), 16, 1024);
            const uint64_t desc_x = tc::smem_desc(base_u32 + 2 * (kVTile<D> + kPTile + kQTile<D>), 16, 1024);
            uint32_t g = 0;
            bool ok = aligned;
            // the tile whose O is still to be added to: a group's first or last of its item
            bool live = false, first = false, end = false;
            uint32_t o_ph = 3;  // a bit a group
            auto add_o = [&]() -> bool {
                const uint32_t t = g - 1, buf = t & 1, ph = (t >> 1) & 1;
                if (!twait(&sh->v_full[buf], ph) || !twait(&sh->p_full[buf], ph)) return false;
                if (first) {
                    if (!twait(&sh->o_empty[buf], (o_ph >> buf) & 1)) return false;
                    o_ph ^= 1u << buf;
                }
                tc::fence_after();
                // f16 both, V's dims and P's columns contiguous
                constexpr uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        tc::mma_bf16(tbase + kTColO + buf * kN, desc_v + (uint64_t)(buf * (kVTile<D> >> 4) + kk * (2048 >> 4)),
                                     desc_p + (uint64_t)(buf * (kPTile >> 4) + kk * (2048 >> 4)), idesc, kk > 0 || !first ? 1u : 0u);
                    tc::commit(&sh->pv_done[buf]);
                    if (end) tc::commit(&sh->o_full[buf]);
                }
                __syncwarp();
                return true;
            };
#pragma unroll 1
            for (uint32_t k = 0; ok; ++k) {
                const int slot_i = k % kItems;
                if (!(ok = twait(&sh->item_full[slot_i], (k / kItems) & 1))) break;
                const int b = __reduce_max_sync(0xffffffffu, sh->items[slot_i].b), n = __reduce_max_sync(0xffffffffu, sh->items[slot_i].n);
                if (b < 0) {
                    if (live) ok = add_o();
                    break;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->item_empty[slot_i]);
                if (!(ok = twait(&sh->q_full[k & 1], (k >> 1) & 1) && twait(&sh->ext_full[k & 1], (k >> 1) & 1))) break;
                constexpr uint32_t idesc = tc::idesc_bf16(kBK, N, false);
#pragma unroll 1
                for (int j = 0; j < n; ++j) {
                    const uint32_t buf = g & 1, ph = (g >> 1) & 1;
                    if (!(ok = twait(&sh->k_full[buf], ph) && twait(&sh->s_empty[buf], ph ^ 1))) break;
                    tc::fence_after();
                    if (leader) {
                        const uint64_t dq = desc_q + (uint64_t)((k & 1) * (kQTile<D> >> 4));
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc::mma_bf16_ts(tbase + kTColS + buf * kN, tbase + kTColK + buf * kTColsK + kk * 8,
                                            dq + (uint64_t)((kk >> 2) * (kQBox >> 4) + (kk & 3) * 2), idesc, kk > 0 ? 1u : 0u);
                        tc::mma_bf16_ts(tbase + kTColS + buf * kN, tbase + kTColK + buf * kTColsK + D / 2,
                                        desc_x + (uint64_t)(((k & 1) * 2 + buf) * 2), idesc, 1u);
                        tc::commit(&sh->s_full[buf]);
                        tc::commit(&sh->k_empty[buf]);
                        if (j == n - 1) tc::commit(&sh->q_empty[k & 1]);
                    }
                    __syncwarp();
                    if (live && !(ok = add_o())) break;
                    live = true;
                    first = j < 2;
                    end = j >= n - 2;
                    ++g;
                }
            }
            if (!ok) fail();
            // every product issued is complete before the tensor memory is given back
            if (leader) tc::commit(&sh->fin);
            __syncwarp();
            twait(&sh->fin, 0);
        } else {
            // ===================== the work list (warp 14), then seq_status (both)
            if (warp == 14) {
                uint32_t k = 0;
                RowsItem it;
                bool ok = aligned;
                do {
                    next_item(p, walk, it);
                    const int slot_i = k % kItems;
                    if (!(ok = twait(&sh->item_empty[slot_i], ((k / kItems) & 1) ^ 1) && !__shfl_sync(0xffffffffu, *abort_flag, 0))) break;
                    if (lane == 0) {
                        sh->items[slot_i] = it;
                        mbar_arrive(&sh->item_full[slot_i]);
                    }
                    __syncwarp();
                    ++k;
                } while (it.b >= 0);
                if (!ok) fail();
            }
            if (warp == 15) {  // the columns' sums of Q, two columns a lane; a group's u is 0 to begin with
                bool ok = aligned;
#pragma unroll 1
                for (uint32_t k = 0; ok; ++k) {
                    const int slot_i = k % kItems;
                    if (!(ok = twait(&sh->item_full[slot_i], (k / kItems) & 1))) break;
                    const int b = sh->items[slot_i].b;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh->item_empty[slot_i]);
                    if (b < 0) break;
                    if (!(ok = twait(&sh->q_full[k & 1], (k >> 1) & 1))) break;
                    const uint8_t *q = qbuf + (k & 1) * kQTile<D>;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int c = lane + 32 * h;
                        float2 sum = make_float2(0.f, 0.f);
#pragma unroll 4
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(q + (i >> 3) * kQBox + t_sw128(c, i & 7));
                            sum = __fadd2_rn(sum, __fadd2_rn(__fadd2_rn(make_float2(bf16_lo(x.x), bf16_hi(x.x)), make_float2(bf16_lo(x.y), bf16_hi(x.y))),
                                                             __fadd2_rn(make_float2(bf16_lo(x.z), bf16_hi(x.z)), make_float2(bf16_lo(x.w), bf16_hi(x.w)))));
                        }
                        const uint4 y = parts3<false>(sum.x + sum.y);
#pragma unroll
                        for (int group = 0; group < 2; ++group) {
                            *reinterpret_cast<uint4 *>(ext + t_sw128(c, ((k & 1) * 2 + group) * 2)) = y;
                            *reinterpret_cast<uint4 *>(ext + t_sw128(c, ((k & 1) * 2 + group) * 2 + 1)) = make_uint4(0, 0, 0, 0);
                        }
                    }
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sh->ext_full[k & 1]);
                        mbar_arrive(&sh->q_empty[k & 1]);
                    }
                }
                if (!ok) fail();
            }
            const int own = p.seq_status ? (int)blockIdx.x * 2 + warp - 14 : p.B;
#pragma unroll 1
            for (int sb = own; sb < p.B; sb += (int)gridDim.x * 2) {
                const bool bad = bad_sequence(p, sb, lane);
                if (lane == 0) p.seq_status[sb] = bad ? SV_ERR_BAD_INPUT : SV_OK;
            }
            if (lane == 0 && own < p.B && gave_up(p.call))
#pragma unroll 1
                for (int sb = own; sb < p.B; sb += (int)gridDim.x * 2) p.seq_status[sb] = SV_ERR_TIMEOUT;
            // the next call's counters, whose grid may be another
            if (warp == 15)
                for (int c = blockIdx.x * 32 + lane; c < kRowsMaxGrid; c += gridDim.x * 32) {
                    p.counters[rows_counter(sh->call + 1, c)] = 0;
                    p.counters[rows_counter(sh->call + 1, c) + 1] = 0;
                }
        }
    }
    tc::fence_before();
    __syncthreads();
    if (warp == 13) {
        tc::fence_after();
        tc::tmem_dealloc(tbase, kTCols);
    }
    if (tid == 0 && *abort_flag) give_up(p.call, p.seq_status, p.B);
}

const void *quant_kernel_fn(int D, int chunks) {
    switch (chunks) {
        case 2: return D == 128 ? reinterpret_cast<const void *>(&quant_tc_kernel<128, 2>) : reinterpret_cast<const void *>(&quant_tc_kernel<64, 2>);
        case 3: return D == 128 ? reinterpret_cast<const void *>(&quant_tc_kernel<128, 3>) : reinterpret_cast<const void *>(&quant_tc_kernel<64, 3>);
        default: return D == 128 ? reinterpret_cast<const void *>(&quant_tc_kernel<128, 4>) : reinterpret_cast<const void *>(&quant_tc_kernel<64, 4>);
    }
}

int quant_smem_bytes(int D) { return D == 128 ? kTSmem<128> : kTSmem<64>; }

}  // namespace chunk
}  // namespace sv
