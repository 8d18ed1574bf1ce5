// sv_quant.cu -- a paged KV cache held in 4 bits: new K/V rows quantised into
// the pages through a slot map, and the rows of an accepted path moved together.
//
// The paged KV of "Chapitre 9", section "Ce que prépare le Chapitre 9", and
// §9.1 (a step appends its candidates' rows and keeps a prefix of them).  A row
// of a slot and KV head is D codes of 4 bits and two bf16 numbers, the step
// between codes and the row's minimum (sv_quant.cuh): D / 2 + 4 bytes for 2 D.
#include "sv_quant.cuh"

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kQT = 256;

// Eight values of a row, as floats.
template <bool F32>
struct Piece {
    uint4 x[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *src, size_t elem) {
        if constexpr (F32) {
            const float *f = static_cast<const float *>(src) + elem;
            x[0] = ldg_stream(f);
            x[1] = ldg_stream(f + 4);
        } else {
            x[0] = ldg_stream(static_cast<const uint16_t *>(src) + elem);
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if constexpr (F32) {
            const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
        } else {
            const uint32_t w[4] = {x[0].x, x[0].y, x[0].z, x[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_lo(w[i]);
                v[2 * i + 1] = bf16_hi(w[i]);
            }
        }
    }
};

__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint32_t times_zero_bf16x2(uint32_t x, uint32_t add) {
    uint32_t y;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(0u), "r"(add));
    return y;
}

// The lowest and highest of a lane's values of a row whose L lanes hold the others (over all of them), and
// whether one of its own is not finite.
template <int L>
__device__ __forceinline__ bool range_of(const Piece<true> (&p)[2], float &lo, float &hi) {
    float nan = 0.f;
    lo = __builtin_huge_valf();
    hi = -lo;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        float v[8];
        p[k].values(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
            nan = __fmaf_rn(v[i], 0.f, nan);  // (0 unless some value is not finite)
        }
    }
#pragma unroll
    for (int off = 1; off < L; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    return nan != 0.f;
}
// Of bf16 values two at a time, the highest as the lowest of the negated ones, both in one word.
template <int L>
__device__ __forceinline__ bool range_of(const Piece<false> (&p)[2], float &lo, float &hi) {
    constexpr uint32_t kSigns = 0x80008000u;
    uint32_t low = p[0].x[0].x, high = low ^ kSigns, nan = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {p[k].x[0].x, p[k].x[0].y, p[k].x[0].z, p[k].x[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            low = min_bf16x2(low, w[i]);
            high = min_bf16x2(high, w[i] ^ kSigns);
            nan = times_zero_bf16x2(w[i], nan);
        }
    }
    uint32_t m = min_bf16x2(__byte_perm(low, high, 0x5410), __byte_perm(low, high, 0x7632));
#pragma unroll
    for (int off = 1; off < L; off <<= 1) m = min_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, off));
    lo = bf16_lo(m);
    hi = -bf16_hi(m);
    return (nan & ~kSigns) != 0;
}

// The codes (two words) and the parameters (a word) of a lane's two pieces of a row
// whose L lanes hold the others; by the whole warp.  The arithmetic is the header's,
// rounding by rounding, so that a row has one encoding wherever it is made.
struct Encoded {
    uint32_t codes[2], params;
};
template <int L, bool F32>
__device__ __forceinline__ Encoded encode(const Piece<F32> (&p)[2], int lane) {
    float lo, hi;
    const bool nan = range_of<L>(p, lo, hi);
    const uint32_t group = ((1u << L) - 1u) << (lane & ~(L - 1));
    const uint32_t word = pack_bf16x2(__fmul_rn(__fsub_rn(hi, lo), quant::kFifteenth), lo);  // (step, minimum)
    const float step = bf16_lo(word), base = bf16_hi(word);
    // (a step or minimum past bf16's range too has no encoding)
    const bool odd = nan || !(step < __builtin_huge_valf()) || !(fabsf(base) < __builtin_huge_valf());
    if ((__ballot_sync(0xffffffffu, odd) & group) != 0) return Encoded{{0u, 0u}, quant::kNotFinite};
    if (step < quant::kSmallestStep) return Encoded{{0u, 0u}, word & 0xffff0000u};
    const float inv = __frcp_rn(step);
    Encoded e;
    e.params = word;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        // codes as sixteenths, held to 0 .. 15 and rounded (ties to even) by a sum with 3 2^18, and four of them
        // as one number below 2^16: dims 0, 2, 4, 6 and 1, 3, 5, 7
        float v[8], u[2] = {0.f, 0.f};
        p[k].values(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = __fmul_rn(__fsub_rn(v[i], base), inv);
            const float g = fminf(__saturatef(__fmul_rn(f, 0.0625f)), 0.9375f);
            const float c = __fsub_rn(__fadd_rn(g, 786432.f), 786432.f);
            u[i & 1] = __fmaf_rn(c, (float)(16u << 4 * (i >> 1)), u[i & 1]);
        }
        // (in the last bits of 2^23)
        e.codes[k] = __byte_perm(__float_as_uint(u[0] + 8388608.f), __float_as_uint(u[1] + 8388608.f), 0x5410);
    }
    return e;
}

// A thread takes two pieces of eight dims of a row's head, half a row apart, of K and
// of V; the lanes of a head lie side by side.  All of a thread's loads are on their way
// before any is looked at, those of rows that the map leaves out (-1) too.  The padding
// lanes of the last warp take part in the votes.
//
// What bounds it: the instructions, of which a row's place and its range's meeting
// take what eight dims' codes do -- 8192 rows of 8 heads of 128 in 11.1 us, 0.57 of the
// measured bandwidth; eight dims a thread took 13.4, the same two rows a thread 13.9.
template <int D, bool F32>
__global__ void __launch_bounds__(kQT) append_quant_kernel(const AppendQuantArgs a) {
    constexpr int kL = D / 16;  // lanes of a head's row
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long vpr = (long long)a.Hkv * kL, total = (long long)a.num_rows * vpr;
    const int slots = a.num_pages * a.page_size;
    const long long i = (long long)blockIdx.x * kQT + threadIdx.x;
    const long long row = total >> 32 ? i / vpr : (long long)((uint32_t)i / (uint32_t)vpr);
    const int part = (int)(i - row * vpr), h = part / kL, w = part % kL;
    int slot = -1;
    Piece<F32> k[2] = {}, v[2] = {};
    if (i < total) {
        slot = a.slot_map[row];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int at = h * D + (w + p * kL) * 8;
            k[p].load(a.k_new, (size_t)(row * a.k_stride) + at);
            v[p].load(a.v_new, (size_t)(row * a.v_stride) + at);
        }
        if (part == 0 && a.row_status) a.row_status[row] = slot >= -1 && slot < slots ? SV_OK : SV_ERR_BAD_INPUT;
    }
    const Encoded kq = encode<kL>(k, lane), vq = encode<kL>(v, lane);
    if (slot < 0 || slot >= slots) return;
    const int pg = slot / a.page_size, off = slot - pg * a.page_size;
    const size_t at = ((size_t)pg * a.Hkv + h) * a.page_size + off;
    uint32_t *const kc = static_cast<uint32_t *>(a.k_codes) + at * (2 * kL) + w;
    uint32_t *const vc = static_cast<uint32_t *>(a.v_codes) + at * (2 * kL) + w;
    kc[0] = kq.codes[0];
    kc[kL] = kq.codes[1];
    vc[0] = vq.codes[0];
    vc[kL] = vq.codes[1];
    if (w == 0) {
        static_cast<uint32_t *>(a.k_params)[at] = kq.params;
        static_cast<uint32_t *>(a.v_params)[at] = vq.params;
    }
}

constexpr int kMT = 256;
constexpr int kMoveRegs = 4;         // pieces a thread holds in a round
constexpr int kMaxRoundPairs = 256;  // (position, head) pairs of a round

// One CTA a sequence.  The path increases strictly, so that a destination
// L + d is never the source of a later position: rounds of consecutive
// positions (every head), each read as a whole before it is written.
template <int D>
__global__ void __launch_bounds__(kMT) compact_quant_kernel(const CompactQuantArgs a) {
    constexpr int kP = D / 32, kPer = 2 * kP;  // 16-byte pieces of a row's codes; of K and V
    constexpr int kRound = kMT * kMoveRegs / kPer < kMaxRoundPairs ? kMT * kMoveRegs / kPer : kMaxRoundPairs;
    __shared__ size_t s_src[kRound], s_dst[kRound];  // (both at `none`: nothing moves)
    constexpr size_t none = ~(size_t)0;
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x;
    const int L = a.prefix_lens[b], acc = a.accepted_len[b];
    __syncthreads();  // every thread has read L before new_kv_lens (may alias) is written
    if (acc < 0) {
        if (threadIdx.x == 0) {
            a.new_kv_lens[b] = L;
            if (a.seq_status) a.seq_status[b] = SV_OK;
        }
        return;
    }
    const int32_t *path = a.path_nodes ? a.path_nodes + (size_t)b * a.path_stride : nullptr;
    const int32_t *trow = a.block_table + (size_t)b * a.max_pages;
    auto page_ok = [&](int slot) {
        const int pg = trow[slot / a.page_size];
        return pg >= 0 && pg < a.num_pages;
    };
    int bad = L < 0 || (long long)L + acc + 1 > a.S_max || (path && acc >= a.path_stride);
    if (!bad && path) {
        for (int d = threadIdx.x; d <= acc; d += kMT) {
            const int src = path[d];
            // (an increasing path from 0 has path[d] >= d: nothing below is looked up)
            if (d == 0 ? src != 0 : src <= path[d - 1] || src < d) bad = 1;
            if ((long long)L + src >= a.S_max) bad = 1;
            if (!bad && (!page_ok(L + src) || !page_ok(L + d))) bad = 1;
        }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        a.new_kv_lens[b] = bad ? L : L + acc + 1;
        if (a.seq_status) a.seq_status[b] = bad ? SV_ERR_BAD_INPUT : SV_OK;
    }
    if (bad || !path) return;
    auto row_at = [&](int h, int slot) -> size_t {
        const int j = slot / a.page_size;
        return ((size_t)trow[j] * a.Hkv + h) * a.page_size + (slot - j * a.page_size);
    };
    uint4 *codes[2] = {static_cast<uint4 *>(a.k_codes), static_cast<uint4 *>(a.v_codes)};
    uint32_t *params[2] = {static_cast<uint32_t *>(a.k_params), static_cast<uint32_t *>(a.v_params)};
    const int npairs = acc * a.Hkv;  // (the root never moves)
    for (int q0 = 0; q0 < npairs; q0 += kRound) {
        const int np = min(kRound, npairs - q0);
        for (int i = threadIdx.x; i < np; i += kMT) {
            const int d = 1 + (q0 + i) / a.Hkv, h = q0 + i - (d - 1) * a.Hkv, src = path[d];
            s_src[i] = src != d ? row_at(h, L + src) : none;
            s_dst[i] = src != d ? row_at(h, L + d) : none;
        }
        __syncthreads();
        uint4 reg[kMoveRegs];
        uint32_t par[kMoveRegs];
#pragma unroll
        for (int k = 0; k < kMoveRegs; ++k) {
            const int it = threadIdx.x + k * kMT, pr = it / kPer, kv = it / kP & 1, w = it % kP;
            if (pr < np && s_src[pr] != none) {
                reg[k] = codes[kv][s_src[pr] * kP + w];
                if (w == 0) par[k] = params[kv][s_src[pr]];
            }
        }
        __syncthreads();  // every source of the round is read
#pragma unroll
        for (int k = 0; k < kMoveRegs; ++k) {
            const int it = threadIdx.x + k * kMT, pr = it / kPer, kv = it / kP & 1, w = it % kP;
            if (pr < np && s_dst[pr] != none) {
                codes[kv][s_dst[pr] * kP + w] = reg[k];
                if (w == 0) params[kv][s_dst[pr]] = par[k];
            }
        }
        __syncthreads();  // before the next round's places replace these, and its sources are read
    }
}

}  // namespace

sv_status launch_append_quant(const AppendQuantArgs &a, int dtype, cudaStream_t st) {
    AppendQuantArgs ka = a;
    void *args[] = {&ka};
    const void *fn = a.D == 128 ? (dtype == SV_F32 ? (const void *)append_quant_kernel<128, true>
                                                   : (const void *)append_quant_kernel<128, false>)
                                : (dtype == SV_F32 ? (const void *)append_quant_kernel<64, true>
                                                   : (const void *)append_quant_kernel<64, false>);
    const long long grid = ((long long)a.num_rows * a.Hkv * (a.D / 16) + kQT - 1) / kQT;
    if (grid >= (1LL << 31)) return SV_ERR_UNSUPPORTED;
    return launch_pdl(fn, dim3((unsigned)grid), dim3(kQT), 0, st, args) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

sv_status launch_compact_quant(const CompactQuantArgs &a, cudaStream_t st) {
    CompactQuantArgs ka = a;
    void *args[] = {&ka};
    const void *fn = a.D == 128 ? (const void *)compact_quant_kernel<128> : (const void *)compact_quant_kernel<64>;
    return launch_pdl(fn, dim3((unsigned)a.B), dim3(kMT), 0, st, args) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
