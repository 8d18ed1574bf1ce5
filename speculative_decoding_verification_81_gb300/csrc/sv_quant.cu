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

// The codes (a word) and the parameters (a word) of eight values of a row whose
// L lanes hold the others; by the whole warp.  The arithmetic is the header's,
// rounding by rounding, so that a row has one encoding wherever it is made.
template <int L>
__device__ __forceinline__ uint2 encode(const float (&v)[8], int lane) {
    float lo = v[0], hi = v[0], nan = v[0] * 0.f;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
        nan = __fmaf_rn(v[i], 0.f, nan);  // (0 unless some value is not finite)
    }
#pragma unroll
    for (int off = 1; off < L; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    const uint32_t group = (L == 32 ? 0xffffffffu : (1u << L) - 1u) << (lane & ~(L - 1));
    const uint32_t word = pack_bf16x2(__fmul_rn(__fsub_rn(hi, lo), quant::kFifteenth), lo);  // (step, minimum)
    const float step = bf16_lo(word), base = bf16_hi(word);
    // (a step or minimum past bf16's range too has no encoding)
    const bool odd = nan != 0.f || !(step < __builtin_huge_valf()) || !(fabsf(base) < __builtin_huge_valf());
    if ((__ballot_sync(0xffffffffu, odd) & group) != 0) return make_uint2(0u, quant::kNotFinite);
    if (step < quant::kSmallestStep) return make_uint2(0u, word & 0xffff0000u);
    const float inv = __frcp_rn(step);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = __fmul_rn(__fsub_rn(v[i], base), inv);
        c[i] = (uint32_t)__float2int_rn(fminf(fmaxf(f, 0.f), 15.f));
    }
    return make_uint2(quant::pack(c), word);
}

// A thread takes eight dims of a row's head, of K and of V; the lanes of a head
// lie side by side.  The padding lanes of the last warp take part in the votes.
template <int D, bool F32>
__global__ void __launch_bounds__(kQT) append_quant_kernel(const AppendQuantArgs a) {
    constexpr int kL = D / 8;  // lanes of a head's row
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long vpr = (long long)a.Hkv * kL, total = (long long)a.num_rows * vpr;
    const long long i = (long long)blockIdx.x * kQT + threadIdx.x;
    const long long row = total >> 32 ? i / vpr : (long long)((uint32_t)i / (uint32_t)vpr);
    const int piece = (int)(i - row * vpr), h = piece / kL, w = piece % kL;
    const int slots = a.num_pages * a.page_size;
    int slot = -1;
    if (i < total) {
        slot = a.slot_map[row];
        if (piece == 0 && a.row_status) a.row_status[row] = slot >= -1 && slot < slots ? SV_OK : SV_ERR_BAD_INPUT;
    }
    const bool on = slot >= 0 && slot < slots;
    Piece<F32> k{}, v{};
    if (on) {
        k.load(a.k_new, (size_t)(row * a.k_stride) + (size_t)piece * 8);
        v.load(a.v_new, (size_t)(row * a.v_stride) + (size_t)piece * 8);
    }
    float x[8];
    k.values(x);
    const uint2 kq = encode<kL>(x, lane);
    v.values(x);
    const uint2 vq = encode<kL>(x, lane);
    if (!on) return;
    const int pg = slot / a.page_size, off = slot - pg * a.page_size;
    const size_t at = ((size_t)pg * a.Hkv + h) * a.page_size + off;
    static_cast<uint32_t *>(a.k_codes)[at * kL + w] = kq.x;
    static_cast<uint32_t *>(a.v_codes)[at * kL + w] = vq.x;
    if (w == 0) {
        static_cast<uint32_t *>(a.k_params)[at] = kq.y;
        static_cast<uint32_t *>(a.v_params)[at] = vq.y;
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
    const long long total = (long long)a.num_rows * a.Hkv * (a.D / 8);
    const long long grid = (total + kQT - 1) / kQT;
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
