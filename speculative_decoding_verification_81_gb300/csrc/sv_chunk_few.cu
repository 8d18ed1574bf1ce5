// sv_chunk_few.cu -- the chunk attention's form for few rows: one request or a
// handful generating, the last tokens of a prompt.
//
// Row r of sequence b is at position p = L_b + r - (b's first row) and sees
// the slots max(0, p - window + 1) .. p.  A cluster of C CTAs takes one row
// and one KV head, whose G = Hq/Hkv <= 8 query heads share K/V: its warps take
// units of 16 consecutive slots in turn,
//     S = scale log2 e K Q^T   (16 slots x 8 heads)
//     P = 2^(S - m), rounded to bf16; l += sum of the f32 P
//     O^T += V^T P             (D dims x 8 heads)
// with a head's running maximum m that moves only when it grows by more than
// 2^8, the sums in registers; then the CTA's warps meet in its shared memory and
// the CTAs in that of the one which owns a slice of the row's values, always in
// the same order.
//
// Why a second form: such a call costs the chain of latencies between its start
// and its last store.  The other form (sv_chunk_tc.cu) passes a tile of 128
// slots through tensor memory and three warps and merges cut items through L2;
// 128-row products have no use here, where 8 rows are all that share a slot.
// The warp's own products of 16 x 8 take K from shared memory as it lies there
// (which of its dims a column is does not matter as long as Q's are taken alike)
// and V with two slots' words exchanged, so nothing is transposed but P, a
// register.  Each half unit's K and V are one copy each (a page holds whole
// halves), all units of a warp or two of them on their way at once.
//
// Measured with K/V from HBM (32 query over 8 KV heads of 128, this form against
// the other): one token after 511 slots 5.0 us against 10.1, after 2047 6.3
// against 13.7, after 8191 12.4 against 18.4; 4 tokens after 2047 9.7 against
// 17.1; 16 rows of a chunk after 900 11.7 against 14.3.  What bounds it: the
// loads before the first K/V (lengths and pages at once, on the guess that
// sequence r has row r: 0.3 us less), the copies' latency, the CTAs' meeting
// (shares sent with their bytes counted at the receiver: 0.1 to 0.3 us less than a
// barrier of the cluster); from about 256 slots a CTA on, what one SM draws from
// HBM and reads from shared memory, 67 GB/s (60 with bank conflicts in the reads of
// K and V, 43 with loads of 16 bytes a lane in place of the copies).
// Tried before: the products by f32 pairs on the ordinary cores (after 8191 slots
// 15.7 us from L2 against 12.5); 4 warps a CTA (after 511 0.1 us less, after 8191
// 3 us more); rows a little apart in shared memory, a copy each, against the bank
// conflicts (after 511 0.3 us more, after 8191 3: 32 copies a unit for 4).
#include <mutex>

#include "sv_chunk.cuh"

namespace sv {
namespace chunk {

namespace {

constexpr int kFewWarps = 8, kFewThreads = 32 * kFewWarps;
constexpr int kUnit = 16, kHalf = 8;               // slots of a unit; a page holds whole halves
constexpr int kFewSlots = 32 * kFewWarps * kUnit;  // slots a CTA takes at most, of a single row: a lane a unit
constexpr int kFewUneven = 1152;                   // and of several: 1024, and 128 for the pages that a table has to spare
constexpr int kFewCluster = 16;
constexpr int kGMax = 8;
template <int D>
constexpr int kUnitBytes = kUnit * D * 4;  // K and V
template <int D>
constexpr int kFewDepth = 128 * 1024 / (kFewWarps * kUnitBytes<D>);  // units of a warp on their way
template <int D>
constexpr int kRingBytes = kFewWarps * kFewDepth<D> * kUnitBytes<D>;

__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
    uint4 x;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "r"(a)
                 : "memory");
    return x;
}

// D (16 x 8, f32) += A (16 x 16) B (16 x 8) of bf16, the warp's fragments: with
// g = lane / 4 and t = lane % 4, a[0..3] hold A at rows g, g + 8, g, g + 8 and
// columns 2t, 2t + 1 (the last two 8 further), b[0..1] B at rows 2t, 2t + 1 and 8
// further, column g, and d[0..3] D at (g, 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1).
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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

// Two floats to another CTA of the cluster; their bytes counted on its barrier.
__device__ __forceinline__ void send_f2(uint32_t to, float2 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to), "f"(v.x),
                 "f"(v.y), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ uint2 ld_shared8(uint32_t a) {
    uint2 x;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x.x), "=r"(x.y) : "r"(a) : "memory");
    return x;
}

__device__ __forceinline__ void swap_if(bool yes, uint2 &a, uint2 &b) {
    const uint2 x = a;
    a = make_uint2(yes ? b.x : a.x, yes ? b.y : a.y);
    b = make_uint2(yes ? x.x : b.x, yes ? x.y : b.y);
}
__device__ __forceinline__ void swap_if(bool yes, uint4 &a, uint4 &b) {
    const uint4 x = a;
    a = make_uint4(yes ? b.x : a.x, yes ? b.y : a.y, yes ? b.z : a.z, yes ? b.w : a.w);
    b = make_uint4(yes ? x.x : b.x, yes ? x.y : b.y, yes ? x.z : b.z, yes ? x.w : b.w);
}

}  // namespace

template <int D>
__global__ void __launch_bounds__(kFewThreads, 1) chunk_few_kernel(const FewParams p) {
    constexpr int kK = D / 32;  // 16-byte pieces of a K (or Q) row a lane: piece 4 i + t
    constexpr int kV = D / 32;  // 8-byte pieces of a V row a lane: piece kV g + i
    constexpr int kDepth = kFewDepth<D>;
    // [warp][unit][K, V][slot][D]; a warp's O [8][D] takes the place of its first unit when it has read its last
    extern __shared__ __align__(16) uint8_t ring[];
    auto warp_o = [&](int w) { return reinterpret_cast<float *>(ring + w * kDepth * kUnitBytes<D>); };
    __shared__ uint64_t full[kFewWarps][kDepth], joined;
    __shared__ float2 warp_ml[kFewWarps][kGMax];
    __shared__ __align__(16) float part[kGMax * D];  // [CTA of the cluster][this CTA's slice]
    __shared__ float2 ml[kFewCluster][kGMax];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int G = p.c.G, C = p.cluster, rank = (int)cluster_ctarank(), pair = (int)blockIdx.x / C;
    const int row = pair / p.c.Hkv, h = pair - row * p.c.Hkv;
    const Shape &shape = p.c.shape;
    const int pairs = G * D / 2, slice = pairs / C;  // pairs of values: a multiple of 32
    if (lane < kDepth) mbar_init(&full[warp][lane], 1);
    if (tid == 0) mbar_init(&joined, 1);
    fence_mbar_init();
    if (tid == 0) mbar_arrive_expect_tx(&joined, (uint32_t)(C * (slice + kGMax) * sizeof(float2)));
    __syncwarp();
    cluster_arrive_relaxed();  // (waited for before the first store to another CTA)
    griddep_wait();
    griddep_launch_dependents();

    // the lengths, a lane a sequence; query head g of the row; and this warp's pages (a lane a
    // unit), on the guess that sequence `row` has one row, so that their load need not wait
    int L = 0, r0 = 0, r1 = 0;
    if (lane < p.c.B) {
        L = p.c.prefix_lens[lane];
        r0 = p.c.row_starts[lane];
        r1 = p.c.row_starts[lane + 1];
    }
    const uint4 none = make_uint4(0, 0, 0, 0);
    uint4 q[kK];
#pragma unroll
    for (int i = 0; i < kK; ++i)
        q[i] = g < G ? ldg_stream(p.q + (size_t)row * p.q_stride + (size_t)(h * G + g) * D + (4 * i + t) * 8) : none;
    const int step = C * kFewWarps, guess = min(row, p.c.B - 1);
    int pages[2] = {-1, -1};
    auto load_pages = [&](int b, int first, int lo, int pos) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int slot = (first + lane * step) * kUnit + x * kHalf;
            if (slot + kHalf > lo && slot <= pos)
                pages[x] = p.c.block_table[(size_t)b * p.c.max_pages + slot / p.c.page_size];
        }
    };
    if (shape.window == 0) load_pages(guess, rank * kFewWarps + warp, 0, shape.S_max - 1);
    const bool ok = lane < p.c.B && lengths_ok(shape, L, r0, r1);
    const uint32_t mine = __ballot_sync(0xffffffffu, ok && r0 <= row && row < r1);
    // the sequences whose status this warp writes: one a warp, of each CTA the last warps first,
    // which have no part in the end where a CTA's slice is short
    const int own = p.c.seq_status ? (kFewWarps - 1 - warp) * (int)gridDim.x + (int)blockIdx.x : p.c.B;
    bool looked = own >= p.c.B;
    auto look = [&] {  // (once, at any time after the report)
        if (looked) return;
        looked = true;
        if (lane == 0 && gave_up(p.c.call))
            for (int sb = own; sb < p.c.B; sb += (int)gridDim.x * kFewWarps) p.c.seq_status[sb] = SV_ERR_TIMEOUT;
        __syncwarp();
    };
    bool lost = false;
    {  // (a row of no sequence has no units)
        const int b = max(__ffs(mine) - 1, 0);
        const int ahead = __shfl_sync(0xffffffffu, L, b), begin = __shfl_sync(0xffffffffu, r0, b);
        const int pos = mine != 0 ? ahead + row - begin : 0;
        const int lo = shape.window > 0 ? max(0, pos - shape.window + 1) : 0;
        // this warp's units, and the cache row of each half's first slot (-1: nothing to read)
        const int first = lo / kUnit + rank * kFewWarps + warp, last = pos / kUnit;
        const int n = mine != 0 && first <= last ? (last - first) / step + 1 : 0;
        if (mine != 0 && (shape.window != 0 || b != guess)) load_pages(b, first, lo, pos);
        int at[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int slot = (first + lane * step) * kUnit + x * kHalf;
            const bool on = lane < n && slot + kHalf > lo && slot <= pos && pages[x] >= 0 && pages[x] < p.c.num_pages;
            at[x] = on ? (pages[x] * p.c.Hkv + h) * p.c.page_size + slot % p.c.page_size : -1;
        }
        uint8_t *const units = ring + warp * kDepth * kUnitBytes<D>;
        auto fetch = [&](int i, int st) {
            const int a0 = __shfl_sync(0xffffffffu, at[0], i), a1 = __shfl_sync(0xffffffffu, at[1], i);
            if (lane == 0) {
                constexpr uint32_t kB = kHalf * D * 2;
                uint8_t *to = units + st * kUnitBytes<D>;
                mbar_arrive_expect_tx(&full[warp][st], ((a0 >= 0) + (a1 >= 0)) * 2 * kB);
                if (a0 >= 0) {
                    bulk_load(to, p.k + (size_t)a0 * D, kB, &full[warp][st]);
                    bulk_load(to + 2 * kB, p.v + (size_t)a0 * D, kB, &full[warp][st]);
                }
                if (a1 >= 0) {
                    bulk_load(to + kB, p.k + (size_t)a1 * D, kB, &full[warp][st]);
                    bulk_load(to + 3 * kB, p.v + (size_t)a1 * D, kB, &full[warp][st]);
                }
            }
        };
#pragma unroll 1
        for (int i = 0; i < kDepth; ++i)
            if (i < n) fetch(i, i);
        // while the copies are on their way, seq_status: lengths, and the ids of the pages that rows see
        if (tid == kFewThreads - 32) begin_call(p.c.call);  // (the thread that may look for its call first)
        for (int sb = own; sb < p.c.B; sb += (int)gridDim.x * kFewWarps) {
            const int rows = __shfl_sync(0xffffffffu, r1 - r0, sb), Ls = __shfl_sync(0xffffffffu, L, sb);
            bool bad = !__shfl_sync(0xffffffffu, (int)ok, sb);
            if (!bad && rows > 0) {
                const int from = shape.window > 0 ? max(0, Ls - shape.window + 1) : 0;
                const int32_t *trow = p.c.block_table + (size_t)sb * p.c.max_pages;
                for (int j = from / p.c.page_size + lane; j <= (Ls + rows - 1) / p.c.page_size; j += 32) {
                    const int pg = trow[j];
                    if (pg < 0 || pg >= p.c.num_pages) bad = true;
                }
            }
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) p.c.seq_status[sb] = bad ? SV_ERR_BAD_INPUT : SV_OK;
        }
        __syncwarp();
        if (n == 0 && warp == kFewWarps - 1) look();
        int st = 0, ph = 0;
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};  // heads 2t and 2t + 1 (l: this lane's slots)
        float o[2 * kV][4];  // [i]: dims 4 kV g + 2 i and the next, heads 2t and 2t + 1 each
#pragma unroll
        for (int i = 0; i < 2 * kV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if (!warp_wait_bounded(&full[warp][st], ph)) {
                lost = true;
                for (int k = i; k < min(n, i + kDepth); ++k) {  // its own copies still on their way, this one too
                    warp_wait_bounded(&full[warp][st], ph);
                    if (++st == kDepth) st = 0, ph ^= 1;
                }
                break;
            }
            const uint32_t here = smem_u32(units) + (uint32_t)(st * kUnitBytes<D>);
            const int slot0 = (first + i * step) * kUnit;
            const bool whole = slot0 >= lo && slot0 + kUnit - 1 <= pos;
            float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < kK; c += 2) {
                // odd rows read the two pieces in the other order: eight lanes of a read (two
                // rows, four pieces) then meet eight bank groups
                const uint32_t at_k = here + g * (D * 2) + (4 * c + t) * 16, odd = g & 1 ? 64 : 0;
                uint4 a0 = ld_shared16(at_k + odd), a1 = ld_shared16(at_k + (odd ^ 64));
                uint4 b0 = ld_shared16(at_k + kHalf * D * 2 + odd), b1 = ld_shared16(at_k + kHalf * D * 2 + (odd ^ 64));
                swap_if(odd != 0, a0, a1);
                swap_if(odd != 0, b0, b1);
                mma16(s, a0.x, b0.x, a0.y, b0.y, q[c].x, q[c].y);
                mma16(s, a0.z, b0.z, a0.w, b0.w, q[c].z, q[c].w);
                mma16(s, a1.x, b1.x, a1.y, b1.y, q[c + 1].x, q[c + 1].y);
                mma16(s, a1.z, b1.z, a1.w, b1.w, q[c + 1].z, q[c + 1].w);
            }
            const int slot = (first + i * step) * kUnit + g;
            const bool see0 = slot >= lo && slot <= pos, see1 = slot + 8 >= lo && slot + 8 <= pos;
            float f[2], e[2][2];
            bool moved = false;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float s0 = see0 ? s[j] * p.c.scale_log2 : kNegInf;
                const float s1 = see1 ? s[2 + j] * p.c.scale_log2 : kNegInf;
                float c = fmaxf(s0, s1);
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) c = fmaxf(c, __shfl_xor_sync(0xffffffffu, c, off));
                const bool up = c > m[j] + kRescaleThreshold;
                f[j] = up ? ex2_approx(m[j] - c) : 1.f;
                if (up) m[j] = c;
                moved = moved || up;
                const float base = m[j] == kNegInf ? 0.f : m[j];
                e[0][j] = ex2_approx(s0 - base);
                e[1][j] = ex2_approx(s1 - base);
                l[j] = l[j] * f[j] + (e[0][j] + e[1][j]);
            }
            if (__any_sync(0xffffffffu, moved) && i > 0) {
#pragma unroll
                for (int x = 0; x < 2 * kV; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[x][y] *= f[y & 1];
            }
            const uint32_t p0 = transposed(pack_bf16x2(e[0][0], e[0][1]));
            const uint32_t p1 = transposed(pack_bf16x2(e[1][0], e[1][1]));
            // a slot's pieces in an order by t, so that the four rows of a read meet other bank groups
            // (sixteen lanes: four rows, four pieces each of a lane's kV), then put right
            uint2 v[4][kV];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int sl = 2 * t + (y & 1) + (y >> 1) * 8;
                const uint32_t at_v = here + kUnitBytes<D> / 2 + sl * (D * 2) + kV * g * 8;
                const bool on = whole || (slot0 + sl >= lo && slot0 + sl <= pos);
#pragma unroll
                for (int c = 0; c < kV; ++c) {
                    v[y][c] = ld_shared8(at_v + (c ^ (t & (kV - 1))) * 8);
                    if (!on) v[y][c] = make_uint2(0, 0);
                }
                if constexpr (kV == 4) {
                    swap_if(t & 2, v[y][0], v[y][2]);
                    swap_if(t & 2, v[y][1], v[y][3]);
                    swap_if(t & 1, v[y][2], v[y][3]);
                }
                swap_if(t & 1, v[y][0], v[y][1]);
            }
#pragma unroll
            for (int c = 0; c < kV; ++c) {
                // even dims as rows g, odd ones as rows g + 8; two slots a word
                mma16(o[2 * c], __byte_perm(v[0][c].x, v[1][c].x, 0x5410), __byte_perm(v[0][c].x, v[1][c].x, 0x7632),
                      __byte_perm(v[2][c].x, v[3][c].x, 0x5410), __byte_perm(v[2][c].x, v[3][c].x, 0x7632), p0, p1);
                mma16(o[2 * c + 1], __byte_perm(v[0][c].y, v[1][c].y, 0x5410), __byte_perm(v[0][c].y, v[1][c].y, 0x7632),
                      __byte_perm(v[2][c].y, v[3][c].y, 0x5410), __byte_perm(v[2][c].y, v[3][c].y, 0x7632), p0, p1);
            }
            __syncwarp();
            if (i + kDepth < n) fetch(i + kDepth, st);
            if (++st == kDepth) st = 0, ph ^= 1;
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);
            if (lane < 4) warp_ml[warp][2 * t + j] = make_float2(m[j], l[j]);
            if (2 * t + j < G) {
#pragma unroll
                for (int c = 0; c < kV; ++c) {
                    *reinterpret_cast<float4 *>(warp_o(warp) + (2 * t + j) * D + 4 * (kV * g + c)) =
                        make_float4(o[2 * c][j], o[2 * c][2 + j], o[2 * c + 1][j], o[2 * c + 1][2 + j]);
                }
            }
        }
    }
    __syncthreads();
    cluster_wait();
    if (mine != 0) {
        // the CTA's sums, each to the CTA that owns it
        for (int x = tid; x < pairs; x += kFewThreads) {
            const int hd = 2 * x / D;
            float M = kNegInf;
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kFewWarps; ++i) M = fmaxf(M, warp_ml[i][hd].x);
#pragma unroll
            for (int i = 0; i < kFewWarps; ++i) {
                const float mi = warp_ml[i][hd].x, w = mi == kNegInf ? 0.f : ex2_approx(mi - M);
                const float2 v = reinterpret_cast<const float2 *>(warp_o(i))[x];
                acc.x = __fmaf_rn(v.x, w, acc.x);
                acc.y = __fmaf_rn(v.y, w, acc.y);
            }
            const int owner = x / slice;
            send_f2(cluster_map(smem_u32(&part[2 * (rank * slice + x - owner * slice)]), (uint32_t)owner), acc,
                    cluster_map(smem_u32(&joined), (uint32_t)owner));
        }
        if (tid < kGMax * C) {
            const int hd = tid % kGMax, dst = tid / kGMax;
            float M = kNegInf, sum = 0.f;
#pragma unroll
            for (int i = 0; i < kFewWarps; ++i) M = fmaxf(M, warp_ml[i][hd].x);
#pragma unroll
            for (int i = 0; i < kFewWarps; ++i) {
                const float2 x = warp_ml[i][hd];
                sum = __fmaf_rn(x.y, x.x == kNegInf ? 0.f : ex2_approx(x.x - M), sum);  // (a sum of NaN goes on)
            }
            send_f2(cluster_map(smem_u32(&ml[rank][hd]), (uint32_t)dst), make_float2(M, sum),
                    cluster_map(smem_u32(&joined), (uint32_t)dst));
        }
    }
    look();
    __syncwarp();
    bool late = false;
    if (mine != 0) {
        late = !warp_wait_bounded(&joined, 0);
        lost = lost || late;
        if (lost && lane == 0) give_up(p.c.call, p.c.seq_status, p.c.B);
        // the cluster's sums of this CTA's slice
        for (int x = tid; x < slice; x += kFewThreads) {
            const int at = rank * slice + x, hd = 2 * at / D, dim = 2 * at - hd * D;
            float M = kNegInf, sum = 0.f;
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int c = 0; c < C; ++c) M = fmaxf(M, ml[c][hd].x);
#pragma unroll 4
            for (int c = 0; c < C; ++c) {
                const float2 y = ml[c][hd], v = reinterpret_cast<const float2 *>(part)[c * slice + x];
                const float w = y.x == kNegInf ? 0.f : ex2_approx(y.x - M);
                sum = __fmaf_rn(y.y, w, sum);
                acc.x = __fmaf_rn(v.x, w, acc.x);
                acc.y = __fmaf_rn(v.y, w, acc.y);
            }
            const float inv = 1.f / sum;  // (a row sees its own slot: 0 or NaN only where its scores are not finite)
            const long long head = (long long)row * p.c.Hq + h * G + hd;
            reinterpret_cast<uint32_t *>(p.c.out)[(head * D + dim) / 2] = pack_bf16x2(acc.x * inv, acc.y * inv);
            if (p.c.lse && dim == 0) p.c.lse[head] = M * kLn2 + logf(sum);
        }
    }
    // A CTA that lost a copy sends some bounded waits after the others began to wait for its
    // shares, and a store to a CTA that has left is undefined.  Every CTA leaves after its own
    // sends; one with all shares needs no more, and one that gave up waits until each of the
    // others has left or stands here too (exited threads count as arrived), then for the shares
    // to land.  (Such a barrier for every call: one token after 511 slots 5.0 -> 5.3 us.)
    if (late) {
        cluster_sync_any();
        warp_wait_bounded(&joined, 0);
    }
}

namespace {

int few_smem(int D) { return D == 128 ? kRingBytes<128> : kRingBytes<64>; }

const void *few_fn(int D) {
    return D == 128 ? reinterpret_cast<const void *>(&chunk_few_kernel<128>)
                    : reinterpret_cast<const void *>(&chunk_few_kernel<64>);
}

// Clusters of 2^i CTAs that the current device holds at once, asked for once a
// device; zeros where the kernel does not run.
struct Capacity {
    int n[5];
};
static_assert(kFewCluster == 1 << 4, "sizes of clusters");

Capacity few_capacity(int D) {
    struct Entry {
        int dev, D;
        Capacity c;
    };
    static std::mutex mu;
    static Entry cache[64];
    static int ncache = 0;
    int dev = 0;
    Capacity c{};
    if (cudaGetDevice(&dev) != cudaSuccess) return c;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < ncache; ++i)
        if (cache[i].dev == dev && cache[i].D == D) return cache[i].c;
    const void *fn = few_fn(D);
    const bool smem_ok = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, few_smem(D)) == cudaSuccess;
    const bool large_ok = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (int i = 0; smem_ok && i < (large_ok ? 5 : 4); ++i) {
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1u << i;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1u << i);
        cfg.blockDim = dim3(kFewThreads);
        cfg.dynamicSmemBytes = (size_t)few_smem(D);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&c.n[i], fn, &cfg) != cudaSuccess) c.n[i] = 0;
    }
    cudaGetLastError();  // (a refused query leaves no error behind)
    if (ncache < 64) cache[ncache++] = Entry{dev, D, c};
    return c;
}

}  // namespace

// The smallest cluster whose warps have a unit each at most (one token after 511
// slots: 4 CTAs 4.9 us, 8 5.1, 2 6.2), or the largest of which the rows and
// KV heads all find room at once.  A CTA then takes up to 4096 slots of a single
// row (after 16383 slots 20.1 us against 25.1 for the other form, after 30000 32.7
// against 34.9; 8 query heads over 1 KV head, after 30000: 18.4 against 41); of
// several rows 1152, since theirs may be uneven, which the other form's list
// evens out (8 tokens after 2047 each: 14.7 us against 22.9; one after 2047 among
// short ones: as long here, 13.7 there).  Lengths are on the device: the table's
// width stands for them, so that short rows over a wider table take the other
// form too (4 tokens after 511 slots 10.6 us for 5.4).
int few_cluster(const ChunkArgs &a) {
    if (a.Hq / a.Hkv > kGMax || a.B > 32) return 0;
    const long long pairs = (long long)a.num_rows * a.Hkv, table = (long long)a.max_pages * a.page_size;
    // (a window's first and last unit are seen in part)
    const long long slots = a.window > 0 && a.window + 2LL * kUnit < table ? a.window + 2LL * kUnit : table;
    const Capacity room = few_capacity(a.D);
    int best = 0;
    for (int i = 0; i < 5 && room.n[i] >= pairs; ++i) {
        best = 1 << i;
        if (slots <= (long long)best * kFewWarps * kUnit) break;
    }
    return slots <= (long long)best * (a.num_rows == 1 ? kFewSlots : kFewUneven) ? best : 0;
}

sv_status launch_few(const ChunkArgs &a, const Params &c, int cluster, cudaStream_t st) {
    FewParams p{};
    p.c = c;
    p.q = static_cast<const uint16_t *>(a.q);
    p.k = static_cast<const uint16_t *>(a.k_pages);
    p.v = static_cast<const uint16_t *>(a.v_pages);
    p.q_stride = a.q_stride;
    p.cluster = cluster;
    void *args[] = {&p};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.num_rows * a.Hkv * cluster));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = (size_t)few_smem(a.D);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, few_fn(a.D), args) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace chunk
}  // namespace sv
