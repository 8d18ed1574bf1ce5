// sv_pages.cu -- the bookkeeping of a paged KV cache on the device: page
// tables and slot maps from request lengths, pages given back when a length
// shrinks, and the write of new K/V rows through a slot map.
//
// The paged KV of "Chapitre 9", section "Ce que prépare le Chapitre 9", with
// §9.1 for the lengths: a step appends its candidates' rows and keeps a
// prefix of them, so a sequence's pages grow before the step and its tail's
// pages come back after it.  The pool is a stack of free page ids, handed
// out in sequence order by prefix sums, so that the result does not depend on
// the order in which threads run.
//
// The two table kernels are latency-bound (a few hundred kilobytes at most):
// every CTA repeats the prefix sums over the sequences in shared memory (two
// loads and two block scans) rather than wait for a first kernel's result,
// then takes its share of the rows and pages.
#include <mutex>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

constexpr int kPT = 512;              // threads of the table kernels
constexpr int kPagesMaxB = 4096;
constexpr int kPerThread = kPagesMaxB / kPT;
constexpr int kRowsPerCta = 512;      // slot-map rows (or pages pushed) a CTA is launched for
constexpr int kSeqsPerCta = 16;       // sequences whose entries and counts a CTA writes
constexpr int kAloneBytes = 116 << 10;  // shared memory that only one CTA an SM finds
static_assert((5 * kPagesMaxB + 1) * 4 <= kAloneBytes, "the largest call");

// Exclusive prefix sum of one value per thread over the CTA; total in *sum.
__device__ __forceinline__ long long block_scan(long long v, long long *warp_sums, long long *sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();  // the sums of an earlier scan have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPT / 32; ++w) {
        const long long s = warp_sums[w];
        if (w < warp) before += s;
        all += s;
    }
    *sum = all;
    return before + x - v;
}

// Last b in [0, n) with base[b] <= x (base ascending, base[0] <= x).
__device__ __forceinline__ int last_at_most(const int *base, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return tokens / page_size + (tokens % page_size != 0);
}

constexpr int kServed = 1 << 30;  // flag beside a page count below it

// Sequence b: valid lengths, then need_b pages past the held_b it has;
// C_b = need_0 + .. + need_b.  Served when it needs none or C_b pages are
// free; its j-th new page is the stack's entry free - 1 - (C_{b-1} + j).
__global__ void __launch_bounds__(kPT) build_tables_kernel(BuildTablesArgs a) {
    extern __shared__ int sm[];
    __shared__ long long warp_sums[kPT / 32];
    int *starts = sm;                  // [B + 1] first row of each sequence
    int *prefix = starts + a.B + 1;    // [B]
    int *held = prefix + a.B;          // [B] pages held, kServed where served
    int *need = held + a.B;            // [B]
    int *taken = need + a.B;           // [B] C_{b-1}
    griddep_wait();
    griddep_launch_dependents();
    const int per = (a.B + kPT - 1) / kPT;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    const int nfree = *a.free_count;
    const bool pool_ok = nfree >= 0 && nfree <= a.num_pages;
    const long long room = (long long)a.max_pages * a.page_size;

    int n[kPerThread], len[kPerThread], cnt[kPerThread];
    long long rows = 0, total_rows, total_need;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {  // every load on its way before the first is used
        const bool in = b0 + i < b1;
        n[i] = in ? a.new_lens[b0 + i] : 0;
        len[i] = in ? a.prefix_lens[b0 + i] : 0;
        cnt[i] = in ? a.page_counts[b0 + i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int b = b0 + i;
        if (b >= b1) break;
        prefix[b] = len[i];
        held[b] = cnt[i];
        rows += max(n[i], 0);
    }
    long long row = block_scan(rows, warp_sums, &total_rows);
    long long sum = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int b = b0 + i;
        if (b >= b1) break;
        starts[b] = (int)min(row, (long long)INT32_MAX);
        row += max(n[i], 0);
        const int L = len[i], h = cnt[i];
        const bool valid = L >= 0 && n[i] >= 0 && (long long)L + n[i] <= room && h >= 0 &&
                           h <= a.max_pages && h >= pages_of(L, a.page_size) && row <= a.num_rows;
        need[b] = valid ? max(pages_of(L + n[i], a.page_size) - h, 0) : -1;
        sum += max(need[b], 0);
    }
    if (threadIdx.x == 0) starts[a.B] = (int)min(total_rows, (long long)INT32_MAX);
    long long c = block_scan(sum, warp_sums, &total_need);
    int last = 0;  // pages taken by the last served sequence of this thread's that needs any
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int b = b0 + i;
        if (b >= b1) break;
        taken[b] = (int)min(c, (long long)INT32_MAX);
        if (need[b] >= 0) {
            c += need[b];
            if (need[b] == 0) held[b] |= kServed;
            else if (pool_ok && c <= nfree) {
                held[b] |= kServed;
                last = (int)c;
            }
        }
    }
    // C_b only grows: the largest of the served ones is what leaves the pool
    __syncthreads();
    if (blockIdx.x == 0) {
        const int most = __reduce_max_sync(0xffffffffu, last);
        if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = most;
        __syncthreads();
        if (threadIdx.x == 0) {
            long long m = 0;
            for (int w = 0; w < kPT / 32; ++w) m = max(m, warp_sums[w]);
            *a.new_free_count = nfree - (int)m;
            a.row_starts[a.B] = starts[a.B];
        }
    }

    // The page of row r of the slot map (-1: none) and its offset there.
    auto page_of = [&](int r, int &off) -> int {
        off = 0;
        if (r >= starts[a.B]) return -1;
        const int b = last_at_most(starts, a.B, r);
        if (need[b] < 0 || (held[b] & kServed) == 0) return -1;
        const int at = prefix[b] + r - starts[b];
        const int j = at / a.page_size, h = held[b] & ~kServed;
        off = at - j * a.page_size;
        return j < h ? a.block_table[(size_t)b * a.max_pages + j] : a.free_pages[nfree - 1 - (taken[b] + j - h)];
    };
    auto put_slot = [&](int r, int pg, int off) {
        a.slot_map[r] = pg >= 0 && pg < a.num_pages ? pg * a.page_size + off : -1;
    };
    // this CTA's rows of the slot map: the first one's page is on its way while
    // the sequences are written
    const int row0 = blockIdx.x * kPT + threadIdx.x;
    int off0 = 0;
    const int pg0 = row0 < a.num_rows ? page_of(row0, off0) : -1;

    // this CTA's sequences: table entries, counts, first rows, status; a warp each
    const int lane = threadIdx.x & 31;
    const int gwarp = (int)(blockIdx.x * (kPT / 32) + (threadIdx.x >> 5));
    for (int b = gwarp; b < a.B; b += (int)gridDim.x * (kPT / 32)) {
        const bool valid = need[b] >= 0;
        const bool served = valid && (held[b] & kServed) != 0;
        const int h = valid ? held[b] & ~kServed : held[b], nd = need[b];
        bool bad = !valid || (!served && !pool_ok);
        int32_t *trow = a.block_table + (size_t)b * a.max_pages;
        if (valid) {
            for (int j = lane; j < nd; j += 32) {
                int pg = -1;
                if (served) {
                    pg = a.free_pages[nfree - 1 - (taken[b] + j)];
                    if (pg < 0 || pg >= a.num_pages) bad = true;
                }
                trow[h + j] = pg;
            }
            // the held pages that the new rows fall into (without new rows none, not the one that the
            // prefix ends in either)
            const int end = starts[b + 1] - starts[b] + prefix[b];
            const int upto = end > prefix[b] ? min(h, pages_of(end, a.page_size)) : 0;
            for (int j = prefix[b] / a.page_size + lane; j < upto; j += 32) {
                const int pg = trow[j];
                if (pg < 0 || pg >= a.num_pages) bad = true;
            }
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            a.new_page_counts[b] = served ? h + nd : h;
            a.row_starts[b] = starts[b];
            if (a.seq_status)
                a.seq_status[b] = bad ? SV_ERR_BAD_INPUT : served ? SV_OK : SV_ERR_NO_PAGES;
        }
    }

    if (row0 < a.num_rows) put_slot(row0, pg0, off0);
    for (int r = row0 + (int)gridDim.x * kPT; r < a.num_rows; r += (int)gridDim.x * kPT) {
        int off;
        const int pg = page_of(r, off);
        put_slot(r, pg, off);
    }
}

// Sequence b keeps the pages of its first keep_lens[b] tokens; the others go
// on the stack in sequence order: entry j past the kept ones at
// free + R_{b-1} + j, R_b = back_0 + .. + back_b.
__global__ void __launch_bounds__(kPT) release_pages_kernel(ReleasePagesArgs a) {
    extern __shared__ int sm[];
    __shared__ long long warp_sums[kPT / 32];
    int *upto = sm;            // [B + 1] R_{b-1}
    int *kept = upto + a.B + 1;  // [B]
    griddep_wait();
    griddep_launch_dependents();
    const int per = (a.B + kPT - 1) / kPT;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    const int nfree = *a.free_count;
    const bool pool_ok = nfree >= 0 && nfree <= a.num_pages;

    int held[kPerThread], back[kPerThread], keep[kPerThread];
    long long sum = 0, total;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const bool in = b0 + i < b1;
        keep[i] = in ? a.keep_lens[b0 + i] : 0;
        held[i] = in ? a.page_counts[b0 + i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int b = b0 + i;
        if (b >= b1) break;
        const int k = keep[i] >= 0 ? pages_of(keep[i], a.page_size) : 0;
        const bool valid = keep[i] >= 0 && held[i] >= k && held[i] <= a.max_pages;
        back[i] = valid ? held[i] - k : -1;
        kept[b] = k;
        sum += max(back[i], 0);
    }
    long long r = block_scan(sum, warp_sums, &total);
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int b = b0 + i;
        if (b >= b1) break;
        upto[b] = (int)min(r, (long long)INT32_MAX);
        r += max(back[i], 0);
        // the stack has room for every page of the pool and no more
        const bool served = back[i] == 0 || (back[i] > 0 && pool_ok && nfree + r <= a.num_pages);
        if (blockIdx.x == 0) {
            a.new_page_counts[b] = served ? kept[b] : held[i];
            if (a.seq_status) a.seq_status[b] = served ? SV_OK : SV_ERR_BAD_INPUT;
        }
    }
    if (threadIdx.x == 0) upto[a.B] = (int)min(total, (long long)INT32_MAX);
    __syncthreads();
    // R_b only grows: the sequences that fit are the ones up to the first that does not
    int pushed = 0;
    if (pool_ok) {
        const int space = a.num_pages - nfree;
        pushed = upto[a.B] <= space ? upto[a.B] : upto[last_at_most(upto, a.B + 1, space)];
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.new_free_count = nfree + pushed;
    for (int e = blockIdx.x * kPT + threadIdx.x; e < pushed; e += gridDim.x * kPT) {
        const int b = last_at_most(upto, a.B, e);
        a.free_pages[nfree + e] = a.block_table[(size_t)b * a.max_pages + kept[b] + e - upto[b]];
    }
}

// Room in shared memory for any call, asked for once a device and kernel
// (one limit for every call, so that no thread's lowers another's).
static bool large_smem(const void *fn) {
    struct Entry {
        int dev;
        const void *fn;
    };
    static std::mutex mu;
    static Entry done[64];
    static int ndone = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < ndone; ++i)
        if (done[i].dev == dev && done[i].fn == fn) return true;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kAloneBytes) != cudaSuccess) return false;
    if (ndone < 64) done[ndone++] = Entry{dev, fn};
    return true;
}

static sv_status table_launch(const void *fn, int B, int words, long long work, cudaStream_t st,
                              void **args) {
    size_t smem = (size_t)words * sizeof(int);
    const int sms = device_sm_count();
    if (sms <= 0) return SV_ERR_CUDA;
    long long grid = (work + kRowsPerCta - 1) / kRowsPerCta;
    if (grid < (B + kSeqsPerCta - 1) / kSeqsPerCta) grid = (B + kSeqsPerCta - 1) / kSeqsPerCta;
    if (grid > sms) grid = sms;
    if (grid < 1) grid = 1;
    // A grid that takes most SMs has them to itself: the next call's CTAs, launched
    // early, otherwise met four together on the SMs that this one leaves free, and ran
    // as much longer (tables for 2048 requests call after call 9.4 us, so 6.5; for
    // 4096 11.9 or 17.5, so 11.9).
    if (grid > sms / 2 && smem < kAloneBytes) smem = kAloneBytes;
    if (smem > 40 * 1024 && !large_smem(fn)) return SV_ERR_CUDA;
    return launch_pdl(fn, dim3((unsigned)grid), dim3(kPT), smem, st, args) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

sv_status launch_build_tables(const BuildTablesArgs &a, cudaStream_t st) {
    BuildTablesArgs ka = a;
    void *args[] = {&ka};
    return table_launch((const void *)build_tables_kernel, a.B, 5 * a.B + 1, a.num_rows, st, args);
}

sv_status launch_release_pages(const ReleasePagesArgs &a, cudaStream_t st) {
    ReleasePagesArgs ka = a;
    void *args[] = {&ka};
    return table_launch((const void *)release_pages_kernel, a.B, 2 * a.B + 1, a.num_pages, st, args);
}

// ---------------------------------------------------------------- new rows

constexpr int kAT = 256;
constexpr int kAUnroll = 2;

// One 16-byte piece of a bf16 row from 8 source elements.
template <bool F32>
__device__ __forceinline__ uint4 load_piece(const void *src, size_t elem) {
    if constexpr (!F32) return ldg_stream(static_cast<const uint16_t *>(src) + elem);
    const float *f = static_cast<const float *>(src) + elem;
    const uint4 x = ldg_stream(f), y = ldg_stream(f + 4);
    return make_uint4(pack_bf16x2(__uint_as_float(x.x), __uint_as_float(x.y)),
                      pack_bf16x2(__uint_as_float(x.z), __uint_as_float(x.w)),
                      pack_bf16x2(__uint_as_float(y.x), __uint_as_float(y.y)),
                      pack_bf16x2(__uint_as_float(y.z), __uint_as_float(y.w)));
}

// A CTA takes a.rows_per_cta consecutive rows; a thread takes 16-byte pieces
// of them, K and V, kAUnroll of each in flight.
template <bool F32>
__global__ void __launch_bounds__(kAT) append_kv_kernel(AppendArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int r0 = blockIdx.x * a.rows_per_cta;
    const int nrows = min(a.rows_per_cta, a.num_rows - r0);
    const int vpd = a.D / 8, vpr = a.Hkv * vpd;  // pieces of a head's row, of a row
    const int slots = a.num_pages * a.page_size;
    const int total = nrows * vpr;
    uint4 *kp = static_cast<uint4 *>(a.k_pages), *vp = static_cast<uint4 *>(a.v_pages);
    for (int i0 = threadIdx.x; i0 < total; i0 += kAT * kAUnroll) {
        uint4 kr[kAUnroll], vr[kAUnroll];
        long long dst[kAUnroll];
#pragma unroll
        for (int u = 0; u < kAUnroll; ++u) {
            const int i = i0 + u * kAT;
            dst[u] = -1;
            if (i >= total) continue;
            const int rr = i / vpr, piece = i - rr * vpr, h = piece / vpd;
            const int row = r0 + rr, slot = a.slot_map[row];
            if (slot >= 0 && slot < slots) {
                const int pg = slot / a.page_size, off = slot - pg * a.page_size;
                dst[u] = (((long long)pg * a.Hkv + h) * a.page_size + off) * vpd + (piece - h * vpd);
                kr[u] = load_piece<F32>(a.k_new, (size_t)(row * a.k_stride) + piece * 8);
                vr[u] = load_piece<F32>(a.v_new, (size_t)(row * a.v_stride) + piece * 8);
            }
            if (piece == 0 && a.row_status)
                a.row_status[row] = slot >= -1 && slot < slots ? SV_OK : SV_ERR_BAD_INPUT;
        }
#pragma unroll
        for (int u = 0; u < kAUnroll; ++u)
            if (dst[u] >= 0) {
                kp[dst[u]] = kr[u];
                vp[dst[u]] = vr[u];
            }
    }
}

sv_status launch_append_kv(const AppendArgs &a, int dtype, cudaStream_t st) {
    AppendArgs ka = a;
    const int vpr = a.Hkv * a.D / 8;
    ka.rows_per_cta = vpr >= kAT * kAUnroll ? 1 : kAT * kAUnroll / vpr;
    // few rows: spread them over the SMs
    const int sms = device_sm_count();
    if (sms <= 0) return SV_ERR_CUDA;
    const int even = (a.num_rows + sms - 1) / sms;
    if (even < ka.rows_per_cta) ka.rows_per_cta = even;
    void *args[] = {&ka};
    const void *fn = dtype == SV_F32 ? (const void *)append_kv_kernel<true> : (const void *)append_kv_kernel<false>;
    const unsigned grid = (unsigned)((a.num_rows + ka.rows_per_cta - 1) / ka.rows_per_cta);
    return launch_pdl(fn, dim3(grid), dim3(kAT), 0, st, args) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
