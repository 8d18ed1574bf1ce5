// sv_fork.cu -- requests that share pages of a paged cache: forks of a request
// (several continuations of one prompt), the copies of the pages that are only
// partly filled, and pages given back when some of their holders go.
//
// The paged KV of "Chapitre 9", section "Ce que prépare le Chapitre 9".  Beside
// the stack of free pages (sv_pages.cu) a page has a count of its holders but
// one, so that a pool without shared pages has zeros there and the calls that
// know nothing of sharing stay right for it.  Results do not depend on the order
// in which threads run: counts are sums, pages are handed out by prefix sums in
// the order of the forks, and go back in the order of the sequences.
#include <mutex>

#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int kFT = 512;               // threads of the fork kernels
constexpr int kMaxSeqs = 4096;         // sequences, and forks of a call
constexpr int kPer = kMaxSeqs / kFT;   // of a thread
constexpr int kEntriesPerCta = 512;    // table entries a CTA is launched for
constexpr int kAllBytes = (4 * kMaxSeqs + 1 + kMaxSeqs) * 4;  // shared memory of the largest call
static_assert(kAllBytes <= 116 << 10, "two CTAs an SM");

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return tokens / page_size + (tokens % page_size != 0);
}

// Inclusive prefix sum over the warp.
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    return x;
}

// Exclusive prefix sum of one value a thread over the CTA of T threads, the
// total in *sum.  Sums stay below 2^31 (entries of one table).
template <int T>
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int *sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int x = warp_scan(v, lane);
    __syncthreads();  // the sums of an earlier scan have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    const int s = lane < T / 32 ? warp_sums[lane] : 0, y = warp_scan(s, lane);
    *sum = __shfl_sync(0xffffffffu, y, 31);
    return __shfl_sync(0xffffffffu, y - s, warp) + x - v;
}

// Last f in [0, n) with base[f] <= x (base ascending, base[0] <= x).
__device__ __forceinline__ int last_at_most(const int *base, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (base[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// What the forks' sums start from: the counts as they are, no fork refused yet.
__global__ void __launch_bounds__(kFT) copy_shares_kernel(const int32_t *shares, int32_t *new_shares, int num_pages,
                                                          int32_t *status, int n) {
    griddep_wait();
    griddep_launch_dependents();
    const long long first = (long long)blockIdx.x * kFT + threadIdx.x, step = (long long)gridDim.x * kFT;
    for (long long i = first; i < num_pages; i += step) new_shares[i] = max(shares[i], 0);
    if (status)
        for (long long i = first; i < n; i += step) status[i] = SV_OK;
}

// Fork f: the first fork_lens[f] slots of sequence sources[f] for targets[f], which
// holds nothing.  Full pages are shared, the one that the length ends in is
// copied (by another kernel) to a page from the stack.  Every CTA repeats the
// prefix sums over the forks, then takes its share of the entries.
__global__ void __launch_bounds__(kFT) fork_tables_kernel(const ForkArgs a) {
    extern __shared__ int sm[];
    __shared__ int warp_sums[kFT / 32];
    int *starts = sm;              // [F + 1] shared entries before each fork
    int *src = starts + a.F + 1;   // [F] source, -1 where the fork is not served
    int *tgt = src + a.F;          // [F]
    int *taken = tgt + a.F;        // [F] pages taken up to and with this fork
    int *owner = taken + a.F;      // [B] first fork that names the sequence as its target
    griddep_wait();
    griddep_launch_dependents();
    for (int b = threadIdx.x; b < a.B; b += kFT) owner[b] = INT32_MAX;
    const int per = (a.F + kFT - 1) / kFT;
    const int f0 = min((int)threadIdx.x * per, a.F), f1 = min(f0 + per, a.F);
    const int nfree = *a.free_count;
    const bool pool_ok = nfree >= 0 && nfree <= a.num_pages;
    int s[kPer], t[kPer], len[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool in = f0 + i < f1;
        s[i] = in ? a.sources[f0 + i] : -1;
        t[i] = in ? a.targets[f0 + i] : -1;
        len[i] = in ? a.fork_lens[f0 + i] : 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (t[i] >= 0 && t[i] < a.B) atomicMin(&owner[t[i]], f0 + i);
    __syncthreads();
    int need = 0, entries = 0;
    uint32_t valid = 0;  // a bit a fork of this thread's
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (f0 + i >= f1) break;
        const bool named = s[i] >= 0 && s[i] < a.B && t[i] >= 0 && t[i] < a.B && s[i] != t[i] && len[i] >= 0;
        const int held = named ? a.page_counts[s[i]] : -1, empty = named ? a.page_counts[t[i]] : -1;
        if (named && empty == 0 && owner[t[i]] == f0 + i && held <= a.max_pages && pages_of(len[i], a.page_size) <= held) {
            valid |= 1u << i;
            need += len[i] % a.page_size != 0;
        }
    }
    int total, c = block_scan<kFT>(need, warp_sums, &total);
    int last = 0;
    uint32_t served = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int f = f0 + i;
        if (f >= f1) break;
        if (valid >> i & 1) {
            const int part = len[i] % a.page_size != 0;
            c += part;
            if (!part || (pool_ok && c <= nfree)) {
                served |= 1u << i;
                entries += len[i] / a.page_size;
                if (part) last = c;
            }
        }
        taken[f] = c;
        src[f] = served >> i & 1 ? s[i] : -1;
        tgt[f] = t[i];
    }
    int e = block_scan<kFT>(entries, warp_sums, &total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (f0 + i >= f1) break;
        starts[f0 + i] = e;
        if (served >> i & 1) e += len[i] / a.page_size;
    }
    if (threadIdx.x == 0) starts[a.F] = total;
    __syncthreads();
    if (blockIdx.x == 0) {  // (taken only grows: the most of the served ones is what leaves the pool)
        const int most = __reduce_max_sync(0xffffffffu, last);
        if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = most;
        __syncthreads();
        if (threadIdx.x == 0) {
            int m = 0;
            for (int w = 0; w < kFT / 32; ++w) m = max(m, warp_sums[w]);
            *a.new_free_count = nfree - m;
        }
    }
    // counts of the sequences, and the forks' partly filled pages
    const int first = blockIdx.x * kFT + threadIdx.x, step = gridDim.x * kFT;
    for (int b = first; b < a.B; b += step) {
        const int f = owner[b];
        a.new_page_counts[b] = f < INT32_MAX && src[f] >= 0 ? pages_of(a.fork_lens[f], a.page_size) : a.page_counts[b];
    }
    for (int f = first; f < a.F; f += step) {
        const int n = src[f] >= 0 ? a.fork_lens[f] : 0, full = n / a.page_size, part = n - full * a.page_size;
        int from = -1, to = -1, code = SV_OK;
        if (src[f] < 0) {
            // valid but not served, for want of pages: the only reason that a sum of the pool's says
            const int sf = a.sources[f], tf = tgt[f], nf = a.fork_lens[f];
            const bool named = sf >= 0 && sf < a.B && tf >= 0 && tf < a.B && sf != tf && nf >= 0;
            const bool fits = named && a.page_counts[tf] == 0 && owner[tf] == f && a.page_counts[sf] <= a.max_pages &&
                              pages_of(nf, a.page_size) <= a.page_counts[sf];
            code = fits && pool_ok ? SV_ERR_NO_PAGES : SV_ERR_BAD_INPUT;
        } else if (part > 0) {
            from = a.block_table[(size_t)src[f] * a.max_pages + full];
            to = a.free_pages[nfree - taken[f]];
            a.block_table[(size_t)tgt[f] * a.max_pages + full] = to;
            if (from < 0 || from >= a.num_pages || to < 0 || to >= a.num_pages) code = SV_ERR_BAD_INPUT;
        }
        a.copies[3 * (size_t)f] = from;
        a.copies[3 * (size_t)f + 1] = to;
        a.copies[3 * (size_t)f + 2] = part;
        if (code != SV_OK && a.fork_status) atomicMax(&a.fork_status[f], code);
    }
    // the shared entries
    for (long long i = first; i < total; i += step) {
        const int f = last_at_most(starts, a.F, (int)i), j = (int)i - starts[f];
        const int pg = a.block_table[(size_t)src[f] * a.max_pages + j];
        a.block_table[(size_t)tgt[f] * a.max_pages + j] = pg;
        if (pg >= 0 && pg < a.num_pages) atomicAdd(&a.new_shares[pg], 1);
        else if (a.fork_status) atomicMax(&a.fork_status[f], (int)SV_ERR_BAD_INPUT);
    }
}

// ---------------------------------------------------------------- copies

constexpr int kPT = 256;

// A warp copies one page's filled slots of one KV head and plane: they are
// contiguous.  Planes whose rows are a multiple of 16 bytes go by 16, others by 4.
__global__ void __launch_bounds__(kPT) copy_pages_kernel(const __grid_constant__ CopyPagesArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31, units = a.num_planes * a.Hkv;
    const long long all = (long long)a.F * units, step = (long long)gridDim.x * (kPT / 32);
    for (long long u = (long long)blockIdx.x * (kPT / 32) + (threadIdx.x >> 5); u < all; u += step) {
        const int f = (int)(u / units), rest = (int)(u - (long long)f * units), pl = rest / a.Hkv, h = rest - pl * a.Hkv;
        const int from = a.copies[3 * (size_t)f], to = a.copies[3 * (size_t)f + 1], rows = a.copies[3 * (size_t)f + 2];
        const bool none = from == -1 && to == -1;
        const bool ok = !none && from >= 0 && from < a.num_pages && to >= 0 && to < a.num_pages && from != to && rows >= 0 &&
                        rows <= a.page_size;
        if (rest == 0 && lane == 0 && a.copy_status) a.copy_status[f] = none || ok ? SV_OK : SV_ERR_BAD_INPUT;
        if (!ok) continue;
        const int rb = a.row_bytes[pl];
        const size_t head = (size_t)a.page_size * rb;
        const char *x = static_cast<const char *>(a.planes[pl]) + ((size_t)from * a.Hkv + h) * head;
        char *y = static_cast<char *>(a.planes[pl]) + ((size_t)to * a.Hkv + h) * head;
        const long long bytes = (long long)rows * rb;
        if (rb % 16 == 0) {
            constexpr int kAhead = 4;
            for (long long i0 = 16 * lane; i0 < bytes; i0 += 512 * kAhead) {
                uint4 v[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (i0 + 512 * k < bytes) v[k] = ldg_stream(x + i0 + 512 * k);
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if (i0 + 512 * k < bytes) *reinterpret_cast<uint4 *>(y + i0 + 512 * k) = v[k];
            }
        } else {
            for (long long i = 4 * lane; i < bytes; i += 128)
                *reinterpret_cast<uint32_t *>(y + i) = *reinterpret_cast<const uint32_t *>(x + i);
        }
    }
}

// ---------------------------------------------------------------- shared pages given back

constexpr int kRT = 1024;
constexpr int kRPer = kMaxSeqs / kRT;
constexpr int kReleaseCluster = 8;
constexpr long long kClusterEntries = 49152;  // entries of the table up to which one cluster gives pages back
static_assert(kRT / 32 == 32, "a lane a warp of the CTA");

// Entries that the sequences give up, in sequence order; a page whose count of
// other holders is s keeps max(0, s - k) of them after k of its entries, and goes
// to the stack in the place of the last one where k > s.  Four parts, each of which
// needs the ones before it everywhere: the counts, marks and statuses are set; the
// shared pages' entries are counted (atomic sums and a maximum); a warp counts the
// pages of its run of consecutive entries that go to the stack; it pushes them.
//
// Up to kClusterEntries entries one cluster does all four and meets between them;
// above, four launches over the whole GPU do.  Both measured, us, the cluster first:
// tables of 2 thousand entries 8.9 and 11.8, of 31 thousand 11.9 and 14.7, of 300
// thousand (2048 branches of 2048 tokens) 57 and 22.6, where the cluster's eight SMs
// are what bounds it.  One CTA alone is 0.3 us quicker for 2 thousand and 5 us slower
// for 8 thousand.
struct Shares {
    const int *upto, *kept;  // entries before each sequence, pages that it keeps
    int total, nfree;
    bool pool_ok;
};

// The sequences' entries, by a whole CTA; `write`: the counts and statuses too.
__device__ __forceinline__ Shares plan_shares(const ReleaseSharedArgs &a, int *sm, int *warp_sums, bool write) {
    int *upto = sm, *kept = upto + a.B + 1;  // [B + 1], [B]
    const int per = (a.B + kRT - 1) / kRT;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    const int nfree = *a.free_count;
    const bool pool_ok = nfree >= 0 && nfree <= a.num_pages;
    int keep[kRPer], held[kRPer];
#pragma unroll
    for (int i = 0; i < kRPer; ++i) {
        const bool in = b0 + i < b1;
        keep[i] = in ? a.keep_lens[b0 + i] : 0;
        held[i] = in ? a.page_counts[b0 + i] : 0;
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kRPer; ++i) {
        const int b = b0 + i;
        if (b >= b1) break;
        const int k = keep[i] >= 0 ? pages_of(keep[i], a.page_size) : 0;
        const bool valid = keep[i] >= 0 && held[i] >= k && held[i] <= a.max_pages && (pool_ok || held[i] == k);
        kept[b] = k;
        if (write) {
            a.new_page_counts[b] = valid ? k : held[i];
            if (a.seq_status) a.seq_status[b] = valid ? SV_OK : SV_ERR_BAD_INPUT;
        }
        held[i] = valid ? held[i] - k : 0;
        sum += held[i];
    }
    int total, r = block_scan<kRT>(sum, warp_sums, &total);
#pragma unroll
    for (int i = 0; i < kRPer; ++i) {
        if (b0 + i >= b1) break;
        upto[b0 + i] = r;
        r += held[i];
    }
    if (threadIdx.x == 0) upto[a.B] = total;
    __syncthreads();
    return Shares{upto, kept, total, nfree, pool_ok};
}

__device__ __forceinline__ void mark_pages(const ReleaseSharedArgs &a, int rank, int nct) {
    for (long long i = rank * kRT + threadIdx.x; i < a.num_pages; i += nct * kRT) {
        a.new_shares[i] = max(a.shares[i], 0);
        a.last[i] = -1;
    }
}

__device__ __forceinline__ int entry_page(const ReleaseSharedArgs &a, const Shares &s, int e, int &b) {
    b = last_at_most(s.upto, a.B, e);
    return a.block_table[(size_t)b * a.max_pages + s.kept[b] + e - s.upto[b]];
}

__device__ __forceinline__ void count_entries(const ReleaseSharedArgs &a, const Shares &s, int rank, int nct) {
    for (long long x = rank * kRT + threadIdx.x; x < s.total; x += nct * kRT) {
        const int e = (int)x;
        int b;
        const int pg = entry_page(a, s, e, b);
        if (pg < 0 || pg >= a.num_pages) {
            if (a.seq_status) a.seq_status[b] = SV_ERR_BAD_INPUT;
        } else if (a.shares[pg] > 0) {
            atomicSub(&a.new_shares[pg], 1);
            atomicMax(&a.last[pg], e);
        }
    }
}

// A warp's run of entries: warp w of n takes [first, end).
struct Run {
    int first, end;
};
__device__ __forceinline__ Run run_of(int total, int w, int n) {
    const long long run = ((long long)total + n - 1) / n;
    const int first = (int)min(w * run, (long long)total);
    return Run{first, (int)min((long long)first + run, (long long)total)};
}

// Whether the page of entry e, below end, goes to the stack.
__device__ __forceinline__ bool goes(const ReleaseSharedArgs &a, const Shares &s, long long x, int end, int &pg, int &b) {
    if (x >= end) return false;
    const int e = (int)x;
    pg = entry_page(a, s, e, b);
    if (pg < 0 || pg >= a.num_pages) return false;
    if (a.shares[pg] <= 0) return true;
    return __ldcg(&a.last[pg]) == e && __ldcg(&a.new_shares[pg]) < 0;
}

__device__ __forceinline__ int count_pushes(const ReleaseSharedArgs &a, const Shares &s, const Run &run, int lane) {
    int mine = 0;
    for (long long x = run.first; x < run.end; x += 32) {
        const int e = (int)x;
        int pg, b;
        mine += __popc(__ballot_sync(0xffffffffu, goes(a, s, (long long)e + lane, run.end, pg, b)));
    }
    return mine;
}

// The run's pages, to the stack's places from nfree + at on.
__device__ __forceinline__ void push_pages(const ReleaseSharedArgs &a, const Shares &s, const Run &run, int at, int lane) {
    for (long long x = run.first; x < run.end; x += 32) {
        const int e = (int)x;
        int pg, b;
        const bool push = goes(a, s, (long long)e + lane, run.end, pg, b);
        const uint32_t votes = __ballot_sync(0xffffffffu, push);
        if (push) {
            const long long to = (long long)s.nfree + at + __popc(votes & ((1u << lane) - 1u));
            if (to < a.num_pages) a.free_pages[to] = pg;
            else if (a.seq_status) a.seq_status[b] = SV_ERR_BAD_INPUT;  // (some page was free already)
            if (a.shares[pg] > 0) a.new_shares[pg] = 0;  // (only this entry looks at it again)
        }
        at += __popc(votes);
    }
}

__device__ __forceinline__ int new_free(const ReleaseSharedArgs &a, const Shares &s, long long pushed) {
    return s.pool_ok ? (int)min((long long)s.nfree + pushed, (long long)a.num_pages) : s.nfree;
}

__global__ void __launch_bounds__(kRT, 1) release_shared_kernel(const ReleaseSharedArgs a) {
    extern __shared__ int sm[];
    __shared__ int warp_sums[kRT / 32], pushed_by, before[kReleaseCluster];
    const int nct = gridDim.x, rank = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    griddep_wait();
    griddep_launch_dependents();
    mark_pages(a, rank, nct);
    const Shares s = plan_shares(a, sm, warp_sums, rank == 0);
    __threadfence();
    __syncthreads();
    cluster_sync();  // (counts, marks and statuses are set before any entry changes them)
    count_entries(a, s, rank, nct);
    __threadfence();
    __syncthreads();
    cluster_sync();
    const Run run = run_of(s.total, rank * (kRT / 32) + warp, nct * (kRT / 32));
    const int mine = count_pushes(a, s, run, lane);
    int pushed;
    const int ahead = __shfl_sync(0xffffffffu, block_scan<kRT>(lane == 0 ? mine : 0, warp_sums, &pushed), 0);
    if (threadIdx.x == 0) pushed_by = pushed;
    __syncthreads();
    cluster_sync();
    if (threadIdx.x < nct) before[threadIdx.x] = __float_as_int(ld_shared_cluster_f32(reinterpret_cast<float *>(&pushed_by), threadIdx.x));
    __syncthreads();
    int at = ahead;
    long long all = 0;
    for (int c = 0; c < nct; ++c) {
        if (c < rank) at += before[c];
        all += before[c];
    }
    if (rank == 0 && threadIdx.x == 0) *a.new_free_count = new_free(a, s, all);
    push_pages(a, s, run, at, lane);
    cluster_sync();  // (a CTA's shared memory is read by the others until here)
}

template <int kPart>
__global__ void __launch_bounds__(kRT, 1) release_part_kernel(const ReleaseSharedArgs a) {
    extern __shared__ int sm[];
    __shared__ int warp_sums[kRT / 32];
    const int nct = gridDim.x, rank = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int *const pushes = a.last + a.num_pages;  // [kReleaseMaxWarps], a warp's
    griddep_wait();
    griddep_launch_dependents();
    if (kPart == 0) mark_pages(a, rank, nct);
    if (kPart == 0 && rank > 0) return;
    const Shares s = plan_shares(a, sm, warp_sums, kPart == 0);
    const int w = rank * (kRT / 32) + warp, n = nct * (kRT / 32);
    const Run run = run_of(s.total, w, n);
    if (kPart == 1) count_entries(a, s, rank, nct);
    if (kPart == 2) {
        const int mine = count_pushes(a, s, run, lane);
        if (lane == 0) pushes[w] = mine;
    }
    if (kPart == 3) {
        const int first = rank * (kRT / 32);
        int before = 0, behind = 0, all, ahead;
        for (int i = threadIdx.x; i < n; i += kRT) (i < first ? before : behind) += pushes[i];
        block_scan<kRT>(before, warp_sums, &ahead);
        block_scan<kRT>(behind, warp_sums, &all);
        const int own = warp_scan(pushes[first + lane], lane);  // (all of the CTA's, in every warp)
        const int at = ahead + (warp > 0 ? __shfl_sync(0xffffffffu, own, (warp - 1) & 31) : 0);
        if (rank == 0 && threadIdx.x == 0) *a.new_free_count = new_free(a, s, (long long)ahead + all);
        push_pages(a, s, run, at, lane);
    }
}

// Room in shared memory for any call, asked for once a device and kernel.
bool large_smem(const void *fn) {
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
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kAllBytes) != cudaSuccess) return false;
    if (ndone < 64) done[ndone++] = Entry{dev, fn};
    return true;
}

}  // namespace

sv_status launch_fork_tables(const ForkArgs &a, cudaStream_t st) {
    const int sms = device_sm_count();
    if (sms <= 0) return SV_ERR_CUDA;
    ForkArgs ka = a;
    const int32_t *shares = a.shares;
    int32_t *new_shares = a.new_shares, *status = a.fork_status;
    int num_pages = a.num_pages, F = a.F;
    void *cargs[] = {&shares, &new_shares, &num_pages, &status, &F};
    const long long most = num_pages > F ? num_pages : F;
    const long long cgrid = (most + 4 * kFT - 1) / (4 * kFT);
    if (launch_pdl((const void *)copy_shares_kernel, dim3((unsigned)(cgrid < 2 * sms ? cgrid : 2 * sms)), dim3(kFT), 0, st,
                   cargs) != cudaSuccess)
        return SV_ERR_CUDA;
    const size_t smem = (size_t)(4 * a.F + 1 + a.B) * sizeof(int);
    if (smem > 40 * 1024 && !large_smem((const void *)fork_tables_kernel)) return SV_ERR_CUDA;
    long long grid = ((long long)a.F * a.max_pages + kEntriesPerCta - 1) / kEntriesPerCta;
    if (grid < (a.B + kFT - 1) / kFT) grid = (a.B + kFT - 1) / kFT;
    if (grid > sms) grid = sms;
    void *args[] = {&ka};
    return launch_pdl((const void *)fork_tables_kernel, dim3((unsigned)grid), dim3(kFT), smem, st, args) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

sv_status launch_copy_pages(const CopyPagesArgs &a, cudaStream_t st) {
    const int sms = device_sm_count();
    if (sms <= 0) return SV_ERR_CUDA;
    CopyPagesArgs ka = a;
    void *args[] = {&ka};
    long long grid = ((long long)a.F * a.num_planes * a.Hkv + kPT / 32 - 1) / (kPT / 32);
    if (grid > 8LL * sms) grid = 8LL * sms;
    return launch_pdl((const void *)copy_pages_kernel, dim3((unsigned)grid), dim3(kPT), 0, st, args) == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

sv_status launch_release_shared(const ReleaseSharedArgs &a, cudaStream_t st) {
    ReleaseSharedArgs ka = a;
    void *args[] = {&ka};
    const size_t smem = (size_t)(2 * a.B + 1) * sizeof(int);
    if (smem > 40 * 1024) return SV_ERR_UNSUPPORTED;  // (never: B <= 4096)
    const long long entries = (long long)a.B * a.max_pages;
    if (entries > kClusterEntries) {
        const int sms = device_sm_count();
        if (sms <= 0) return SV_ERR_CUDA;
        long long grid = (entries + 2 * kRT - 1) / (2 * kRT);
        if (grid > sms) grid = sms;
        if (grid > kReleaseMaxWarps / (kRT / 32)) grid = kReleaseMaxWarps / (kRT / 32);
        const void *parts[] = {(const void *)release_part_kernel<0>, (const void *)release_part_kernel<1>,
                               (const void *)release_part_kernel<2>, (const void *)release_part_kernel<3>};
        for (const void *part : parts)
            if (launch_pdl(part, dim3((unsigned)grid), dim3(kRT), smem, st, args) != cudaSuccess) return SV_ERR_CUDA;
        return SV_OK;
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kReleaseCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kReleaseCluster);
    cfg.blockDim = dim3(kRT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelExC(&cfg, (const void *)release_shared_kernel, args) == cudaSuccess ? SV_OK : SV_ERR_CUDA;
}

}  // namespace sv
