// sv_chunk.cuh -- geometry, parameters and shared-memory layout of the chunk
// attention kernel (sv_chunk_tc.cu) and its host side (sv_chunk.cu).
#pragma once

#include "sv_chunk_call.h"
#include "sv_chunk_list.h"
#include "sv_device.cuh"
#include "sv_internal.h"

namespace sv {
namespace chunk {

constexpr int kBK = kTileSlots;          // slots of a K/V tile
constexpr int kRows = 128;               // rows of a Q tile (the MMA's M)
constexpr int kBox = kBK * 64 * 2;       // 128 rows of 64 dims: 16 KB
constexpr int kThreads = 32 * 12;
constexpr int kSoftmaxRegs = 200, kOtherRegs = 104;  // 256 x 200 + 128 x 104 = 384 x 168
constexpr int kLaunchRegs = 168;
constexpr int kItems = 4;                // items published ahead
constexpr int kWarpPlanB = 128;          // sequences up to which one warp plans alone
constexpr int kNone = INT32_MIN;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units the maximum grows before O is rescaled

// Tensor-memory columns: S (then P) of streams 0 and 1, O of streams 0 and 1.
constexpr uint32_t kCols = 512, kColS = 0, kColO = 256;

template <int D>
constexpr int kTileBytes = kBK * D * 2;
template <int D>
constexpr int kStagesOf = D == 128 ? 5 : 12;  // K and V tiles in flight

struct Params {
    uint16_t *out;
    float *lse;                    // or null
    const int32_t *block_table;
    const int32_t *prefix_lens;
    const int32_t *row_starts;
    int32_t *seq_status;           // or null
    Shape shape;                   // tpt = 128 / G tokens of a Q tile
    int B, Hq, Hkv, G;
    int max_pages, num_pages, page_size;
    float scale_log2;
    float *part_o;   // [grid][2][Q tile][D / 4][128] float4: a cut item's unnormalised O
    float *part_ml;  // [grid][2][Q tile][128] float2: (max in log2 units, sum)
    int *counters;   // [2 sets][grid][Q tile][quarter]: CTAs arrived at a cut item (sv_chunk_call.h)
    CallWords *call;  // the form's
};

// This CTA's share added to the workspace's word, by one thread: the call's number.
__device__ __forceinline__ unsigned long long begin_call(CallWords *words) {
    return call_number(atomicAdd(&words->shares, call_share((int)blockIdx.x, (int)gridDim.x)));
}

// The number of the call, whose share this thread has added, or another of the CTA before it met.
__device__ __forceinline__ unsigned long long this_call(const CallWords *words) {
    const unsigned long long shares = *reinterpret_cast<const volatile unsigned long long *>(&words->shares);
    return call_number(shares - call_share((int)blockIdx.x, (int)gridDim.x));
}

// A wait of this CTA gave up: the whole call is reported, by one thread.
__device__ __noinline__ inline void give_up(CallWords *words, int32_t *seq_status, int B) {
    atomicExch(&words->gave_up, call_tag(this_call(words)));
    __threadfence();
    if (seq_status)
#pragma unroll 1
        for (int b = 0; b < B; ++b) seq_status[b] = SV_ERR_TIMEOUT;
}

// Whether a wait of the call has given up, asked by a thread that has written a status.
__device__ __forceinline__ bool gave_up(const CallWords *words) {
    __threadfence();
    return *reinterpret_cast<const volatile unsigned long long *>(&words->gave_up) == call_tag(this_call(words));
}

// A run of K/V tiles of one item.
struct Item {
    int b;             // sequence; -1: the end of the list
    int h;             // KV head
    int row0, ntok;    // first row, tokens (1 .. 2 tpt)
    int pos0;          // position of the first token
    int kt0, n;        // first K/V tile and number of tiles of this run
    int single;        // the sequence's only item: its K/V is read once
    int c_first, nc;   // CTAs that share the item's tiles: c_first .. c_first + nc - 1
    int ci;            // this CTA's index among them
    int counters;      // a cut item's arrival counters, from p.counters on
};

struct Shared {
    uint64_t full[12], empty[12];      // K/V ring
    uint64_t q_full[2], q_empty[2];    // Q tiles
    uint64_t s_full[2], p_full[2];     // per stream: S ready; P ready
    uint64_t o_full[2], o_empty[2];    // per stream: O complete; O read
    uint64_t x_full[2];                // per stream: its share of a one-tile item posted
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t fin;
    float2 xml[2][kRows];              // a stream's (m, sum) of a one-tile item
    Item items[kItems];
    long long warp_units[kThreads / 32];
    int warp_items[kThreads / 32], warp_most[kThreads / 32];
    uint32_t tmem;
    int abort_flag;
};

// The form for a few rows over short tables (sv_chunk_few.cu).
struct FewParams {
    Params c;  // (of which the workspace's parts but `call` are unused)
    const uint16_t *q, *k, *v;
    long long q_stride;  // elements between rows of q
    int cluster;         // CTAs of a row and KV head
};

// CTAs a row and KV head in that form, 0 where the call does not take it.
int few_cluster(const ChunkArgs &args);
sv_status launch_few(const ChunkArgs &args, const Params &params, int cluster, cudaStream_t stream);

const void *kernel_fn(int D);
int smem_bytes(int D);

}  // namespace chunk
}  // namespace sv
