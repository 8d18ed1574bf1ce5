// sv_chunk.cu -- host side of the chunk attention: tensor maps over the paged
// caches and the packed Q rows, the launch plan and workspace, the launch of
// the kernel in sv_chunk_tc.cu.
#include <mutex>

#include "sv_chunk.cuh"
#include "sv_quant_rows.h"

namespace sv {

namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                                         cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeFn>(ptr) : nullptr;
    }();
    return fn;
}

bool encode(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
            const cuuint32_t *box) {
    const EncodeFn enc = encode_fn();
    const cuuint32_t unit[3] = {1, 1, 1};
    return enc && enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims,
                      strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [rows, D] view of a paged cache, boxes of `box_rows` rows x 64 dims.
bool cache_map(CUtensorMap *map, const void *base, long long rows, int D, int box_rows) {
    const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)D * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    return encode(map, base, 2, dims, strides, box);
}

// [num_rows, Hq, D] view of Q, boxes of `tokens` rows x G heads x 64 dims; rows past the end read zeros.
bool q_map(CUtensorMap *map, const void *q, int num_rows, int Hq, int D, long long stride, int G, int tokens) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)num_rows};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tokens};
    return encode(map, q, 3, dims, strides, box);
}

// SMs of the current device once the kernel is known to run on it as
// planned, asked for once a device: the attribute calls cost more than a
// launch.  0 when it cannot run.
int ready_sms(int D, bool quant) {
    struct Entry {
        int dev, D, sms;
        bool quant;
    };
    static std::mutex mu;
    static Entry cache[64];
    static int ncache = 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < ncache; ++i)
        if (cache[i].dev == dev && cache[i].D == D && cache[i].quant == quant) return cache[i].sms;
    const void *fn = quant ? chunk::quant_kernel_fn(D) : chunk::kernel_fn(D);
    const int smem = quant ? chunk::quant_smem_bytes(D) : chunk::smem_bytes(D);
    const int threads = quant ? chunk::kThreadsOf<true> : chunk::kThreadsOf<false>;
    const int regs = quant ? chunk::kLaunchRegsOf<true> : chunk::kLaunchRegsOf<false>;
    int max_optin = 0, sms = device_sm_count(), occ = 0;
    cudaFuncAttributes at;
    // the kernel hands its launch registers out again (setmaxnreg): it must
    // have been built with as many as that split adds up to
    if (cudaDeviceGetAttribute(&max_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        smem > max_optin || cudaFuncGetAttributes(&at, fn) != cudaSuccess || at.numRegs < regs ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem) != cudaSuccess || occ < 1)
        return 0;
    if (ncache < 64) cache[ncache++] = Entry{dev, D, sms, quant};
    return sms;
}

}  // namespace

sv_status plan_chunk(int Hq, int Hkv, int D, bool quant, ChunkPlan *plan) {
    if ((D != 64 && D != 128) || Hq / Hkv > chunk::kRows) return SV_ERR_UNSUPPORTED;
    ChunkPlan pl{};
    pl.grid = ready_sms(D, quant);
    if (pl.grid <= 0) return SV_ERR_CUDA;
    const size_t tiles = (size_t)pl.grid * 2 * 2;
    static_assert(3 * sizeof(chunk::CallWords) <= chunk::kCallBytes, "the forms' words");
    size_t off = chunk::kCallBytes;
    pl.off_counters = off;
    off = align_up(off + sizeof(int) * (size_t)pl.grid * 2 * chunk::kCtaCounters, 256);
    pl.off_rows = off;
    off = align_up(off + sizeof(int) * 2 * chunk::kRowsMaxGrid, 256);
    static_assert(chunk::kRowsCols * 2 <= chunk::kRows, "twice the CTAs find room for their shares' rows");
    if (off > 64 * 1024 || pl.grid > chunk::kCallShares) return SV_ERR_UNSUPPORTED;  // (what starts as zeros; 1020 SMs)
    pl.off_part_ml = off;
    off = align_up(off + tiles * chunk::kRows * 2 * sizeof(float), 256);
    pl.off_part_o = off;
    off = align_up(off + tiles * chunk::kRows * (size_t)D * sizeof(float), 256);
    pl.bytes = off;
    *plan = pl;
    return SV_OK;
}

sv_status launch_chunk_attention(const ChunkArgs &a, const ChunkPlan &pl, void *ws, cudaStream_t st) {
    const int G = a.Hq / a.Hkv, tpt = chunk::kRows / G;
    char *base = static_cast<char *>(ws);
    chunk::QuantParams p{};
    p.out = static_cast<uint16_t *>(a.out);
    p.lse = a.lse;
    p.block_table = a.block_table;
    p.prefix_lens = a.prefix_lens;
    p.row_starts = a.row_starts;
    p.seq_status = a.seq_status;
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = G;
    const int S_max = a.max_pages * a.page_size;
    // (a window as long as the table hides nothing)
    p.shape = chunk::Shape{tpt, a.window < S_max ? a.window : 0, a.num_rows, S_max};
    p.max_pages = a.max_pages;
    p.num_pages = a.num_pages;
    p.page_size = a.page_size;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.part_o = reinterpret_cast<float *>(base + pl.off_part_o);
    p.part_ml = reinterpret_cast<float *>(base + pl.off_part_ml);
    p.counters = reinterpret_cast<int *>(base + pl.off_counters);
    p.call = reinterpret_cast<chunk::CallWords *>(base);
    if (a.k_params) {
        p.k_codes = static_cast<const uint8_t *>(a.k_pages);
        p.v_codes = static_cast<const uint8_t *>(a.v_pages);
        p.k_params = static_cast<const uint32_t *>(a.k_params);
        p.v_params = static_cast<const uint32_t *>(a.v_params);
        p.parents = a.parents;
        if (const int form = chunk::rows_form(a); form >= 0) {
            p.call += 2;
            p.counters = reinterpret_cast<int *>(base + pl.off_rows);
            return chunk::launch_rows(a, p, form, st);
        }
    } else if (const int cluster = chunk::few_cluster(a)) {
        ++p.call;
        return chunk::launch_few(a, p, cluster, st);
    }
    const long long rows = (long long)a.num_pages * a.Hkv * a.page_size;
    const int box_rows = a.page_size < chunk::kBK ? a.page_size : chunk::kBK;
    CUtensorMap tmk{}, tmv{}, tmq, tmq1;
    const bool paged = a.k_params || (cache_map(&tmk, a.k_pages, rows, a.D, box_rows) && cache_map(&tmv, a.v_pages, rows, a.D, box_rows));
    if (!paged || !q_map(&tmq, a.q, a.num_rows, a.Hq, a.D, a.q_stride, G, tpt) ||
        !q_map(&tmq1, a.q, a.num_rows, a.Hq, a.D, a.q_stride, G, 1))
        return SV_ERR_CUDA;
    chunk::Params plain = p;
    void *args[] = {&tmk, &tmv, &tmq, &tmq1, a.k_params ? static_cast<void *>(&p) : &plain};
    const cudaError_t rc =
        a.k_params ? launch_pdl(chunk::quant_kernel_fn(a.D), dim3(pl.grid), dim3(chunk::kThreadsOf<true>), chunk::quant_smem_bytes(a.D), st, args)
                   : launch_pdl(chunk::kernel_fn(a.D), dim3(pl.grid), dim3(chunk::kThreadsOf<false>), chunk::smem_bytes(a.D), st, args);
    return rc == cudaSuccess
               ? SV_OK
               : SV_ERR_CUDA;
}

}  // namespace sv
