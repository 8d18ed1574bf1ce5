// sv_api.cu -- the extern "C" boundary of libspecverify: argument checks on
// the host (nothing is launched when they fail), then the kernel launches.
// Declarations and the contract of every call are in include/specverify.h.
#include <cmath>
#include <cstdint>

#include "sv_internal.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

cudaStream_t as_stream(sv_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

}  // namespace

extern "C" {

int sv_version(void) { return 100; }  // 0.1.0

const char *sv_status_string(sv_status s) {
    switch (s) {
        case SV_OK: return "SV_OK";
        case SV_ERR_INVALID_ARG: return "SV_ERR_INVALID_ARG: invalid argument";
        case SV_ERR_WORKSPACE: return "SV_ERR_WORKSPACE: workspace missing or too small";
        case SV_ERR_UNSUPPORTED: return "SV_ERR_UNSUPPORTED: shape outside the supported range";
        case SV_ERR_CUDA: return "SV_ERR_CUDA: a CUDA runtime call failed";
        case SV_ERR_TIMEOUT: return "SV_ERR_TIMEOUT: a bounded wait in a kernel gave up";
        case SV_ERR_BAD_INPUT: return "SV_ERR_BAD_INPUT: invalid per-sequence input";
        case SV_ERR_NO_PAGES: return "SV_ERR_NO_PAGES: too few free pages";
    }
    return "unknown sv_status";
}

size_t sv_workspace_size(sv_op op, int B, int T_or_N, int V, sv_dtype dtype, int Hq, int Hkv,
                         int D) {
    if (op == SV_OP_CHUNK_ATTENTION) {
        if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
        sv::ChunkPlan pl;
        return sv::plan_chunk(Hq, Hkv, D, false, &pl) == SV_OK ? pl.bytes : 0;
    }
    if (op == SV_OP_RELEASE_SHARED_PAGES) return T_or_N > 0 ? ((size_t)T_or_N + sv::kReleaseMaxWarps) * sizeof(int) : 0;
    if (B <= 0 || T_or_N <= 0) return 0;
    switch (op) {
        case SV_OP_CHUNK_ATTENTION:
        case SV_OP_RELEASE_SHARED_PAGES: break;  // (above)
        case SV_OP_TREE_ATTENTION: {
            if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
            sv::AttnPlan pl;
            // (the workspace does not depend on the cache length)
            if (sv::plan_attention(B, T_or_N, Hq, Hkv, D, 1 << 30, &pl) != SV_OK) return 0;
            return pl.bytes;
        }
        case SV_OP_VERIFY_CHAIN:
        case SV_OP_VERIFY_TREE_GREEDY: {
            if (V <= 0 || (dtype != SV_F32 && dtype != SV_BF16)) return 0;
            // the shapes the calls refuse as unsupported have no size
            if (T_or_N > (op == SV_OP_VERIFY_CHAIN ? 63 : 1024) || V >= (1 << 30)) return 0;
            const sv::VocabPlan pl = sv::plan_vocab(op == SV_OP_VERIFY_CHAIN, B, T_or_N, V, dtype);
            if ((size_t)B * pl.rows_per_seq * pl.nchunks >= (1u << 31)) return 0;
            return pl.bytes;
        }
        case SV_OP_VERIFY_TREE_STOCHASTIC: {
            if (V <= 0 || (dtype != SV_F32 && dtype != SV_BF16)) return 0;
            if (T_or_N > 1024 || V > (1 << 22)) return 0;
            const sv::VocabPlan pl = sv::plan_vocab_stree(B, T_or_N, V, dtype);
            if ((size_t)B * pl.rows_per_seq * pl.nchunks >= (1u << 31)) return 0;
            return pl.bytes;
        }
        case SV_OP_VERIFY_STEP_CHAIN:
        case SV_OP_VERIFY_STEP_TREE_GREEDY: {
            const bool chain = op == SV_OP_VERIFY_STEP_CHAIN;
            if (V <= 0 || (dtype != SV_F32 && dtype != SV_BF16)) return 0;
            if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return 0;
            if (T_or_N > (chain ? 63 : 1024) || V >= (1 << 30) || (!chain && Hkv > 256)) return 0;
            const sv::VocabPlan pl = sv::plan_vocab(chain, B, T_or_N, V, dtype);
            if ((size_t)B * pl.rows_per_seq * pl.nchunks >= (1u << 31)) return 0;
            return sv::step_workspace_size(chain, B, T_or_N, V, dtype, Hq, Hkv, D);
        }
    }
    return 0;
}

sv_status sv_tree_attention(const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *prefix_lens, const int32_t *parents,
                            const int32_t *node_counts, int B, int T, int Hq, int Hkv, int D,
                            int S_max, float scale, void *out, int32_t *seq_status,
                            void *workspace, size_t workspace_bytes, sv_stream_t stream) {
    if (!q || !k_cache || !v_cache || !prefix_lens || !out) return SV_ERR_INVALID_ARG;
    if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || S_max < T) return SV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || !(scale > 0.f) || !std::isfinite(scale)) return SV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return SV_ERR_INVALID_ARG;
    if ((long long)B * Hkv * S_max >= (1LL << 31)) return SV_ERR_UNSUPPORTED;
    sv::AttnPlan pl;
    const sv_status st = sv::plan_attention(B, T, Hq, Hkv, D, S_max, &pl);
    if (st != SV_OK) return st;
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SV_ERR_WORKSPACE;
    sv::AttnArgs a{q,   k_cache, v_cache, prefix_lens, parents,    B,       T, Hq, Hkv, D,
                   S_max, scale, out,  seq_status, nullptr, 0, 0, 0, node_counts};
    return sv::launch_tree_attention(a, pl, workspace, as_stream(stream));
}

static bool valid_page_size(int ps) {
    // a power of two from 8 (one swizzle atom of rows) up, or a multiple of the 128-key tile
    return ps >= 8 && ((ps & (ps - 1)) == 0 || ps % 128 == 0);
}

sv_status sv_tree_attention_paged(const void *q, const void *k_pages, const void *v_pages,
                                  const int32_t *block_table, int max_pages, int num_pages,
                                  int page_size, const int32_t *prefix_lens,
                                  const int32_t *parents, const int32_t *node_counts, int B,
                                  int T, int Hq, int Hkv, int D, float scale, void *out,
                                  int32_t *seq_status, void *workspace, size_t workspace_bytes,
                                  sv_stream_t stream) {
    if (!q || !k_pages || !v_pages || !block_table || !prefix_lens || !out) return SV_ERR_INVALID_ARG;
    if (B <= 0 || T <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_pages <= 0 || num_pages <= 0)
        return SV_ERR_INVALID_ARG;
    if (!valid_page_size(page_size)) return SV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || !(scale > 0.f) || !std::isfinite(scale)) return SV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
        return SV_ERR_INVALID_ARG;
    const long long S_max = (long long)max_pages * page_size;
    if (S_max < T) return SV_ERR_INVALID_ARG;
    if ((long long)num_pages * Hkv * page_size >= (1LL << 31) || S_max >= (1LL << 30))
        return SV_ERR_UNSUPPORTED;
    sv::AttnPlan pl;
    const sv_status st = sv::plan_attention(B, T, Hq, Hkv, D, (int)S_max, &pl);
    if (st != SV_OK) return st;
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SV_ERR_WORKSPACE;
    sv::AttnArgs a{q,  k_pages, v_pages, prefix_lens, parents,     B,         T,        Hq,
                   Hkv, D,      (int)S_max, scale,     out,         seq_status, block_table,
                   max_pages, num_pages, page_size, node_counts};
    return sv::launch_tree_attention(a, pl, workspace, as_stream(stream));
}

sv_status sv_verify_chain(const void *target_logits, const void *draft_logits, sv_dtype dtype,
                          const int32_t *draft_tokens, const int32_t *draft_lens,
                          const float *u_accept, const float *u_sample, int B, int N, int V,
                          int32_t *accepted_len, int32_t *out_tokens, float *probs_out,
                          int32_t *seq_status, void *workspace, size_t workspace_bytes,
                          sv_stream_t stream) {
    if (!target_logits || !draft_logits || !draft_tokens || !u_accept || !u_sample ||
        !accepted_len || !out_tokens)
        return SV_ERR_INVALID_ARG;
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
    if (B <= 0 || N <= 0 || V <= 0) return SV_ERR_INVALID_ARG;
    if (!aligned16(target_logits) || !aligned16(draft_logits)) return SV_ERR_INVALID_ARG;
    if (N > 63 || V >= (1 << 30)) return SV_ERR_UNSUPPORTED;
    const sv::VocabPlan pl = sv::plan_vocab(true, B, N, V, dtype);
    if ((size_t)B * pl.rows_per_seq * pl.nchunks >= (1u << 31)) return SV_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SV_ERR_WORKSPACE;
    sv::ChainArgs a{target_logits, draft_logits, draft_tokens, draft_lens, u_accept, u_sample,
                    B,             N,            V,            accepted_len, out_tokens,
                    probs_out,     seq_status};
    return sv::launch_verify_chain(a, dtype, pl, workspace, as_stream(stream));
}

sv_status sv_verify_tree_greedy(const void *target_logits, sv_dtype dtype,
                                const int32_t *node_tokens, const int32_t *parents,
                                const int32_t *node_counts, int B, int T, int V,
                                int32_t *accepted_len, int32_t *path_nodes, int32_t *out_tokens,
                                int32_t *seq_status, void *workspace, size_t workspace_bytes,
                                sv_stream_t stream) {
    if (!target_logits || !node_tokens || !accepted_len || !path_nodes || !out_tokens)
        return SV_ERR_INVALID_ARG;
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
    if (B <= 0 || T <= 0 || V <= 0) return SV_ERR_INVALID_ARG;
    if (!aligned16(target_logits)) return SV_ERR_INVALID_ARG;
    if (T > 1024 || V >= (1 << 30)) return SV_ERR_UNSUPPORTED;
    const sv::VocabPlan pl = sv::plan_vocab(false, B, T, V, dtype);
    if ((size_t)B * pl.rows_per_seq * pl.nchunks >= (1u << 31)) return SV_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SV_ERR_WORKSPACE;
    sv::TreeArgs a{target_logits, node_tokens, parents,    node_counts, B, T, V, accepted_len,
                   path_nodes,    out_tokens,  seq_status};
    return sv::launch_verify_tree_greedy(a, dtype, pl, workspace, as_stream(stream));
}

sv_status sv_verify_tree_stochastic(const void *target_logits, const void *draft_logits,
                                    sv_dtype dtype, const int32_t *node_tokens,
                                    const int32_t *parents, const int32_t *node_counts,
                                    const float *u_accept, const float *u_sample, int B, int T,
                                    int V,
                                    int32_t *accepted_len, int32_t *path_nodes, int32_t *out_tokens,
                                    int32_t *seq_status, void *workspace, size_t workspace_bytes,
                                    sv_stream_t stream) {
    if (!target_logits || !draft_logits || !node_tokens || !u_accept || !u_sample ||
        !accepted_len || !path_nodes || !out_tokens)
        return SV_ERR_INVALID_ARG;
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
    if (B <= 0 || T <= 0 || V <= 0) return SV_ERR_INVALID_ARG;
    if (!aligned16(target_logits) || !aligned16(draft_logits)) return SV_ERR_INVALID_ARG;
    if (T > 1024 || V > (1 << 22)) return SV_ERR_UNSUPPORTED;
    const sv::VocabPlan pl = sv::plan_vocab_stree(B, T, V, dtype);
    if ((size_t)B * pl.rows_per_seq * pl.nchunks >= (1u << 31)) return SV_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SV_ERR_WORKSPACE;
    sv::STreeArgs a{target_logits, draft_logits, node_tokens, parents,    node_counts, u_accept,
                    u_sample,      B,            T,           V,          accepted_len, path_nodes,
                    out_tokens,    seq_status};
    return sv::launch_verify_tree_stochastic(a, dtype, pl, workspace, as_stream(stream));
}

sv_status sv_compact_kv(void *k_cache, void *v_cache, const int32_t *prefix_lens,
                        int32_t *new_kv_lens, const int32_t *path_nodes, int path_stride,
                        const int32_t *accepted_len, int B, int Hkv, int D, int S_max,
                        int32_t *seq_status, sv_stream_t stream) {
    if (!k_cache || !v_cache || !prefix_lens || !new_kv_lens || !accepted_len)
        return SV_ERR_INVALID_ARG;
    if (B <= 0 || Hkv <= 0 || D <= 0 || S_max <= 0) return SV_ERR_INVALID_ARG;
    if (path_nodes && path_stride <= 0) return SV_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return SV_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256) return SV_ERR_UNSUPPORTED;
    sv::CompactArgs a{k_cache, v_cache, prefix_lens, new_kv_lens, path_nodes, path_stride,
                      accepted_len, B, Hkv, D, S_max, seq_status, nullptr, 0, 0};
    return sv::launch_compact_kv(a, as_stream(stream));
}

sv_status sv_compact_kv_paged(void *k_pages, void *v_pages, const int32_t *block_table,
                              int max_pages, int num_pages, int page_size,
                              const int32_t *prefix_lens, int32_t *new_kv_lens,
                              const int32_t *path_nodes, int path_stride,
                              const int32_t *accepted_len, int B, int Hkv, int D,
                              int32_t *seq_status, sv_stream_t stream) {
    if (!k_pages || !v_pages || !block_table || !prefix_lens || !new_kv_lens || !accepted_len)
        return SV_ERR_INVALID_ARG;
    if (B <= 0 || Hkv <= 0 || D <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0)
        return SV_ERR_INVALID_ARG;
    if (path_nodes && path_stride <= 0) return SV_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages)) return SV_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256) return SV_ERR_UNSUPPORTED;
    const long long S_max = (long long)max_pages * page_size;
    if (S_max >= (1LL << 30) || (long long)num_pages * Hkv * page_size >= (1LL << 31))
        return SV_ERR_UNSUPPORTED;
    sv::CompactArgs a{k_pages, v_pages,    prefix_lens, new_kv_lens, path_nodes, path_stride,
                      accepted_len, B, Hkv, D, (int)S_max, seq_status, block_table, max_pages,
                      page_size};
    a.num_pages = num_pages;
    return sv::launch_compact_kv(a, as_stream(stream));
}

static bool page_tables_ok(int B, int page_size, int max_pages, int num_pages) {
    return B <= 4096 && (long long)max_pages * page_size < (1LL << 30) &&
           (long long)B * max_pages < (1LL << 31) && (long long)num_pages * page_size < (1LL << 31);
}

sv_status sv_build_block_tables(const int32_t *prefix_lens, const int32_t *new_lens,
                                const int32_t *page_counts, const int32_t *free_pages,
                                const int32_t *free_count, int B, int page_size, int max_pages,
                                int num_pages, int num_rows, int32_t *block_table,
                                int32_t *row_starts, int32_t *slot_map, int32_t *new_page_counts,
                                int32_t *new_free_count, int32_t *seq_status, sv_stream_t stream) {
    if (!prefix_lens || !new_lens || !page_counts || !free_pages || !free_count || !block_table ||
        !row_starts || !slot_map || !new_page_counts || !new_free_count)
        return SV_ERR_INVALID_ARG;
    if (B <= 0 || page_size <= 0 || max_pages <= 0 || num_pages <= 0 || num_rows <= 0)
        return SV_ERR_INVALID_ARG;
    // the CTAs read the old counts while one of them writes the new ones
    if (new_page_counts == page_counts || new_free_count == free_count) return SV_ERR_INVALID_ARG;
    if (!page_tables_ok(B, page_size, max_pages, num_pages) || num_rows >= (1 << 30))
        return SV_ERR_UNSUPPORTED;
    sv::BuildTablesArgs a{prefix_lens, new_lens,    page_counts, free_pages,      free_count,
                          B,           page_size,   max_pages,   num_pages,       num_rows,
                          block_table, row_starts,  slot_map,    new_page_counts, new_free_count,
                          seq_status};
    return sv::launch_build_tables(a, as_stream(stream));
}

sv_status sv_release_pages(const int32_t *keep_lens, const int32_t *page_counts,
                           const int32_t *block_table, int32_t *free_pages,
                           const int32_t *free_count, int B, int page_size, int max_pages,
                           int num_pages, int32_t *new_page_counts, int32_t *new_free_count,
                           int32_t *seq_status, sv_stream_t stream) {
    if (!keep_lens || !page_counts || !block_table || !free_pages || !free_count ||
        !new_page_counts || !new_free_count)
        return SV_ERR_INVALID_ARG;
    if (B <= 0 || page_size <= 0 || max_pages <= 0 || num_pages <= 0) return SV_ERR_INVALID_ARG;
    if (new_page_counts == page_counts || new_free_count == free_count) return SV_ERR_INVALID_ARG;
    if (!page_tables_ok(B, page_size, max_pages, num_pages)) return SV_ERR_UNSUPPORTED;
    sv::ReleasePagesArgs a{keep_lens, page_counts, block_table, free_pages,
                           free_count, B,          page_size,   max_pages,
                           num_pages, new_page_counts, new_free_count, seq_status};
    return sv::launch_release_pages(a, as_stream(stream));
}

sv_status sv_append_kv_paged(const void *k_new, const void *v_new, sv_dtype dtype,
                             long long k_stride, long long v_stride, const int32_t *slot_map,
                             int num_rows, int Hkv, int D, int page_size, int num_pages,
                             void *k_pages, void *v_pages, int32_t *row_status,
                             sv_stream_t stream) {
    if (!k_new || !v_new || !slot_map || !k_pages || !v_pages) return SV_ERR_INVALID_ARG;
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
    if (num_rows <= 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0)
        return SV_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_pages) || !aligned16(v_pages))
        return SV_ERR_INVALID_ARG;
    const long long per16 = dtype == SV_F32 ? 4 : 8, row = (long long)Hkv * D;
    if (k_stride < row || v_stride < row || k_stride % per16 != 0 || v_stride % per16 != 0)
        return SV_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256 || row >= (1LL << 30) || num_rows >= (1 << 30) ||
        (long long)num_pages * Hkv * page_size >= (1LL << 31))
        return SV_ERR_UNSUPPORTED;
    sv::AppendArgs a{k_new, v_new, k_stride,  v_stride,  slot_map, num_rows,
                     Hkv,   D,     page_size, num_pages, k_pages,  v_pages, row_status};
    return sv::launch_append_kv(a, dtype, as_stream(stream));
}

}  // extern "C"

// The chunk attention over pages in bf16 or, with k_params, held in 4 bits.
static sv_status chunk_attention(const void *q, long long q_stride, const void *k_pages, const void *v_pages,
                                 const int32_t *block_table, int max_pages, int num_pages, int page_size,
                                 const int32_t *prefix_lens, const int32_t *row_starts, int B, int num_rows, int Hq,
                                 int Hkv, int D, float scale, int window, void *out, float *lse, int32_t *seq_status,
                                 void *workspace, size_t workspace_bytes, sv_stream_t stream, const void *k_params,
                                 const void *v_params, const int32_t *parents) {
    if (!q || !k_pages || !v_pages || !block_table || !prefix_lens || !row_starts || !out)
        return SV_ERR_INVALID_ARG;
    if (B <= 0 || num_rows <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || max_pages <= 0 || num_pages <= 0 ||
        window < 0)
        return SV_ERR_INVALID_ARG;
    if (!valid_page_size(page_size)) return SV_ERR_INVALID_ARG;
    if (Hq % Hkv != 0 || !(scale > 0.f) || !std::isfinite(scale)) return SV_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(out))
        return SV_ERR_INVALID_ARG;
    if (q_stride < (long long)Hq * D || q_stride % 8 != 0 || out == q) return SV_ERR_INVALID_ARG;
    if (B > 4096 || num_rows >= (1 << 30) || (long long)Hq * D >= (1LL << 30) || q_stride >= (1LL << 38) ||
        (long long)max_pages * page_size >= (1LL << 30) || (long long)B * max_pages >= (1LL << 31) ||
        (long long)num_pages * Hkv * page_size >= (1LL << 31))
        return SV_ERR_UNSUPPORTED;
    sv::ChunkPlan pl;
    const sv_status st = sv::plan_chunk(Hq, Hkv, D, k_params != nullptr, &pl);
    if (st != SV_OK) return st;
    if (!workspace || workspace_bytes < pl.bytes || !aligned16(workspace)) return SV_ERR_WORKSPACE;
    sv::ChunkArgs a{q,         q_stride,    k_pages,    v_pages, block_table, max_pages,
                    num_pages, page_size,   prefix_lens, row_starts, B,       num_rows,
                    Hq,        Hkv,         D,          scale,   window,      out,
                    lse,       seq_status,  k_params,   v_params, parents};
    return sv::launch_chunk_attention(a, pl, workspace, as_stream(stream));
}

extern "C" {

sv_status sv_chunk_attention_paged(const void *q, long long q_stride, const void *k_pages,
                                   const void *v_pages, const int32_t *block_table, int max_pages,
                                   int num_pages, int page_size, const int32_t *prefix_lens,
                                   const int32_t *row_starts, int B, int num_rows, int Hq, int Hkv,
                                   int D, float scale, int window, void *out, float *lse,
                                   int32_t *seq_status, void *workspace, size_t workspace_bytes,
                                   sv_stream_t stream) {
    return chunk_attention(q, q_stride, k_pages, v_pages, block_table, max_pages, num_pages, page_size, prefix_lens,
                           row_starts, B, num_rows, Hq, Hkv, D, scale, window, out, lse, seq_status, workspace,
                           workspace_bytes, stream, nullptr, nullptr, nullptr);
}

sv_status sv_chunk_attention_quant(const void *q, long long q_stride, const void *k_codes,
                                   const void *k_params, const void *v_codes, const void *v_params,
                                   const int32_t *block_table, int max_pages, int num_pages,
                                   int page_size, const int32_t *prefix_lens,
                                   const int32_t *row_starts, const int32_t *parents, int B,
                                   int num_rows, int Hq, int Hkv, int D, float scale, int window,
                                   void *out, float *lse, int32_t *seq_status, void *workspace,
                                   size_t workspace_bytes, sv_stream_t stream) {
    if (!k_params || !v_params || !aligned16(k_params) || !aligned16(v_params) || (parents && window > 0))
        return SV_ERR_INVALID_ARG;
    return chunk_attention(q, q_stride, k_codes, v_codes, block_table, max_pages, num_pages, page_size, prefix_lens,
                           row_starts, B, num_rows, Hq, Hkv, D, scale, window, out, lse, seq_status, workspace,
                           workspace_bytes, stream, k_params, v_params, parents);
}

sv_status sv_append_kv_quant(const void *k_new, const void *v_new, sv_dtype dtype,
                             long long k_stride, long long v_stride, const int32_t *slot_map,
                             int num_rows, int Hkv, int D, int page_size, int num_pages,
                             void *k_codes, void *k_params, void *v_codes, void *v_params,
                             int32_t *row_status, sv_stream_t stream) {
    if (!k_new || !v_new || !slot_map || !k_codes || !k_params || !v_codes || !v_params) return SV_ERR_INVALID_ARG;
    if (dtype != SV_F32 && dtype != SV_BF16) return SV_ERR_INVALID_ARG;
    if (num_rows <= 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages <= 0) return SV_ERR_INVALID_ARG;
    for (const void *p : {k_new, v_new, (const void *)k_codes, (const void *)k_params, (const void *)v_codes, (const void *)v_params})
        if (!aligned16(p)) return SV_ERR_INVALID_ARG;
    const long long per16 = dtype == SV_F32 ? 4 : 8, row = (long long)Hkv * D;
    if (k_stride < row || v_stride < row || k_stride % per16 != 0 || v_stride % per16 != 0) return SV_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || row >= (1LL << 30) || num_rows >= (1 << 30) || k_stride >= (1LL << 32) ||
        v_stride >= (1LL << 32) || (long long)num_pages * Hkv * page_size >= (1LL << 31))
        return SV_ERR_UNSUPPORTED;
    sv::AppendQuantArgs a{k_new,     v_new,     k_stride, v_stride, slot_map, num_rows, Hkv,       D,
                          page_size, num_pages, k_codes,  k_params, v_codes,  v_params, row_status};
    return sv::launch_append_quant(a, dtype, as_stream(stream));
}

sv_status sv_compact_kv_quant(void *k_codes, void *k_params, void *v_codes, void *v_params,
                              const int32_t *block_table, int max_pages, int num_pages,
                              int page_size, const int32_t *prefix_lens, int32_t *new_kv_lens,
                              const int32_t *path_nodes, int path_stride,
                              const int32_t *accepted_len, int B, int Hkv, int D,
                              int32_t *seq_status, sv_stream_t stream) {
    if (!k_codes || !k_params || !v_codes || !v_params || !block_table || !prefix_lens || !new_kv_lens || !accepted_len)
        return SV_ERR_INVALID_ARG;
    if (B <= 0 || Hkv <= 0 || D <= 0 || max_pages <= 0 || num_pages <= 0 || page_size <= 0) return SV_ERR_INVALID_ARG;
    if (path_nodes && path_stride <= 0) return SV_ERR_INVALID_ARG;
    if (!aligned16(k_codes) || !aligned16(k_params) || !aligned16(v_codes) || !aligned16(v_params))
        return SV_ERR_INVALID_ARG;
    const long long S_max = (long long)max_pages * page_size;
    if ((D != 64 && D != 128) || S_max >= (1LL << 30) || (long long)num_pages * Hkv * page_size >= (1LL << 31))
        return SV_ERR_UNSUPPORTED;
    sv::CompactQuantArgs a{k_codes,     k_params,    v_codes,    v_params,    block_table,  max_pages, num_pages,
                           page_size,   prefix_lens, new_kv_lens, path_nodes, path_stride,  accepted_len, B,
                           Hkv,         D,           (int)S_max, seq_status};
    return sv::launch_compact_quant(a, as_stream(stream));
}

sv_status sv_fork_tables(const int32_t *sources, const int32_t *targets, const int32_t *fork_lens,
                         const int32_t *page_counts, const int32_t *free_pages,
                         const int32_t *free_count, const int32_t *shares, int F, int B,
                         int page_size, int max_pages, int num_pages, int32_t *block_table,
                         int32_t *copies, int32_t *new_page_counts, int32_t *new_free_count,
                         int32_t *new_shares, int32_t *fork_status, sv_stream_t stream) {
    if (!sources || !targets || !fork_lens || !page_counts || !free_pages || !free_count || !shares || !block_table ||
        !copies || !new_page_counts || !new_free_count || !new_shares)
        return SV_ERR_INVALID_ARG;
    if (F <= 0 || B <= 0 || page_size <= 0 || max_pages <= 0 || num_pages <= 0) return SV_ERR_INVALID_ARG;
    // the CTAs read the old counts while some of them write the new ones
    if (new_page_counts == page_counts || new_free_count == free_count || new_shares == shares) return SV_ERR_INVALID_ARG;
    if (F > 4096 || !page_tables_ok(B, page_size, max_pages, num_pages)) return SV_ERR_UNSUPPORTED;
    sv::ForkArgs a{sources,   targets,   fork_lens,   page_counts, free_pages,      free_count,     shares,     F, B,
                   page_size, max_pages, num_pages,   block_table, copies,          new_page_counts, new_free_count,
                   new_shares, fork_status};
    return sv::launch_fork_tables(a, as_stream(stream));
}

sv_status sv_copy_pages(const int32_t *copies, int F, void *const *planes, const int *row_bytes,
                        int num_planes, int Hkv, int page_size, int num_pages,
                        int32_t *copy_status, sv_stream_t stream) {
    if (!copies || !planes || !row_bytes) return SV_ERR_INVALID_ARG;
    if (F <= 0 || num_planes <= 0 || Hkv <= 0 || page_size <= 0 || num_pages <= 0) return SV_ERR_INVALID_ARG;
    if (num_planes > sv::kMaxPlanes || F > (1 << 20) || (long long)num_pages * Hkv * page_size >= (1LL << 31))
        return SV_ERR_UNSUPPORTED;
    sv::CopyPagesArgs a{};
    for (int i = 0; i < num_planes; ++i) {
        if (!planes[i] || !aligned16(planes[i]) || row_bytes[i] <= 0 || row_bytes[i] % 4 != 0) return SV_ERR_INVALID_ARG;
        if (row_bytes[i] > 4096) return SV_ERR_UNSUPPORTED;
        a.planes[i] = planes[i];
        a.row_bytes[i] = row_bytes[i];
    }
    a.copies = copies;
    a.F = F;
    a.num_planes = num_planes;
    a.Hkv = Hkv;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.copy_status = copy_status;
    return sv::launch_copy_pages(a, as_stream(stream));
}

sv_status sv_release_shared_pages(const int32_t *keep_lens, const int32_t *page_counts,
                                  const int32_t *block_table, int32_t *free_pages,
                                  const int32_t *free_count, const int32_t *shares, int B,
                                  int page_size, int max_pages, int num_pages,
                                  int32_t *new_page_counts, int32_t *new_free_count,
                                  int32_t *new_shares, int32_t *seq_status, void *workspace,
                                  size_t workspace_bytes, sv_stream_t stream) {
    if (!keep_lens || !page_counts || !block_table || !free_pages || !free_count || !shares || !new_page_counts ||
        !new_free_count || !new_shares)
        return SV_ERR_INVALID_ARG;
    if (B <= 0 || page_size <= 0 || max_pages <= 0 || num_pages <= 0) return SV_ERR_INVALID_ARG;
    if (new_page_counts == page_counts || new_free_count == free_count || new_shares == shares) return SV_ERR_INVALID_ARG;
    if (!page_tables_ok(B, page_size, max_pages, num_pages)) return SV_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < ((size_t)num_pages + sv::kReleaseMaxWarps) * sizeof(int) || reinterpret_cast<uintptr_t>(workspace) % sizeof(int) != 0)
        return SV_ERR_WORKSPACE;
    sv::ReleaseSharedArgs a{keep_lens, page_counts, block_table,     free_pages,     free_count, shares,     B,
                            page_size, max_pages,   num_pages,       new_page_counts, new_free_count, new_shares, seq_status,
                            static_cast<int *>(workspace)};
    return sv::launch_release_shared(a, as_stream(stream));
}

}  // extern "C"
