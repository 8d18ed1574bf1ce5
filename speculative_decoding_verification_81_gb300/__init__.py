"""libspecverify: the target model's verification step of speculative
decoding on one GB300 (sm_103a) -- tree/chain verification attention,
full-vocabulary stochastic (chain and tree) and greedy (tree) acceptance, KV
compaction, the fused step that runs them side by side, the paged cache around
it (page tables, new rows, attention of prompt chunks), the same cache held in 4
bits and requests that share its pages -- as hand-written CUDA kernels behind a
C ABI (include/specverify.h), with this thin Python binding on top.
"""
from .api import (SV_BF16, SV_ERR_BAD_INPUT, SV_ERR_CUDA, SV_ERR_INVALID_ARG, SV_ERR_NO_PAGES,
                  SV_ERR_TIMEOUT, SV_ERR_UNSUPPORTED, SV_ERR_WORKSPACE, SV_F32, SV_OK, SV_OP_CHUNK_ATTENTION,
                  SV_OP_RELEASE_SHARED_PAGES,
                  SV_OP_TREE_ATTENTION,
                  SV_OP_VERIFY_CHAIN, SV_OP_VERIFY_STEP_CHAIN, SV_OP_VERIFY_STEP_TREE_GREEDY,
                  SV_OP_VERIFY_TREE_GREEDY, SV_OP_VERIFY_TREE_STOCHASTIC, SpecVerifyError, lib,
                  status_string, sv_append_kv_paged, sv_append_kv_quant, sv_build_block_tables,
                  sv_chunk_attention_paged, sv_chunk_attention_quant, sv_compact_kv,
                  sv_compact_kv_paged, sv_compact_kv_quant, sv_copy_pages, sv_fork_tables, sv_release_pages,
                  sv_release_shared_pages, sv_tree_attention,
                  sv_tree_attention_paged, sv_verify_chain, sv_verify_step_chain,
                  sv_verify_step_tree_greedy, sv_verify_tree_greedy, sv_verify_tree_stochastic,
                  sv_workspace_size, workspace)

__all__ = [
    "SV_BF16", "SV_F32", "SV_OK", "SV_ERR_BAD_INPUT", "SV_ERR_CUDA", "SV_ERR_INVALID_ARG",
    "SV_ERR_TIMEOUT", "SV_ERR_UNSUPPORTED", "SV_ERR_WORKSPACE", "SV_ERR_NO_PAGES",
    "SV_OP_TREE_ATTENTION",
    "SV_OP_VERIFY_CHAIN", "SV_OP_VERIFY_TREE_GREEDY", "SV_OP_VERIFY_TREE_STOCHASTIC",
    "SV_OP_VERIFY_STEP_CHAIN", "SV_OP_VERIFY_STEP_TREE_GREEDY",
    "SpecVerifyError", "lib", "status_string", "sv_compact_kv", "sv_compact_kv_paged",
    "sv_tree_attention", "sv_tree_attention_paged", "sv_verify_chain", "sv_verify_tree_greedy",
    "sv_verify_tree_stochastic", "sv_verify_step_chain", "sv_verify_step_tree_greedy",
    "SV_OP_CHUNK_ATTENTION", "sv_append_kv_paged", "sv_build_block_tables",
    "sv_chunk_attention_paged", "sv_release_pages",
    "SV_OP_RELEASE_SHARED_PAGES", "sv_append_kv_quant", "sv_chunk_attention_quant", "sv_compact_kv_quant",
    "sv_fork_tables", "sv_copy_pages", "sv_release_shared_pages",
    "sv_workspace_size", "workspace",
]
