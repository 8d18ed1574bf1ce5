"""Thin Python binding of libspecverify (ctypes).

Each function has the name of the C entry point it calls and only marshals
arguments: torch tensors on the GPU become device pointers, the current torch
stream becomes the launch stream, and a non-OK status becomes an exception.
Every step of the computation runs in the library's CUDA kernels; there is no
fallback.  If the library is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import warnings

import torch

from . import build as _build

SV_OK = 0
SV_ERR_INVALID_ARG = 1
SV_ERR_WORKSPACE = 2
SV_ERR_UNSUPPORTED = 3
SV_ERR_CUDA = 4
SV_ERR_TIMEOUT = 5
SV_ERR_BAD_INPUT = 6
SV_ERR_NO_PAGES = 7

SV_F32 = 0
SV_BF16 = 1

SV_OP_TREE_ATTENTION = 0
SV_OP_VERIFY_CHAIN = 1
SV_OP_VERIFY_TREE_GREEDY = 2
SV_OP_VERIFY_TREE_STOCHASTIC = 3
SV_OP_VERIFY_STEP_CHAIN = 4
SV_OP_VERIFY_STEP_TREE_GREEDY = 5
SV_OP_CHUNK_ATTENTION = 6
SV_OP_RELEASE_SHARED_PAGES = 7

EXPORTS = ("sv_workspace_size", "sv_tree_attention", "sv_verify_chain", "sv_verify_tree_greedy",
           "sv_compact_kv", "sv_status_string", "sv_version", "sv_verify_chain_noalloc",
           "sv_tree_attention_paged", "sv_compact_kv_paged", "sv_verify_tree_stochastic",
           "sv_verify_step_chain", "sv_verify_step_tree_greedy", "sv_build_block_tables",
           "sv_release_pages", "sv_append_kv_paged", "sv_chunk_attention_paged", "sv_append_kv_quant",
           "sv_chunk_attention_quant", "sv_compact_kv_quant", "sv_fork_tables", "sv_copy_pages",
           "sv_release_shared_pages")

# Length of the fixed scratch array behind sv_verify_chain_noalloc.
SV_NOALLOC_SCRATCH_BYTES = 4 << 20


class SpecVerifyError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB_PATH):
            raise ImportError(f"libspecverify.so is not built ({_build.LIB_PATH}); "
                              "run __graft_entry__.build() or python -m "
                              "speculative_decoding_verification_81_gb300.build")
        _lib = load(_build.LIB_PATH)
        _bind_to(_lib)
    return _lib


def use_library(path: str) -> ctypes.CDLL:
    """Route every call of this module to the library at `path` (a build of
    the same sources, e.g. the phase-stamped one of the ``phases`` tool)."""
    global _lib
    _lib = load(path)
    _bind_to(_lib)
    return _lib


_bind = None   # the marshalling extension, and the library it calls
_bound = None


def _load_bind(path):
    """The extension at `path`; None, with a warning, when it does not import."""
    name = f"{__package__}._sv_bind"
    try:
        loader = importlib.machinery.ExtensionFileLoader(name, path)
        module = importlib.util.module_from_spec(importlib.util.spec_from_file_location(name, path, loader=loader))
        loader.exec_module(module)
        return module
    except (ImportError, OSError) as e:
        warnings.warn(f"the paged-cache calls go without their extension: {e}")
        return None


def _bind_to(L):
    global _bind, _bound
    path = _build.bind_path()
    if _bind is None and os.path.exists(path):
        _bind = _load_bind(path)
    if _bind is not None:
        def addresses(*names):
            return (ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in names)
        _bind.use(*addresses("sv_build_block_tables", "sv_release_pages", "sv_append_kv_paged", "sv_chunk_attention_paged"))
        _bind.use_quant(*addresses("sv_append_kv_quant", "sv_chunk_attention_quant", "sv_compact_kv_quant",
                                   "sv_fork_tables", "sv_copy_pages", "sv_release_shared_pages", "sv_workspace_size"))
        _bound = L


def _native():
    """The extension that marshals the plain form of the paged-cache calls, when
    it is built and calls the library in use.  Its functions return None, having
    launched nothing, for every call they do not take: the checks below then
    name what is wrong with it, or make it."""
    return _bind if lib() is _bound else None


def load(path: str) -> ctypes.CDLL:
    """Load a build of libspecverify and declare its entry points' C types."""
    L = ctypes.CDLL(path)
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.sv_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
    L.sv_workspace_size.restype = Z
    L.sv_tree_attention.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, ctypes.c_float, P, P, P,
                                    Z, P]
    L.sv_verify_chain.argtypes = [P, P, I, P, P, P, P, I, I, I, P, P, P, P, P, Z, P]
    L.sv_verify_tree_greedy.argtypes = [P, I, P, P, P, I, I, I, P, P, P, P, P, Z, P]
    L.sv_verify_chain_noalloc.argtypes = [P, P, I, P, P, P, I, I, I, P, P, P, P, P]
    L.sv_compact_kv.argtypes = [P, P, P, P, P, I, P, I, I, I, I, P, P]
    L.sv_tree_attention_paged.argtypes = [P, P, P, P, I, I, I, P, P, P, I, I, I, I, I,
                                          ctypes.c_float, P, P, P, Z, P]
    L.sv_compact_kv_paged.argtypes = [P, P, P, I, I, I, P, P, P, I, P, I, I, I, P, P]
    L.sv_verify_tree_stochastic.argtypes = [P, P, I, P, P, P, P, P, I, I, I, P, P, P, P, P, Z,
                                            P]
    F = ctypes.c_float
    L.sv_verify_step_chain.argtypes = [P, P, P, P, I, I, I, I, F, P, P, P, P, I, P, P, P, P, I, I,
                                       I, P, P, P, P, P, P, Z, P]
    L.sv_verify_step_tree_greedy.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, I, P,
                                             I, P, P, P, P, P, P, Z, P]
    Q = ctypes.c_longlong
    L.sv_build_block_tables.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, P, P]
    L.sv_release_pages.argtypes = [P, P, P, P, P, I, I, I, I, P, P, P, P]
    L.sv_append_kv_paged.argtypes = [P, P, I, Q, Q, P, I, I, I, I, I, P, P, P, P]
    L.sv_chunk_attention_paged.argtypes = [P, Q, P, P, P, I, I, I, P, P, I, I, I, I, I, F, I, P, P, P,
                                           P, Z, P]
    L.sv_append_kv_quant.argtypes = [P, P, I, Q, Q, P, I, I, I, I, I, P, P, P, P, P, P]
    L.sv_chunk_attention_quant.argtypes = [P, Q, P, P, P, P, P, I, I, I, P, P, P, I, I, I, I, I, F, I, P, P, P,
                                           P, Z, P]
    L.sv_compact_kv_quant.argtypes = [P, P, P, P, P, I, I, I, P, P, P, I, P, I, I, I, P, P]
    L.sv_fork_tables.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, P, P]
    L.sv_copy_pages.argtypes = [P, I, P, P, I, I, I, I, P, P]
    L.sv_release_shared_pages.argtypes = [P, P, P, P, P, P, I, I, I, I, P, P, P, P, P, Z, P]
    for fn in ("sv_build_block_tables", "sv_release_pages", "sv_append_kv_paged",
               "sv_chunk_attention_paged", "sv_append_kv_quant", "sv_chunk_attention_quant",
               "sv_compact_kv_quant", "sv_fork_tables", "sv_copy_pages", "sv_release_shared_pages",
               "sv_tree_attention", "sv_verify_chain", "sv_verify_tree_greedy", "sv_compact_kv",
               "sv_verify_chain_noalloc", "sv_tree_attention_paged", "sv_compact_kv_paged",
               "sv_verify_tree_stochastic", "sv_verify_step_chain", "sv_verify_step_tree_greedy"):
        getattr(L, fn).restype = I
    L.sv_status_string.argtypes = [I]
    L.sv_status_string.restype = ctypes.c_char_p
    L.sv_version.argtypes = []
    L.sv_version.restype = I
    return L


def status_string(status: int) -> str:
    return lib().sv_status_string(int(status)).decode()


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, rc):
    if rc != SV_OK:
        raise SpecVerifyError(fn, rc)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float32:
        return SV_F32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _on_device(t):
    return t.is_cuda


def _req(t, name, dtype=None, ndim=None):
    if not _on_device(t) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    return t


def _shape(t, name, shape):
    """The kernels index every array by the call's sizes: a tensor of another
    shape would be read or written out of bounds, so it is refused here."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _opt(t, name, dtype, shape):
    """An optional array (an input or a caller-provided output): checked when given."""
    if t is not None:
        _shape(_req(t, name, dtype, len(shape)), name, shape)
    return t


def sv_workspace_size(op: int, B: int, T_or_N: int, V: int = 0, dtype: int = SV_BF16, Hq: int = 0,
                      Hkv: int = 0, D: int = 0) -> int:
    return int(lib().sv_workspace_size(op, B, T_or_N, V, dtype, Hq, Hkv, D))


_ws_cache: dict = {}


def workspace(op: int, B: int, T_or_N: int, V: int = 0, dtype: int = SV_BF16, Hq: int = 0,
              Hkv: int = 0, D: int = 0, device=None) -> torch.Tensor:
    """A zero-filled workspace for one call shape, cached per (shape, device).
    Calls sharing it must not overlap on the GPU."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    key = (op, B, T_or_N, V, dtype, Hq, Hkv, D, str(device))
    ws = _ws_cache.get(key)
    if ws is None:
        n = sv_workspace_size(op, B, T_or_N, V, dtype, Hq, Hkv, D)
        if n == 0:
            raise SpecVerifyError("sv_workspace_size", SV_ERR_UNSUPPORTED)
        ws = torch.zeros(n, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def sv_tree_attention(q, k_cache, v_cache, prefix_lens, parents=None, scale=None, out=None,
                      seq_status=None, ws=None, stream=None, node_counts=None):
    """q [B,T,Hq,D] bf16; k_cache/v_cache [B,Hkv,S_max,D] bf16; prefix_lens [B] int32;
    parents [B,T] int32 or None (chain); node_counts [B] int32 or None (every
    sequence has T nodes).  Returns out [B,T,Hq,D] bf16."""
    _req(q, "q", torch.bfloat16, 4)
    _req(k_cache, "k_cache", torch.bfloat16, 4)
    _req(v_cache, "v_cache", torch.bfloat16, 4)
    _req(prefix_lens, "prefix_lens", torch.int32, 1)
    B, T, Hq, D = q.shape
    _, Hkv, S_max, _ = k_cache.shape
    _shape(k_cache, "k_cache", (B, Hkv, S_max, D))
    _shape(v_cache, "v_cache", k_cache.shape)
    _shape(prefix_lens, "prefix_lens", (B,))
    _opt(parents, "parents", torch.int32, (B, T))
    _opt(node_counts, "node_counts", torch.int32, (B,))
    _opt(out, "out", torch.bfloat16, q.shape)
    _opt(seq_status, "seq_status", torch.int32, (B,))
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(SV_OP_TREE_ATTENTION, B, T, Hq=Hq, Hkv=Hkv, D=D, device=q.device)
    rc = lib().sv_tree_attention(_p(q), _p(k_cache), _p(v_cache), _p(prefix_lens), _p(parents),
                                 _p(node_counts), B, T, Hq, Hkv, D, S_max, float(scale), _p(out),
                                 _p(seq_status), _p(ws), ws.numel(), _stream(stream))
    _check("sv_tree_attention", rc)
    return out


def sv_tree_attention_paged(q, k_pages, v_pages, block_table, prefix_lens, parents=None,
                            scale=None, out=None, seq_status=None, ws=None, stream=None,
                            node_counts=None):
    """q [B,T,Hq,D] bf16; k_pages/v_pages [num_pages,Hkv,page_size,D] bf16;
    block_table [B,max_pages] int32; prefix_lens [B] int32; parents [B,T] int32
    or None (chain).  Returns out [B,T,Hq,D] bf16."""
    _req(q, "q", torch.bfloat16, 4)
    _req(k_pages, "k_pages", torch.bfloat16, 4)
    _req(v_pages, "v_pages", torch.bfloat16, 4)
    _req(block_table, "block_table", torch.int32, 2)
    _req(prefix_lens, "prefix_lens", torch.int32, 1)
    B, T, Hq, D = q.shape
    num_pages, Hkv, page_size, _ = k_pages.shape
    max_pages = block_table.shape[1]
    _shape(k_pages, "k_pages", (num_pages, Hkv, page_size, D))
    _shape(v_pages, "v_pages", k_pages.shape)
    _shape(block_table, "block_table", (B, max_pages))
    _shape(prefix_lens, "prefix_lens", (B,))
    _opt(parents, "parents", torch.int32, (B, T))
    _opt(node_counts, "node_counts", torch.int32, (B,))
    _opt(out, "out", torch.bfloat16, q.shape)
    _opt(seq_status, "seq_status", torch.int32, (B,))
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = workspace(SV_OP_TREE_ATTENTION, B, T, Hq=Hq, Hkv=Hkv, D=D, device=q.device)
    rc = lib().sv_tree_attention_paged(_p(q), _p(k_pages), _p(v_pages), _p(block_table), max_pages,
                                       num_pages, page_size, _p(prefix_lens), _p(parents),
                                       _p(node_counts), B, T, Hq, Hkv, D, float(scale), _p(out),
                                       _p(seq_status), _p(ws), ws.numel(), _stream(stream))
    _check("sv_tree_attention_paged", rc)
    return out


def _chain_shapes(B, N, V, draft_logits, draft_tokens, u_accept, u_sample, accepted_len,
                  out_tokens, probs_out, seq_status):
    _shape(draft_logits, "draft_logits", (B, N, V))
    _shape(draft_tokens, "draft_tokens", (B, N))
    _shape(u_accept, "u_accept", (B, N))
    _shape(u_sample, "u_sample", (B,))
    _opt(accepted_len, "accepted_len", torch.int32, (B,))
    _opt(out_tokens, "out_tokens", torch.int32, (B, N + 1))
    _opt(probs_out, "probs_out", torch.float32, (B, N, 2))
    _opt(seq_status, "seq_status", torch.int32, (B,))


def sv_verify_chain(target_logits, draft_logits, draft_tokens, u_accept, u_sample,
                    accepted_len=None, out_tokens=None, probs_out=None, seq_status=None, ws=None,
                    stream=None, draft_lens=None):
    """target [B,N+1,V], draft [B,N,V] (bf16 or f32); draft_tokens [B,N] int32;
    u_accept [B,N] f32; u_sample [B] f32; draft_lens [B] int32 or None (every
    sequence drafted N tokens).  Returns (accepted_len [B], out_tokens [B,N+1])."""
    _req(target_logits, "target_logits", None, 3)
    _req(draft_logits, "draft_logits", target_logits.dtype, 3)
    _req(draft_tokens, "draft_tokens", torch.int32, 2)
    _req(u_accept, "u_accept", torch.float32, 2)
    _req(u_sample, "u_sample", torch.float32, 1)
    dt = _dtype_code(target_logits)
    B, N1, V = target_logits.shape
    N = N1 - 1
    _chain_shapes(B, N, V, draft_logits, draft_tokens, u_accept, u_sample, accepted_len,
                  out_tokens, probs_out, seq_status)
    _opt(draft_lens, "draft_lens", torch.int32, (B,))
    dev = target_logits.device
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(B, N + 1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(SV_OP_VERIFY_CHAIN, B, N, V, dt, device=dev)
    rc = lib().sv_verify_chain(_p(target_logits), _p(draft_logits), dt, _p(draft_tokens),
                               _p(draft_lens), _p(u_accept), _p(u_sample), B, N, V, _p(accepted_len),
                               _p(out_tokens), _p(probs_out), _p(seq_status), _p(ws), ws.numel(),
                               _stream(stream))
    _check("sv_verify_chain", rc)
    return accepted_len, out_tokens


def _tree_shapes(B, T, node_tokens, parents, node_counts, accepted_len, path_nodes, out_tokens,
                 seq_status):
    _shape(node_tokens, "node_tokens", (B, T))
    _opt(parents, "parents", torch.int32, (B, T))
    _opt(node_counts, "node_counts", torch.int32, (B,))
    _opt(accepted_len, "accepted_len", torch.int32, (B,))
    _opt(path_nodes, "path_nodes", torch.int32, (B, T))
    _opt(out_tokens, "out_tokens", torch.int32, (B, T))
    _opt(seq_status, "seq_status", torch.int32, (B,))


def sv_verify_tree_greedy(target_logits, node_tokens, parents, accepted_len=None, path_nodes=None,
                          out_tokens=None, seq_status=None, ws=None, stream=None,
                          node_counts=None):
    """target [B,T,V] (bf16 or f32); node_tokens, parents [B,T] int32 (parents
    None: a chain, i.e. greedy chain verification); node_counts [B] int32 or
    None (every sequence has T nodes).
    Returns (accepted_len [B], path_nodes [B,T], out_tokens [B,T])."""
    _req(target_logits, "target_logits", None, 3)
    _req(node_tokens, "node_tokens", torch.int32, 2)
    dt = _dtype_code(target_logits)
    B, T, V = target_logits.shape
    _tree_shapes(B, T, node_tokens, parents, node_counts, accepted_len, path_nodes, out_tokens,
                 seq_status)
    dev = target_logits.device
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=dev)
    if path_nodes is None:
        path_nodes = torch.empty(B, T, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(B, T, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(SV_OP_VERIFY_TREE_GREEDY, B, T, V, dt, device=dev)
    rc = lib().sv_verify_tree_greedy(_p(target_logits), dt, _p(node_tokens), _p(parents),
                                     _p(node_counts), B, T, V,
                                     _p(accepted_len), _p(path_nodes), _p(out_tokens),
                                     _p(seq_status), _p(ws), ws.numel(), _stream(stream))
    _check("sv_verify_tree_greedy", rc)
    return accepted_len, path_nodes, out_tokens


def sv_verify_tree_stochastic(target_logits, draft_logits, node_tokens, parents, u_accept,
                              u_sample, accepted_len=None, path_nodes=None, out_tokens=None,
                              seq_status=None, ws=None, stream=None, node_counts=None):
    """target, draft [B,T,V] (bf16 or f32; draft row u: the distribution u's
    children were drawn from); node_tokens, parents [B,T] int32 (parents None:
    a chain); u_accept [B,T] f32; u_sample [B] f32; node_counts [B] int32 or
    None (every sequence has T nodes).
    Returns (accepted_len [B], path_nodes [B,T], out_tokens [B,T])."""
    _req(target_logits, "target_logits", None, 3)
    _req(draft_logits, "draft_logits", target_logits.dtype, 3)
    _req(node_tokens, "node_tokens", torch.int32, 2)
    _req(u_accept, "u_accept", torch.float32, 2)
    _req(u_sample, "u_sample", torch.float32, 1)
    dt = _dtype_code(target_logits)
    B, T, V = target_logits.shape
    _shape(draft_logits, "draft_logits", (B, T, V))
    _shape(u_accept, "u_accept", (B, T))
    _shape(u_sample, "u_sample", (B,))
    _tree_shapes(B, T, node_tokens, parents, node_counts, accepted_len, path_nodes, out_tokens,
                 seq_status)
    dev = target_logits.device
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=dev)
    if path_nodes is None:
        path_nodes = torch.empty(B, T, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(B, T, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(SV_OP_VERIFY_TREE_STOCHASTIC, B, T, V, dt, device=dev)
    rc = lib().sv_verify_tree_stochastic(_p(target_logits), _p(draft_logits), dt, _p(node_tokens),
                                         _p(parents), _p(node_counts), _p(u_accept),
                                         _p(u_sample), B, T, V,
                                         _p(accepted_len), _p(path_nodes), _p(out_tokens),
                                         _p(seq_status), _p(ws), ws.numel(), _stream(stream))
    _check("sv_verify_tree_stochastic", rc)
    return accepted_len, path_nodes, out_tokens


def _attn_shapes(q, k_cache, v_cache, prefix_lens, out, seq_status):
    _req(q, "q", torch.bfloat16, 4)
    _req(k_cache, "k_cache", torch.bfloat16, 4)
    _req(v_cache, "v_cache", torch.bfloat16, 4)
    _req(prefix_lens, "prefix_lens", torch.int32, 1)
    B, T, Hq, D = q.shape
    _, Hkv, S_max, _ = k_cache.shape
    _shape(k_cache, "k_cache", (B, Hkv, S_max, D))
    _shape(v_cache, "v_cache", k_cache.shape)
    _shape(prefix_lens, "prefix_lens", (B,))
    _opt(out, "attn_out", torch.bfloat16, q.shape)
    _opt(seq_status, "attn_status", torch.int32, (B,))
    return B, T, Hq, D, Hkv, S_max


def sv_verify_step_chain(q, k_cache, v_cache, prefix_lens, target_logits, draft_logits,
                         draft_tokens, u_accept, u_sample, attn_out=None, accepted_len=None,
                         out_tokens=None, new_kv_lens=None, probs_out=None, attn_status=None,
                         verify_status=None, draft_lens=None, scale=None, ws=None, stream=None):
    """The fused chain step.  q [B,N+1,Hq,D] bf16; caches [B,Hkv,S_max,D] bf16;
    prefix_lens [B] int32; logits and draws as sv_verify_chain.
    Returns (attn_out, accepted_len, out_tokens, new_kv_lens)."""
    B, T, Hq, D, Hkv, S_max = _attn_shapes(q, k_cache, v_cache, prefix_lens, attn_out,
                                            attn_status)
    _req(target_logits, "target_logits", None, 3)
    _req(draft_logits, "draft_logits", target_logits.dtype, 3)
    _req(draft_tokens, "draft_tokens", torch.int32, 2)
    _req(u_accept, "u_accept", torch.float32, 2)
    _req(u_sample, "u_sample", torch.float32, 1)
    dt = _dtype_code(target_logits)
    N = T - 1
    V = target_logits.shape[2]
    _shape(target_logits, "target_logits", (B, T, V))
    _chain_shapes(B, N, V, draft_logits, draft_tokens, u_accept, u_sample, accepted_len,
                  out_tokens, probs_out, verify_status)
    _opt(draft_lens, "draft_lens", torch.int32, (B,))
    _opt(new_kv_lens, "new_kv_lens", torch.int32, (B,))
    dev = q.device
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if attn_out is None:
        attn_out = torch.empty_like(q)
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(B, N + 1, dtype=torch.int32, device=dev)
    if new_kv_lens is None:
        new_kv_lens = torch.empty_like(prefix_lens)
    if ws is None:
        ws = workspace(SV_OP_VERIFY_STEP_CHAIN, B, N, V, dt, Hq, Hkv, D, device=dev)
    rc = lib().sv_verify_step_chain(
        _p(q), _p(k_cache), _p(v_cache), _p(prefix_lens), Hq, Hkv, D, S_max, float(scale),
        _p(attn_out), _p(attn_status), _p(target_logits), _p(draft_logits), dt, _p(draft_tokens),
        _p(draft_lens), _p(u_accept), _p(u_sample), B, N, V, _p(accepted_len), _p(out_tokens),
        _p(probs_out), _p(verify_status), _p(new_kv_lens), _p(ws), ws.numel(), _stream(stream))
    _check("sv_verify_step_chain", rc)
    return attn_out, accepted_len, out_tokens, new_kv_lens


def sv_verify_step_tree_greedy(q, k_cache, v_cache, prefix_lens, parents, target_logits,
                               node_tokens, attn_out=None, accepted_len=None, path_nodes=None,
                               out_tokens=None, new_kv_lens=None, attn_status=None,
                               verify_status=None, node_counts=None, scale=None, ws=None,
                               stream=None):
    """The fused tree step (greedy acceptance; the caches are compacted in
    place).  q [B,T,Hq,D] bf16; caches [B,Hkv,S_max,D] bf16; parents [B,T]
    int32 or None (a chain); logits [B,T,V]; node_tokens [B,T] int32.
    Returns (attn_out, accepted_len, path_nodes, out_tokens, new_kv_lens)."""
    B, T, Hq, D, Hkv, S_max = _attn_shapes(q, k_cache, v_cache, prefix_lens, attn_out,
                                            attn_status)
    _req(target_logits, "target_logits", None, 3)
    _req(node_tokens, "node_tokens", torch.int32, 2)
    dt = _dtype_code(target_logits)
    V = target_logits.shape[2]
    _shape(target_logits, "target_logits", (B, T, V))
    _tree_shapes(B, T, node_tokens, parents, node_counts, accepted_len, path_nodes, out_tokens,
                 verify_status)
    _opt(new_kv_lens, "new_kv_lens", torch.int32, (B,))
    dev = q.device
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if attn_out is None:
        attn_out = torch.empty_like(q)
    if accepted_len is None:
        accepted_len = torch.empty(B, dtype=torch.int32, device=dev)
    if path_nodes is None:
        path_nodes = torch.empty(B, T, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty(B, T, dtype=torch.int32, device=dev)
    if new_kv_lens is None:
        new_kv_lens = torch.empty_like(prefix_lens)
    if ws is None:
        ws = workspace(SV_OP_VERIFY_STEP_TREE_GREEDY, B, T, V, dt, Hq, Hkv, D, device=dev)
    rc = lib().sv_verify_step_tree_greedy(
        _p(q), _p(k_cache), _p(v_cache), _p(prefix_lens), _p(parents), _p(node_counts), B, T, Hq,
        Hkv, D, S_max, float(scale), _p(attn_out), _p(attn_status), _p(target_logits), dt,
        _p(node_tokens), V, _p(accepted_len), _p(path_nodes), _p(out_tokens), _p(verify_status),
        _p(new_kv_lens), _p(ws), ws.numel(), _stream(stream))
    _check("sv_verify_step_tree_greedy", rc)
    return attn_out, accepted_len, path_nodes, out_tokens, new_kv_lens


def sv_compact_kv(k_cache, v_cache, prefix_lens, accepted_len, path_nodes=None, new_kv_lens=None,
                  seq_status=None, stream=None):
    """In place on k_cache/v_cache [B,Hkv,S_max,D] bf16.  path_nodes [B,P] int32 or
    None (chain).  Returns new_kv_lens [B] int32 (may be prefix_lens itself)."""
    _req(k_cache, "k_cache", torch.bfloat16, 4)
    _req(v_cache, "v_cache", torch.bfloat16, 4)
    _req(prefix_lens, "prefix_lens", torch.int32, 1)
    _req(accepted_len, "accepted_len", torch.int32, 1)
    B, Hkv, S_max, D = k_cache.shape
    _shape(v_cache, "v_cache", k_cache.shape)
    _shape(prefix_lens, "prefix_lens", (B,))
    _shape(accepted_len, "accepted_len", (B,))
    _opt(new_kv_lens, "new_kv_lens", torch.int32, (B,))
    _opt(seq_status, "seq_status", torch.int32, (B,))
    stride = 0
    if path_nodes is not None:
        _req(path_nodes, "path_nodes", torch.int32, 2)
        _shape(path_nodes, "path_nodes", (B, path_nodes.shape[1]))
        stride = path_nodes.shape[1]
    if new_kv_lens is None:
        new_kv_lens = torch.empty_like(prefix_lens)
    rc = lib().sv_compact_kv(_p(k_cache), _p(v_cache), _p(prefix_lens), _p(new_kv_lens),
                             _p(path_nodes), stride, _p(accepted_len), B, Hkv, D, S_max,
                             _p(seq_status), _stream(stream))
    _check("sv_compact_kv", rc)
    return new_kv_lens


def sv_compact_kv_paged(k_pages, v_pages, block_table, prefix_lens, accepted_len,
                        path_nodes=None, new_kv_lens=None, seq_status=None, stream=None):
    """In place on k_pages/v_pages [num_pages,Hkv,page_size,D] bf16 through
    block_table [B,max_pages] int32.  path_nodes [B,P] int32 or None (chain).
    Returns new_kv_lens [B] int32 (may be prefix_lens itself)."""
    _req(k_pages, "k_pages", torch.bfloat16, 4)
    _req(v_pages, "v_pages", torch.bfloat16, 4)
    _req(block_table, "block_table", torch.int32, 2)
    _req(prefix_lens, "prefix_lens", torch.int32, 1)
    _req(accepted_len, "accepted_len", torch.int32, 1)
    num_pages, Hkv, page_size, D = k_pages.shape
    B, max_pages = block_table.shape
    _shape(v_pages, "v_pages", k_pages.shape)
    _shape(prefix_lens, "prefix_lens", (B,))
    _shape(accepted_len, "accepted_len", (B,))
    _opt(new_kv_lens, "new_kv_lens", torch.int32, (B,))
    _opt(seq_status, "seq_status", torch.int32, (B,))
    stride = 0
    if path_nodes is not None:
        _req(path_nodes, "path_nodes", torch.int32, 2)
        _shape(path_nodes, "path_nodes", (B, path_nodes.shape[1]))
        stride = path_nodes.shape[1]
    if new_kv_lens is None:
        new_kv_lens = torch.empty_like(prefix_lens)
    rc = lib().sv_compact_kv_paged(_p(k_pages), _p(v_pages), _p(block_table), max_pages, num_pages,
                                   page_size, _p(prefix_lens), _p(new_kv_lens), _p(path_nodes),
                                   stride, _p(accepted_len), B, Hkv, D, _p(seq_status),
                                   _stream(stream))
    _check("sv_compact_kv_paged", rc)
    return new_kv_lens


class _Launch:
    """The device and stream of one call: every tensor on the first one's
    device, that device current while the call allocates and launches, its
    current stream (or the given one) the launch stream, on which outputs the
    call allocates are first used."""

    def __init__(self, device, stream):
        # (kernels launched on another device's stream would run there, on this device's addresses)
        if stream is not None and getattr(stream, "device", device) != device:
            raise ValueError(f"stream must be one of {device}, got one of {stream.device}")
        self.device, self.given = device, stream
        self.contexts = ()
        if device.type == "cuda":
            if device.index != torch.cuda.current_device():
                self.contexts += (torch.cuda.device(device),)
            if stream is not None:
                self.contexts += (torch.cuda.stream(stream),)

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        s = torch.cuda.current_stream(self.device) if self.given is None else self.given
        return s.cuda_stream

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)


def _arr(t, name, dtype, shape, device):
    """A contiguous array of the call's sizes on the call's device; its pointer."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device or not _on_device(t) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on {device}")
    return t.data_ptr()


def _opt_arr(t, name, dtype, shape, device):
    return None if t is None else _arr(t, name, dtype, shape, device)


def _rows(t, name, heads, device):
    """Rows [num_rows, heads, D] that may lie apart (parts of a wider row): the
    pointer and the elements between rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a tensor of 3 dims")
    n, h, d = t.shape
    if heads is not None and h != heads:
        raise ValueError(f"{name} must have {heads} heads, got {h}")
    sr, sh, sd = t.stride()
    if n == 1:
        sr = h * d  # the stride of a dimension of one says nothing
    if (t.device != device or not _on_device(t) or (d > 1 and sd != 1) or (h > 1 and sh != d)
            or sr < h * d):
        raise ValueError(f"{name} must be a CUDA tensor on {device} with its last two dims dense")
    return t.data_ptr(), sr


def _need_int(v, name):
    if isinstance(v, bool) or not isinstance(v, int):
        raise TypeError(f"{name} must be an int, got {type(v).__name__}")
    _fits32(**{name: v})
    return v


def _fits32(**sizes):
    """The library takes 32-bit sizes, and ctypes keeps the low 32 bits of a
    longer one without a word: it would be another call."""
    for name, v in sizes.items():
        if not -(1 << 31) <= v < 1 << 31:
            raise ValueError(f"{name} must fit in 32 bits, got {v}")


def sv_build_block_tables(prefix_lens, new_lens, page_counts, block_table, free_pages, free_count,
                          page_size, num_rows, row_starts=None, slot_map=None,
                          new_page_counts=None, new_free_count=None, seq_status=None, stream=None):
    """prefix_lens, new_lens, page_counts [B] int32; block_table [B,max_pages]
    int32 (the new pages' entries written in place); free_pages [num_pages]
    int32, free_count [1] int32 (a stack); num_rows: rows of the packed batch.
    Returns (row_starts [B+1], slot_map [num_rows], new_page_counts [B],
    new_free_count [1]), int32 (they may share one allocation)."""
    if row_starts is slot_map is new_page_counts is new_free_count is stream is None and (native := _native()) is not None:
        r = native.build_block_tables(prefix_lens, new_lens, page_counts, block_table, free_pages, free_count,
                                      page_size, num_rows, seq_status)
        if r is not None:
            return r
    i32 = torch.int32
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor of 2 dims")
    dev = block_table.device
    B, max_pages = block_table.shape
    _need_int(page_size, "page_size")
    _need_int(num_rows, "num_rows")
    if num_rows <= 0:
        raise ValueError(f"num_rows must be positive, got {num_rows}")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a tensor of 1 dim")
    num_pages = free_pages.shape[0]
    _fits32(B=B, max_pages=max_pages, num_pages=num_pages)
    p_tab = _arr(block_table, "block_table", i32, (B, max_pages), dev)
    p_pre = _arr(prefix_lens, "prefix_lens", i32, (B,), dev)
    p_new = _arr(new_lens, "new_lens", i32, (B,), dev)
    p_cnt = _arr(page_counts, "page_counts", i32, (B,), dev)
    p_stk = _arr(free_pages, "free_pages", i32, (num_pages,), dev)
    p_fc = _arr(free_count, "free_count", i32, (1,), dev)
    p_st = _opt_arr(seq_status, "seq_status", i32, (B,), dev)
    with _Launch(dev, stream) as s:
        if row_starts is None:
            row_starts = torch.empty(B + 1, dtype=i32, device=dev)
        if slot_map is None:
            slot_map = torch.empty(num_rows, dtype=i32, device=dev)
        if new_page_counts is None:
            new_page_counts = torch.empty(B, dtype=i32, device=dev)
        if new_free_count is None:
            new_free_count = torch.empty(1, dtype=i32, device=dev)
        rc = lib().sv_build_block_tables(
            p_pre, p_new, p_cnt, p_stk, p_fc, B, page_size, max_pages, num_pages, num_rows, p_tab,
            _arr(row_starts, "row_starts", i32, (B + 1,), dev),
            _arr(slot_map, "slot_map", i32, (num_rows,), dev),
            _arr(new_page_counts, "new_page_counts", i32, (B,), dev),
            _arr(new_free_count, "new_free_count", i32, (1,), dev), p_st, s)
    _check("sv_build_block_tables", rc)
    return row_starts, slot_map, new_page_counts, new_free_count


def sv_release_pages(keep_lens, page_counts, block_table, free_pages, free_count, page_size,
                     new_page_counts=None, new_free_count=None, seq_status=None, stream=None):
    """keep_lens, page_counts [B] int32; block_table [B,max_pages] int32;
    free_pages [num_pages] int32 (the pages given back written in place),
    free_count [1] int32.  Returns (new_page_counts [B], new_free_count [1]), int32."""
    if new_page_counts is new_free_count is stream is None and (native := _native()) is not None:
        r = native.release_pages(keep_lens, page_counts, block_table, free_pages, free_count, page_size,
                                 seq_status)
        if r is not None:
            return r
    i32 = torch.int32
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor of 2 dims")
    dev = block_table.device
    B, max_pages = block_table.shape
    _need_int(page_size, "page_size")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a tensor of 1 dim")
    num_pages = free_pages.shape[0]
    _fits32(B=B, max_pages=max_pages, num_pages=num_pages)
    p_tab = _arr(block_table, "block_table", i32, (B, max_pages), dev)
    p_keep = _arr(keep_lens, "keep_lens", i32, (B,), dev)
    p_cnt = _arr(page_counts, "page_counts", i32, (B,), dev)
    p_stk = _arr(free_pages, "free_pages", i32, (num_pages,), dev)
    p_fc = _arr(free_count, "free_count", i32, (1,), dev)
    p_st = _opt_arr(seq_status, "seq_status", i32, (B,), dev)
    with _Launch(dev, stream) as s:
        if new_page_counts is None:
            new_page_counts = torch.empty(B, dtype=i32, device=dev)
        if new_free_count is None:
            new_free_count = torch.empty(1, dtype=i32, device=dev)
        rc = lib().sv_release_pages(
            p_keep, p_cnt, p_tab, p_stk, p_fc, B, page_size, max_pages, num_pages,
            _arr(new_page_counts, "new_page_counts", i32, (B,), dev),
            _arr(new_free_count, "new_free_count", i32, (1,), dev), p_st, s)
    _check("sv_release_pages", rc)
    return new_page_counts, new_free_count


def _pages(k_pages, v_pages):
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be a tensor of 4 dims")
    dev = k_pages.device
    return (_arr(k_pages, "k_pages", torch.bfloat16, k_pages.shape, dev),
            _arr(v_pages, "v_pages", torch.bfloat16, k_pages.shape, dev), dev)


def sv_append_kv_paged(k_new, v_new, slot_map, k_pages, v_pages, row_status=None, stream=None):
    """k_new, v_new [num_rows,Hkv,D] bf16 or f32 (rows may lie apart: parts of a
    fused projection); slot_map [num_rows] int32 (-1: padding).  Writes the
    rows into k_pages/v_pages [num_pages,Hkv,page_size,D] bf16, in place."""
    if stream is None and (native := _native()) is not None:
        r = native.append_kv_paged(k_new, v_new, slot_map, k_pages, v_pages, row_status)
        if r is not None:
            return
    p_k, p_v, dev = _pages(k_pages, v_pages)
    num_pages, Hkv, page_size, D = k_pages.shape
    p_kn, k_stride = _rows(k_new, "k_new", Hkv, dev)
    p_vn, v_stride = _rows(v_new, "v_new", Hkv, dev)
    num_rows = k_new.shape[0]
    _fits32(num_rows=num_rows, num_pages=num_pages, Hkv=Hkv, page_size=page_size, D=D)
    if k_new.shape[2] != D or v_new.shape != k_new.shape:
        raise ValueError(f"k_new and v_new must have shape [num_rows, {Hkv}, {D}]")
    if k_new.dtype != v_new.dtype:
        raise TypeError("k_new and v_new must have one dtype")
    if k_new.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"k_new must be bfloat16 or float32, got {k_new.dtype}")
    dt = SV_BF16 if k_new.dtype == torch.bfloat16 else SV_F32
    p_slot = _arr(slot_map, "slot_map", torch.int32, (num_rows,), dev)
    p_st = _opt_arr(row_status, "row_status", torch.int32, (num_rows,), dev)
    with _Launch(dev, stream) as s:
        rc = lib().sv_append_kv_paged(p_kn, p_vn, dt, k_stride, v_stride, p_slot, num_rows, Hkv, D,
                                      page_size, num_pages, p_k, p_v, p_st, s)
    _check("sv_append_kv_paged", rc)


_WS_ZEROED = 1 << 16  # bytes at a chunk attention workspace's start that must begin as zeros
_chunk_ws: dict = {}


def _chunk_workspace(Hq, Hkv, D, device, stream):
    """A workspace for one call on `stream`: kept for the stream's later calls,
    which run after it, or, in a capture, the graph's own (zeroed by it), so
    that two graphs never share one."""
    capturing = device.type == "cuda" and torch.cuda.is_current_stream_capturing()
    key = (D, device.index, stream)
    ws = None if capturing else _chunk_ws.get(key)
    if ws is None:
        n = sv_workspace_size(SV_OP_CHUNK_ATTENTION, 0, 0, Hq=Hq, Hkv=Hkv, D=D)
        if n == 0:
            raise SpecVerifyError("sv_workspace_size", SV_ERR_UNSUPPORTED)
        ws = torch.empty(n, dtype=torch.uint8, device=device)
        ws[:_WS_ZEROED].zero_()
        if not capturing:
            _chunk_ws[key] = ws
    return ws


def sv_chunk_attention_paged(q, k_pages, v_pages, block_table, prefix_lens, row_starts, scale=None,
                             window=0, out=None, lse=None, return_lse=False, seq_status=None,
                             ws=None, stream=None):
    """q [num_rows,Hq,D] bf16 (rows may lie apart: part of a fused projection);
    k_pages/v_pages [num_pages,Hkv,page_size,D] bf16; block_table
    [B,max_pages], prefix_lens [B], row_starts [B+1] int32; window: slots a
    row sees at most (0: all before it).  Without ws the call keeps one a
    stream and D (40 MB at D = 128).  Returns out [num_rows,Hq,D] bf16, or (out, lse [num_rows,Hq]
    f32) with return_lse or a given lse."""
    if scale is None and isinstance(q, torch.Tensor) and q.dim() == 3:
        scale = 1.0 / math.sqrt(q.shape[2] or 1)
    if out is lse is ws is stream is None and (native := _native()) is not None:
        r = native.chunk_attention_paged(q, k_pages, v_pages, block_table, prefix_lens, row_starts, scale, window,
                                         return_lse, seq_status, _chunk_ws)
        if r is not None:
            return r
    bf16, i32 = torch.bfloat16, torch.int32
    p_k, p_v, dev = _pages(k_pages, v_pages)
    num_pages, Hkv, page_size, D = k_pages.shape
    p_q, q_stride = _rows(q, "q", None, dev)
    num_rows, Hq, dq = q.shape
    if q.dtype != bf16:
        raise TypeError(f"q must be {bf16}, got {q.dtype}")
    if dq != D:
        raise ValueError(f"q must have shape [num_rows, Hq, {D}], got {tuple(q.shape)}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor of 2 dims")
    B, max_pages = block_table.shape
    _fits32(num_rows=num_rows, Hq=Hq, B=B, max_pages=max_pages, num_pages=num_pages, Hkv=Hkv, page_size=page_size, D=D)
    p_tab = _arr(block_table, "block_table", i32, (B, max_pages), dev)
    p_pre = _arr(prefix_lens, "prefix_lens", i32, (B,), dev)
    p_row = _arr(row_starts, "row_starts", i32, (B + 1,), dev)
    p_st = _opt_arr(seq_status, "seq_status", i32, (B,), dev)
    _need_int(window, "window")
    with _Launch(dev, stream) as s:
        if out is None:
            out = torch.empty((num_rows, Hq, D), dtype=bf16, device=dev)
        if lse is None and return_lse:
            lse = torch.empty((num_rows, Hq), dtype=torch.float32, device=dev)
        if ws is None:
            ws = _chunk_workspace(Hq, Hkv, D, dev, s)
        rc = lib().sv_chunk_attention_paged(
            p_q, q_stride, p_k, p_v, p_tab, max_pages, num_pages, page_size, p_pre, p_row, B,
            num_rows, Hq, Hkv, D, float(scale), window,
            _arr(out, "out", bf16, (num_rows, Hq, D), dev),
            _opt_arr(lse, "lse", torch.float32, (num_rows, Hq), dev), p_st,
            _arr(ws, "ws", torch.uint8, ws.shape, dev), ws.numel(), s)
    _check("sv_chunk_attention_paged", rc)
    return out if lse is None else (out, lse)


def _given_ws(ws, dev):
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a tensor")
    return _arr(ws, "ws", torch.uint8, ws.shape, dev)


def _quant_pages(k_codes, k_params, v_codes, v_params):
    """The four arrays of a cache held in 4 bits: their pointers, the device and
    the sizes (num_pages, Hkv, page_size, D)."""
    if not isinstance(k_codes, torch.Tensor) or k_codes.dim() != 4:
        raise ValueError("k_codes must be a tensor of 4 dims")
    dev, u8, bf16 = k_codes.device, torch.uint8, torch.bfloat16
    num_pages, Hkv, page_size, half = k_codes.shape
    _fits32(num_pages=num_pages, Hkv=Hkv, page_size=page_size, D=2 * half)
    params = torch.Size((num_pages, Hkv, page_size, 2))
    return (_arr(k_codes, "k_codes", u8, k_codes.shape, dev), _arr(k_params, "k_params", bf16, params, dev),
            _arr(v_codes, "v_codes", u8, k_codes.shape, dev), _arr(v_params, "v_params", bf16, params, dev),
            dev, num_pages, Hkv, page_size, 2 * half)


def sv_append_kv_quant(k_new, v_new, slot_map, k_codes, k_params, v_codes, v_params, row_status=None, stream=None):
    """k_new, v_new [num_rows,Hkv,D] bf16 or f32 (rows may lie apart: parts of a
    fused projection); slot_map [num_rows] int32 (-1: padding).  Writes the
    rows in 4 bits into k_codes/v_codes [num_pages,Hkv,page_size,D/2] uint8 and
    k_params/v_params [num_pages,Hkv,page_size,2] bf16 (step, minimum), in place."""
    if stream is None and (native := _native()) is not None:
        if native.append_kv_quant(k_new, v_new, slot_map, k_codes, k_params, v_codes, v_params, row_status) is not None:
            return
    p_k, p_kp, p_v, p_vp, dev, num_pages, Hkv, page_size, D = _quant_pages(k_codes, k_params, v_codes, v_params)
    p_kn, k_stride = _rows(k_new, "k_new", Hkv, dev)
    p_vn, v_stride = _rows(v_new, "v_new", Hkv, dev)
    num_rows = k_new.shape[0]
    _fits32(num_rows=num_rows)
    if k_new.shape[2] != D or v_new.shape != k_new.shape:
        raise ValueError(f"k_new and v_new must have shape [num_rows, {Hkv}, {D}]")
    if k_new.dtype != v_new.dtype:
        raise TypeError("k_new and v_new must have one dtype")
    if k_new.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"k_new must be bfloat16 or float32, got {k_new.dtype}")
    dt = SV_BF16 if k_new.dtype == torch.bfloat16 else SV_F32
    p_slot = _arr(slot_map, "slot_map", torch.int32, (num_rows,), dev)
    p_st = _opt_arr(row_status, "row_status", torch.int32, (num_rows,), dev)
    with _Launch(dev, stream) as s:
        rc = lib().sv_append_kv_quant(p_kn, p_vn, dt, k_stride, v_stride, p_slot, num_rows, Hkv, D, page_size,
                                      num_pages, p_k, p_kp, p_v, p_vp, p_st, s)
    _check("sv_append_kv_quant", rc)


def sv_chunk_attention_quant(q, k_codes, k_params, v_codes, v_params, block_table, prefix_lens, row_starts,
                             parents=None, scale=None, window=0, out=None, lse=None, return_lse=False,
                             seq_status=None, ws=None, stream=None):
    """sv_chunk_attention_paged over a cache held in 4 bits (arrays as
    sv_append_kv_quant's).  parents [num_rows] int32: each sequence's rows (64 at
    most) are the nodes of a tree, a row's parent by its number in the sequence, -1
    for the first; None: every row sees the rows before it."""
    if scale is None and isinstance(q, torch.Tensor) and q.dim() == 3:
        scale = 1.0 / math.sqrt(q.shape[2] or 1)
    if out is lse is ws is stream is None and (native := _native()) is not None:
        r = native.chunk_attention_quant(q, k_codes, k_params, v_codes, v_params, block_table, prefix_lens, row_starts,
                                         parents, scale, window, return_lse, seq_status, _chunk_ws)
        if r is not None:
            return r
    bf16, i32 = torch.bfloat16, torch.int32
    p_k, p_kp, p_v, p_vp, dev, num_pages, Hkv, page_size, D = _quant_pages(k_codes, k_params, v_codes, v_params)
    p_q, q_stride = _rows(q, "q", None, dev)
    num_rows, Hq, dq = q.shape
    if q.dtype != bf16:
        raise TypeError(f"q must be {bf16}, got {q.dtype}")
    if dq != D:
        raise ValueError(f"q must have shape [num_rows, Hq, {D}], got {tuple(q.shape)}")
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor of 2 dims")
    B, max_pages = block_table.shape
    _fits32(num_rows=num_rows, Hq=Hq, B=B, max_pages=max_pages)
    p_tab = _arr(block_table, "block_table", i32, (B, max_pages), dev)
    p_pre = _arr(prefix_lens, "prefix_lens", i32, (B,), dev)
    p_row = _arr(row_starts, "row_starts", i32, (B + 1,), dev)
    p_par = _opt_arr(parents, "parents", i32, (num_rows,), dev)
    p_st = _opt_arr(seq_status, "seq_status", i32, (B,), dev)
    _need_int(window, "window")
    with _Launch(dev, stream) as s:
        if out is None:
            out = torch.empty((num_rows, Hq, D), dtype=bf16, device=dev)
        if lse is None and return_lse:
            lse = torch.empty((num_rows, Hq), dtype=torch.float32, device=dev)
        if ws is None:
            ws = _chunk_workspace(Hq, Hkv, D, dev, s)
        rc = lib().sv_chunk_attention_quant(
            p_q, q_stride, p_k, p_kp, p_v, p_vp, p_tab, max_pages, num_pages, page_size, p_pre, p_row, p_par, B,
            num_rows, Hq, Hkv, D, float(scale), window, _arr(out, "out", bf16, (num_rows, Hq, D), dev),
            _opt_arr(lse, "lse", torch.float32, (num_rows, Hq), dev), p_st,
            _given_ws(ws, dev), ws.numel(), s)
    _check("sv_chunk_attention_quant", rc)
    return out if lse is None else (out, lse)


def sv_compact_kv_quant(k_codes, k_params, v_codes, v_params, block_table, prefix_lens, accepted_len,
                        path_nodes=None, new_kv_lens=None, seq_status=None, stream=None):
    """sv_compact_kv_paged in a cache held in 4 bits.  path_nodes [B,P] int32 or
    None (chain).  Returns new_kv_lens [B] int32 (may be prefix_lens itself)."""
    if new_kv_lens is stream is None and (native := _native()) is not None:
        r = native.compact_kv_quant(k_codes, k_params, v_codes, v_params, block_table, prefix_lens, accepted_len,
                                    path_nodes, seq_status)
        if r is not None:
            return r
    i32 = torch.int32
    p_k, p_kp, p_v, p_vp, dev, num_pages, Hkv, page_size, D = _quant_pages(k_codes, k_params, v_codes, v_params)
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor of 2 dims")
    B, max_pages = block_table.shape
    stride = 0
    if path_nodes is not None:
        if not isinstance(path_nodes, torch.Tensor) or path_nodes.dim() != 2:
            raise ValueError("path_nodes must be a tensor of 2 dims")
        stride = path_nodes.shape[1]
    _fits32(B=B, max_pages=max_pages, path_stride=stride)
    p_tab = _arr(block_table, "block_table", i32, (B, max_pages), dev)
    p_pre = _arr(prefix_lens, "prefix_lens", i32, (B,), dev)
    p_acc = _arr(accepted_len, "accepted_len", i32, (B,), dev)
    p_path = _opt_arr(path_nodes, "path_nodes", i32, (B, stride), dev)
    p_st = _opt_arr(seq_status, "seq_status", i32, (B,), dev)
    with _Launch(dev, stream) as s:
        if new_kv_lens is None:
            new_kv_lens = torch.empty(B, dtype=i32, device=dev)
        rc = lib().sv_compact_kv_quant(p_k, p_kp, p_v, p_vp, p_tab, max_pages, num_pages, page_size, p_pre,
                                       _arr(new_kv_lens, "new_kv_lens", i32, (B,), dev), p_path, stride, p_acc, B,
                                       Hkv, D, p_st, s)
    _check("sv_compact_kv_quant", rc)
    return new_kv_lens


def _pool(block_table, free_pages, free_count, shares, page_size):
    """The table and the pool of pages of a call: pointers, device and sizes."""
    i32 = torch.int32
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise ValueError("block_table must be a tensor of 2 dims")
    dev = block_table.device
    B, max_pages = block_table.shape
    _need_int(page_size, "page_size")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a tensor of 1 dim")
    num_pages = free_pages.shape[0]
    _fits32(B=B, max_pages=max_pages, num_pages=num_pages)
    return (_arr(block_table, "block_table", i32, (B, max_pages), dev),
            _arr(free_pages, "free_pages", i32, (num_pages,), dev), _arr(free_count, "free_count", i32, (1,), dev),
            _arr(shares, "shares", i32, (num_pages,), dev), dev, B, max_pages, num_pages)


def _given(t, name, shape, device):
    """An int32 output: the caller's, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=torch.int32, device=device)
    _arr(t, name, torch.int32, shape, device)
    return t


def sv_fork_tables(sources, targets, fork_lens, page_counts, block_table, free_pages, free_count, shares, page_size,
                   copies=None, new_page_counts=None, new_free_count=None, new_shares=None, fork_status=None,
                   stream=None):
    """sources, targets, fork_lens [F] int32: the first fork_lens slots of a
    sequence for another one, which holds no page; page_counts [B], block_table
    [B,max_pages] (the targets' entries written in place), free_pages, shares
    [num_pages], free_count [1] int32.  Returns (copies [F,3] for sv_copy_pages,
    new_page_counts [B], new_free_count [1], new_shares [num_pages]), int32."""
    if copies is new_page_counts is new_free_count is new_shares is stream is None and (native := _native()) is not None:
        r = native.fork_tables(sources, targets, fork_lens, page_counts, block_table, free_pages, free_count, shares,
                               page_size, fork_status)
        if r is not None:
            return r
    i32 = torch.int32
    p_tab, p_stk, p_fc, p_sh, dev, B, max_pages, num_pages = _pool(block_table, free_pages, free_count, shares, page_size)
    if not isinstance(sources, torch.Tensor) or sources.dim() != 1:
        raise ValueError("sources must be a tensor of 1 dim")
    F = sources.shape[0]
    _fits32(F=F)
    p_src = _arr(sources, "sources", i32, (F,), dev)
    p_tgt = _arr(targets, "targets", i32, (F,), dev)
    p_len = _arr(fork_lens, "fork_lens", i32, (F,), dev)
    p_cnt = _arr(page_counts, "page_counts", i32, (B,), dev)
    p_st = _opt_arr(fork_status, "fork_status", i32, (F,), dev)
    with _Launch(dev, stream) as s:
        copies = _given(copies, "copies", (F, 3), dev)
        new_page_counts = _given(new_page_counts, "new_page_counts", (B,), dev)
        new_free_count = _given(new_free_count, "new_free_count", (1,), dev)
        new_shares = _given(new_shares, "new_shares", (num_pages,), dev)
        rc = lib().sv_fork_tables(p_src, p_tgt, p_len, p_cnt, p_stk, p_fc, p_sh, F, B, page_size, max_pages, num_pages,
                                  p_tab, copies.data_ptr(), new_page_counts.data_ptr(), new_free_count.data_ptr(),
                                  new_shares.data_ptr(), p_st, s)
    _check("sv_fork_tables", rc)
    return copies, new_page_counts, new_free_count, new_shares


_MAX_PLANES = 64  # of a launch of sv_copy_pages


def sv_copy_pages(copies, planes, copy_status=None, stream=None):
    """copies [F,3] int32, rows (from, to, slots); planes: a list of tensors
    [num_pages,Hkv,page_size,X] of any type (pages of K, V, codes, parameters, of
    any number of layers; 64 a launch).  The first slots of page `from` are written
    to page `to`."""
    if stream is None and (native := _native()) is not None:
        if native.copy_pages(copies, planes, copy_status) is not None:
            return
    if not isinstance(planes, (list, tuple)) or not planes or not all(isinstance(t, torch.Tensor) for t in planes):
        raise TypeError("planes must be a list of tensors")
    if planes[0].dim() != 4:
        raise ValueError("planes must have 4 dims")
    dev, first = planes[0].device, planes[0].shape[:3]
    for i, t in enumerate(planes):
        if t.dim() != 4 or t.shape[:3] != first:
            raise ValueError(f"planes[{i}] must have shape {tuple(first)} + (X,), got {tuple(t.shape)}")
        _arr(t, f"planes[{i}]", t.dtype, t.shape, dev)
    if not isinstance(copies, torch.Tensor) or copies.dim() != 2:
        raise ValueError("copies must be a tensor of 2 dims")
    F, n = copies.shape[0], len(planes)
    num_pages, Hkv, page_size = first
    row_bytes = [t.shape[3] * t.element_size() for t in planes]
    _fits32(F=F, num_pages=num_pages, Hkv=Hkv, page_size=page_size, row_bytes=max(row_bytes))
    p_c = _arr(copies, "copies", torch.int32, (F, 3), dev)
    p_st = _opt_arr(copy_status, "copy_status", torch.int32, (F,), dev)
    if n > _MAX_PLANES:  # (several launches, and none before every plane is known to be taken)
        for t, b in zip(planes, row_bytes):
            if b <= 0 or b % 4 or t.data_ptr() % 16:
                _check("sv_copy_pages", SV_ERR_INVALID_ARG)
            if b > 4096:
                _check("sv_copy_pages", SV_ERR_UNSUPPORTED)
    with _Launch(dev, stream) as s:
        for i in range(0, n, _MAX_PLANES):
            part, sizes = planes[i:i + _MAX_PLANES], row_bytes[i:i + _MAX_PLANES]
            m = len(part)
            rc = lib().sv_copy_pages(p_c, F, (ctypes.c_void_p * m)(*(t.data_ptr() for t in part)),
                                     (ctypes.c_int * m)(*sizes), m, Hkv, page_size, num_pages, p_st, s)
            _check("sv_copy_pages", rc)


def sv_release_shared_pages(keep_lens, page_counts, block_table, free_pages, free_count, shares, page_size,
                            new_page_counts=None, new_free_count=None, new_shares=None, seq_status=None, ws=None,
                            stream=None):
    """sv_release_pages where pages may be shared: a page goes to the stack (in
    place) with its last holder.  Returns (new_page_counts [B], new_free_count
    [1], new_shares [num_pages]), int32."""
    if new_page_counts is new_free_count is new_shares is ws is stream is None and (native := _native()) is not None:
        r = native.release_shared_pages(keep_lens, page_counts, block_table, free_pages, free_count, shares, page_size,
                                        seq_status)
        if r is not None:
            return r
    i32 = torch.int32
    p_tab, p_stk, p_fc, p_sh, dev, B, max_pages, num_pages = _pool(block_table, free_pages, free_count, shares, page_size)
    p_keep = _arr(keep_lens, "keep_lens", i32, (B,), dev)
    p_cnt = _arr(page_counts, "page_counts", i32, (B,), dev)
    p_st = _opt_arr(seq_status, "seq_status", i32, (B,), dev)
    with _Launch(dev, stream) as s:
        new_page_counts = _given(new_page_counts, "new_page_counts", (B,), dev)
        new_free_count = _given(new_free_count, "new_free_count", (1,), dev)
        new_shares = _given(new_shares, "new_shares", (num_pages,), dev)
        if ws is None:  # (any contents: no call needs another's)
            ws = torch.empty(sv_workspace_size(SV_OP_RELEASE_SHARED_PAGES, 0, num_pages), dtype=torch.uint8, device=dev)
        rc = lib().sv_release_shared_pages(p_keep, p_cnt, p_tab, p_stk, p_fc, p_sh, B, page_size, max_pages, num_pages,
                                           new_page_counts.data_ptr(), new_free_count.data_ptr(), new_shares.data_ptr(),
                                           p_st, _given_ws(ws, dev), ws.numel(), s)
    _check("sv_release_shared_pages", rc)
    return new_page_counts, new_free_count, new_shares


def sv_verify_chain_noalloc(target_logits, draft_logits, draft_tokens, u_accept, u_sample,
                            accepted_len, out_tokens, probs_out=None, seq_status=None, stream=None):
    """sv_verify_chain without a workspace, for callers that cannot allocate
    device memory at the call site; the outputs must be passed in.  Uses the
    library's fixed scratch array: calls must not overlap on the GPU."""
    _req(target_logits, "target_logits", None, 3)
    _req(draft_logits, "draft_logits", target_logits.dtype, 3)
    _req(draft_tokens, "draft_tokens", torch.int32, 2)
    _req(u_accept, "u_accept", torch.float32, 2)
    _req(u_sample, "u_sample", torch.float32, 1)
    _req(accepted_len, "accepted_len", torch.int32, 1)
    _req(out_tokens, "out_tokens", torch.int32, 2)
    dt = _dtype_code(target_logits)
    B, N1, V = target_logits.shape
    _chain_shapes(B, N1 - 1, V, draft_logits, draft_tokens, u_accept, u_sample, accepted_len,
                  out_tokens, probs_out, seq_status)
    rc = lib().sv_verify_chain_noalloc(_p(target_logits), _p(draft_logits), dt, _p(draft_tokens),
                                       _p(u_accept), _p(u_sample), B, N1 - 1, V,
                                       _p(accepted_len), _p(out_tokens), _p(probs_out),
                                       _p(seq_status), _stream(stream))
    _check("sv_verify_chain_noalloc", rc)
    return accepted_len, out_tokens
