"""The calls of a cache held in 4 bits and of requests that share pages without a GPU:
what the library refuses on the host, what the binding refuses before it calls it, the
addresses and sizes that it passes, and the work list of the attention's form for few
rows against counting."""
import ctypes
import os
import subprocess
import types

import numpy as np
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv
from speculative_decoding_verification_81_gb300 import api
from speculative_decoding_verification_81_gb300 import build as svbuild
from test_pages_binding import FAKE, MISALIGNED, OTHER, STREAM, Recorder, _i32, _refused
from test_pages_binding import rec  # noqa: F401  (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = sv.SV_ERR_INVALID_ARG, sv.SV_ERR_UNSUPPORTED, sv.SV_ERR_WORKSPACE
bf16, u8 = torch.bfloat16, torch.uint8


@pytest.fixture(scope="module")
def L():
    svbuild.build()
    return sv.lib()


# ---------------------------------------------------------------- the library's checks

def test_append_quant_host_validation(L):
    def call(**kw):
        a = dict(k=FAKE, v=FAKE, dt=sv.SV_BF16, ks=1024, vs=1024, sm=FAKE, rows=4, Hkv=8, D=128, ps=16, np=8, kc=FAKE,
                 kp=FAKE, vc=FAKE, vp=FAKE)
        a.update(kw)
        return L.sv_append_kv_quant(*a.values(), None, None)
    for name in ("k", "v", "sm", "kc", "kp", "vc", "vp"):
        assert call(**{name: None}) == INVALID, name
    for name in ("k", "v", "kc", "kp", "vc", "vp"):
        assert call(**{name: MISALIGNED}) == INVALID, name
    for name in ("rows", "Hkv", "D", "ps", "np"):
        assert call(**{name: 0}) == INVALID, name
    assert call(dt=5) == INVALID
    assert call(ks=1016) == INVALID                 # rows would overlap
    assert call(vs=1028) == INVALID                 # rows off their 16-byte boundaries
    assert call(dt=sv.SV_F32, vs=1026) == INVALID
    assert call(D=96) == UNSUPPORTED
    assert call(D=256, ks=2048, vs=2048) == UNSUPPORTED
    assert call(np=1 << 24) == UNSUPPORTED          # rows of the cache
    assert call(rows=1 << 30) == UNSUPPORTED
    assert call(ks=1 << 32) == UNSUPPORTED


def test_chunk_attention_quant_host_validation(L):
    def call(**kw):
        a = dict(q=FAKE, qs=4096, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, bt=FAKE, mp=8, np=64, ps=16, pl=FAKE, rs=FAKE,
                 par=None, B=2, rows=9, Hq=32, Hkv=8, D=128, scale=0.088, win=0, out=OTHER)
        a.update(kw)
        return L.sv_chunk_attention_quant(*a.values(), None, None, None, 0, None)
    for name in ("q", "kc", "kp", "vc", "vp", "bt", "pl", "rs", "out"):
        assert call(**{name: None}) == INVALID, name
    for name in ("mp", "np", "ps", "B", "rows", "Hq", "Hkv", "D"):
        assert call(**{name: 0}) == INVALID, name
    for name in ("q", "kc", "kp", "vc", "vp", "out"):
        assert call(**{name: MISALIGNED}) == INVALID, name
    assert call(out=FAKE) == INVALID                # written over its own queries
    assert call(qs=4088) == INVALID
    assert call(qs=4100) == INVALID
    assert call(ps=24) == INVALID
    assert call(ps=4) == INVALID
    assert call(Hq=30) == INVALID
    assert call(win=-1) == INVALID
    assert call(par=FAKE, win=5) == INVALID         # a tree has no window
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == INVALID, scale
    assert call(D=96) == UNSUPPORTED
    assert call(Hq=1032, qs=1032 * 128) == UNSUPPORTED  # 129 heads a group
    assert call(B=4097) == UNSUPPORTED
    assert call(mp=1 << 26) == UNSUPPORTED
    assert call(np=1 << 24) == UNSUPPORTED
    assert call(rows=1 << 30) == UNSUPPORTED


def test_compact_quant_host_validation(L):
    def call(**kw):
        a = dict(kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, bt=FAKE, mp=8, np=64, ps=16, pre=FAKE, new=FAKE, path=None, stride=0,
                 acc=FAKE, B=2, Hkv=8, D=128)
        a.update(kw)
        return L.sv_compact_kv_quant(*a.values(), None, None)
    for name in ("kc", "kp", "vc", "vp", "bt", "pre", "new", "acc"):
        assert call(**{name: None}) == INVALID, name
    for name in ("kc", "kp", "vc", "vp"):
        assert call(**{name: MISALIGNED}) == INVALID, name
    for name in ("mp", "np", "ps", "B", "Hkv", "D"):
        assert call(**{name: 0}) == INVALID, name
    assert call(path=FAKE) == INVALID               # paths of no length
    assert call(D=96) == UNSUPPORTED
    assert call(mp=1 << 26) == UNSUPPORTED
    assert call(np=1 << 24) == UNSUPPORTED


def test_fork_and_shared_release_host_validation(L):
    def fork(**kw):
        a = dict(src=FAKE, tgt=FAKE, len=FAKE, cnt=FAKE, stk=FAKE, fc=FAKE, sh=FAKE, F=3, B=4, ps=16, mp=8, np=64, tab=FAKE,
                 copies=FAKE, nc=OTHER, nf=OTHER, ns=OTHER)
        a.update(kw)
        return L.sv_fork_tables(*a.values(), None, None)

    def release(**kw):
        a = dict(keep=FAKE, cnt=FAKE, tab=FAKE, stk=FAKE, fc=FAKE, sh=FAKE, B=4, ps=16, mp=8, np=64, nc=OTHER, nf=OTHER,
                 ns=OTHER, st=None, ws=FAKE, n=0)
        a.update(kw)
        return L.sv_release_shared_pages(*a.values(), None)
    for call, names, sizes in ((fork, "src tgt len cnt stk fc sh tab copies nc nf ns", "F B ps mp np"),
                               (release, "keep cnt tab stk fc sh nc nf ns", "B ps mp np")):
        for name in names.split():
            assert call(**{name: None}) == INVALID, name
        for name in sizes.split():
            assert call(**{name: 0}) == INVALID, name
        for name in ("nc", "nf", "ns"):             # new arrays over the old ones
            assert call(**{name: FAKE}) == INVALID, name
        assert call(B=4097) == UNSUPPORTED
        assert call(mp=1 << 26) == UNSUPPORTED
        assert call(ps=1 << 20, np=1 << 12) == UNSUPPORTED
    assert fork(F=4097) == UNSUPPORTED
    need = sv.sv_workspace_size(sv.SV_OP_RELEASE_SHARED_PAGES, 0, 64)
    assert need > 64 * 4 and sv.sv_workspace_size(sv.SV_OP_RELEASE_SHARED_PAGES, 0, 0) == 0
    assert release(n=need - 1) == WORKSPACE
    assert release(ws=None, n=need) == WORKSPACE
    assert release(ws=ctypes.c_void_p(0x10002), n=need) == WORKSPACE


def test_copy_pages_host_validation(L):
    def call(planes=(0x10000, 0x20000), rows=(64, 4), **kw):
        a = dict(copies=FAKE, F=3, n=len(planes), Hkv=8, ps=16, np=64)
        a.update(kw)
        return L.sv_copy_pages(a["copies"], a["F"], (ctypes.c_void_p * len(planes))(*planes), (ctypes.c_int * len(rows))(*rows),
                               a["n"], a["Hkv"], a["ps"], a["np"], None, None)
    assert call(copies=None) == INVALID
    for name in ("F", "n", "Hkv", "ps", "np"):
        assert call(**{name: 0}) == INVALID, name
    assert call(planes=(0x10000, 0)) == INVALID
    assert call(planes=(0x10000, 0x20004)) == INVALID
    for rows in ((64, 0), (64, -4), (64, 6)):
        assert call(rows=rows) == INVALID, rows
    assert call(rows=(64, 8192)) == UNSUPPORTED
    assert call(planes=(0x10000,) * 65, rows=(4,) * 65) == UNSUPPORTED
    assert call(np=1 << 24) == UNSUPPORTED


# ---------------------------------------------------------------- the binding

def cache():
    return dict(k_codes=torch.zeros((9, 2, 16, 32), dtype=u8), k_params=torch.zeros((9, 2, 16, 2), dtype=bf16),
                v_codes=torch.zeros((9, 2, 16, 32), dtype=u8), v_params=torch.zeros((9, 2, 16, 2), dtype=bf16))


def append_kw(dtype=bf16):
    qkv = torch.zeros((6, 9, 64), dtype=dtype)
    return dict(k_new=qkv[:, 5:7], v_new=qkv[:, 7:9], slot_map=_i32(6), **cache(), row_status=_i32(6), stream=STREAM)


def attention_kw():
    return dict(q=torch.zeros((6, 8, 64), dtype=bf16)[:, :4], **cache(), block_table=_i32(3, 5), prefix_lens=_i32(3),
                row_starts=_i32(4), parents=_i32(6), out=torch.zeros((6, 4, 64), dtype=bf16), lse=torch.zeros((6, 4)),
                seq_status=_i32(3), ws=torch.zeros(256, dtype=u8), stream=STREAM)


def compact_kw():
    return dict(**cache(), block_table=_i32(3, 5), prefix_lens=_i32(3), accepted_len=_i32(3), path_nodes=_i32(3, 7),
                new_kv_lens=_i32(3), seq_status=_i32(3), stream=STREAM)


def fork_kw():
    return dict(sources=_i32(2), targets=_i32(2), fork_lens=_i32(2), page_counts=_i32(3), block_table=_i32(3, 5),
                free_pages=_i32(20), free_count=_i32(1), shares=_i32(20), page_size=16, copies=_i32(2, 3),
                new_page_counts=_i32(3), new_free_count=_i32(1), new_shares=_i32(20), fork_status=_i32(2), stream=STREAM)


def copy_kw():
    return dict(copies=_i32(2, 3), planes=[torch.zeros((9, 2, 16, 32), dtype=u8), torch.zeros((9, 2, 16, 2), dtype=bf16)],
                copy_status=_i32(2), stream=STREAM)


def release_kw():
    return dict(keep_lens=_i32(3), page_counts=_i32(3), block_table=_i32(3, 5), free_pages=_i32(20), free_count=_i32(1),
                shares=_i32(20), page_size=16, new_page_counts=_i32(3), new_free_count=_i32(1), new_shares=_i32(20),
                seq_status=_i32(3), ws=torch.zeros(80, dtype=u8), stream=STREAM)


CALLS = {"sv_append_kv_quant": append_kw, "sv_chunk_attention_quant": attention_kw, "sv_compact_kv_quant": compact_kw,
         "sv_fork_tables": fork_kw, "sv_copy_pages": copy_kw, "sv_release_shared_pages": release_kw}
CODES = ("k_codes", "k_params", "v_codes", "v_params")
# what each call passes: positions of arrays (None: the order of its names), of sizes
PASSED = {
    "sv_append_kv_quant": (dict(zip((0, 1, 5, 11, 12, 13, 14, 15), ("k_new", "v_new", "slot_map", *CODES, "row_status"))),
                           {2: sv.SV_BF16, 3: 576, 4: 576, 6: 6, 7: 2, 8: 64, 9: 16, 10: 9}),
    "sv_chunk_attention_quant": (dict(zip((0, 2, 3, 4, 5, 6, 10, 11, 12, 20, 21, 22, 23),
                                          ("q", *CODES, "block_table", "prefix_lens", "row_starts", "parents", "out", "lse",
                                           "seq_status", "ws"))),
                                 {1: 512, 7: 5, 8: 9, 9: 16, 13: 3, 14: 6, 15: 4, 16: 2, 17: 64, 18: 0.125, 19: 0, 24: 256}),
    "sv_compact_kv_quant": (dict(zip((0, 1, 2, 3, 4, 8, 9, 10, 12, 16),
                                     (*CODES, "block_table", "prefix_lens", "new_kv_lens", "path_nodes", "accepted_len",
                                      "seq_status"))), {5: 5, 6: 9, 7: 16, 11: 7, 13: 3, 14: 2, 15: 64}),
    "sv_fork_tables": (dict(zip((0, 1, 2, 3, 4, 5, 6, 12, 13, 14, 15, 16, 17),
                                ("sources", "targets", "fork_lens", "page_counts", "free_pages", "free_count", "shares",
                                 "block_table", "copies", "new_page_counts", "new_free_count", "new_shares", "fork_status"))),
                       {7: 2, 8: 3, 9: 16, 10: 5, 11: 20}),
    "sv_copy_pages": ({0: "copies", 8: "copy_status"}, {1: 2, 4: 2, 5: 2, 6: 16, 7: 9}),
    "sv_release_shared_pages": (dict(zip((0, 1, 2, 3, 4, 5, 10, 11, 12, 13, 14),
                                         ("keep_lens", "page_counts", "block_table", "free_pages", "free_count", "shares",
                                          "new_page_counts", "new_free_count", "new_shares", "seq_status", "ws"))),
                                {6: 3, 7: 16, 8: 5, 9: 20, 15: 80}),
}


@pytest.mark.parametrize("name", CALLS)
def test_marshalling(rec, name):  # noqa: F811
    kw = CALLS[name]()
    getattr(api, name)(**kw)
    called, a = rec.calls[-1]
    arrays, sizes = PASSED[name]
    assert called == name and a[-1] == STREAM.cuda_stream
    for i, n in arrays.items():
        assert a[i] == kw[n].data_ptr(), n
    for i, x in sizes.items():
        assert a[i] == x, i
    if name == "sv_copy_pages":
        assert list(a[2]) == [t.data_ptr() for t in kw["planes"]] and list(a[3]) == [32, 4]


def wrong(name):
    """Arguments that the call refuses, one at a time."""
    kw = CALLS[name]()
    for n, t in kw.items():
        if n in ("stream", "page_size"):
            continue
        if n == "planes":
            yield n, [], "none"
            yield n, t[0], "no list"
            yield n, [t[0], t[1][:8]], "of other pages"
            yield n, [t[0], t[1].transpose(0, 1)], "of other pages"
            yield n, [t[0], t[1].to("meta")], "elsewhere"
            yield n, [t[0][0]], "of 3 dims"
            continue
        if n not in ("k_codes", "q", "ws", "block_table", "sources", "copies", "free_pages"):  # (these set the sizes)
            yield n, t[:-1], "short"
        yield n, t.to(torch.float64), "of another type"
        yield n, t.to("meta") if n not in ("k_codes", "block_table", "copies") else t.flatten(), "elsewhere, or flat"
        yield n, t.tolist(), "no tensor"
        if t.dim() > 1 and n not in ("k_new", "v_new", "q"):
            yield n, torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2], "with gaps"


@pytest.mark.parametrize("name", CALLS)
def test_refusals(rec, name):  # noqa: F811
    for n, bad, why in wrong(name):
        kw = CALLS[name]()
        kw[n] = bad
        calls = len(rec.calls)
        try:
            getattr(api, name)(**kw)
        except (ValueError, TypeError):
            assert len(rec.calls) == calls
        else:
            pytest.fail(f"{name} took {n} {why}")
    for bad in (16.0, None, True):
        if "page_size" in CALLS[name]():
            _refused(rec, getattr(api, name), **{**CALLS[name](), "page_size": bad})


def test_refused_shapes_of_rows(rec):  # noqa: F811
    for n, bad in (("k_new", torch.zeros((6, 3, 64), dtype=bf16)), ("v_new", torch.zeros((5, 2, 64), dtype=bf16)),
                   ("k_new", torch.zeros((6, 2, 64), dtype=torch.float16)), ("v_new", torch.zeros((6, 2, 64))),
                   ("k_new", torch.zeros((2, 6, 64), dtype=bf16).transpose(0, 1)), ("k_codes", torch.zeros((9, 2, 16, 64), dtype=u8))):
        _refused(rec, api.sv_append_kv_quant, **{**append_kw(), n: bad})
    for n, bad in (("q", torch.zeros((6, 4, 128), dtype=bf16)), ("q", torch.zeros((4, 6, 64), dtype=bf16).transpose(0, 1)),
                   ("window", 2.0), ("window", None)):
        _refused(rec, api.sv_chunk_attention_quant, **{**attention_kw(), n: bad})


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(rec, name):  # noqa: F811
    for device, refused in (("cpu", False), ("cuda:1", True)):
        kw = {**CALLS[name](), "stream": types.SimpleNamespace(cuda_stream=77, device=torch.device(device))}
        if refused:
            _refused(rec, getattr(api, name), **kw)
        else:
            getattr(api, name)(**kw)
            assert rec.calls[-1][1][-1] == 77


def test_the_extension_leaves_what_it_does_not_take(L):
    """Arrays that are not on a GPU, no arrays, no arguments: its functions return None."""
    native = api._native()
    if native is None:
        pytest.skip("the extension is not built")
    order = {"append_kv_quant": "k_new v_new slot_map k_codes k_params v_codes v_params row_status",
             "compact_kv_quant": "k_codes k_params v_codes v_params block_table prefix_lens accepted_len path_nodes seq_status",
             "fork_tables": "sources targets fork_lens page_counts block_table free_pages free_count shares page_size fork_status",
             "copy_pages": "copies planes copy_status",
             "release_shared_pages": "keep_lens page_counts block_table free_pages free_count shares page_size seq_status"}
    for name, args in order.items():
        kw = CALLS["sv_" + name]()
        assert getattr(native, name)(*(kw[n] for n in args.split())) is None
        assert getattr(native, name)(*([None] * len(args.split()))) is None
        assert getattr(native, name)() is None
    kw = attention_kw()
    names = "q k_codes k_params v_codes v_params block_table prefix_lens row_starts parents".split()
    assert native.chunk_attention_quant(*(kw[n] for n in names), 0.125, 0, True, None, {}) is None
    assert native.chunk_attention_quant(*[None] * 14) is None


# ---------------------------------------------------------------- the work list

SRC = r"""
#include "sv_quant_list.h"
using namespace sv::chunk;
extern "C" int c_items(int tok, int window, int L, int n) { return rows_seq({tok, window, 1 << 29, 1 << 29}, L, 5, 5 + n).items; }
extern "C" int c_tiles(int tok, int window, int L, int n, int i) {
    const RowsShape p{tok, window, 1 << 29, 1 << 29};
    return rows_tiles(p, rows_seq(p, L, 5, 5 + n), i);
}
extern "C" int c_first(int tok, int window, int pos) { return rows_first_tile({tok, window, 1 << 29, 1 << 29}, pos); }
extern "C" long long c_before(int tok, int window, int L, int n, int i) {
    const RowsShape p{tok, window, 1 << 29, 1 << 29};
    return rows_units_before(p, rows_seq(p, L, 5, 5 + n), i);
}
extern "C" int c_valid(int L, int r0, int r1, int rows, int smax) { return rows_seq({4, 0, rows, smax}, L, r0, r1).n; }
extern "C" int c_ctas(long long U, int grid) { return rows_ctas(U, grid); }
extern "C" int c_cost() { return kRowsItemCost; }
"""


@pytest.fixture(scope="module")
def C(tmp_path_factory):
    d = tmp_path_factory.mktemp("quant_list")
    (d / "shim.cpp").write_text(SRC)
    inc = os.path.join(ROOT, "speculative_decoding_verification_81_gb300", "csrc")
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined", "-fno-sanitize-recover",
                           "-static-libubsan", f"-I{inc}", str(d / "shim.cpp"), "-o", str(d / "shim.so")])
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.c_before.restype = ctypes.c_longlong
    lib.c_ctas.argtypes = [ctypes.c_longlong, ctypes.c_int]
    return lib


def test_units_against_counting(C):
    rng = np.random.default_rng(2)
    cost = C.c_cost()
    for _ in range(400):
        tok = int(rng.integers(1, 65))
        window = int(rng.choice([0, 0, 1, 5, 128, 129, 1000]))
        past, n = int(rng.integers(0, 3000)), int(rng.integers(1, 400))
        items = C.c_items(tok, window, past, n)
        assert items == -(-n // tok)
        units = 0
        for i in range(items):
            assert C.c_before(tok, window, past, n, i) == units
            t0, t1 = i * tok, min(n, (i + 1) * tok)
            lo = max(0, past + t0 - window + 1) if window else 0
            assert C.c_first(tok, window, past + t0) == lo // 128
            tiles = (past + t1 - 1) // 128 - lo // 128 + 1
            assert C.c_tiles(tok, window, past, n, i) == tiles
            units += cost + tiles
        assert C.c_before(tok, window, past, n, items) == units


def test_lengths_that_are_none_have_no_rows(C):
    assert C.c_valid(10, 3, 7, 20, 100) == 4
    for L, r0, r1 in ((-1, 3, 7), (98, 3, 7), (10, -1, 3), (10, 7, 3), (10, 3, 21), (10, 3, 3)):
        assert C.c_valid(L, r0, r1, 20, 100) == 0


def test_ctas_of_a_list(C):
    assert C.c_ctas(1, 304) == 1 and C.c_ctas(10 ** 12, 304) == 304
    assert all(1 <= C.c_ctas(u, 304) <= u for u in range(1, 2000))
