"""The paged-cache calls (tables, pages back, new rows, attention of chunks)
without a GPU: what the library refuses on the host, and what the binding
refuses before it calls it."""
import ctypes
import types

import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv
from speculative_decoding_verification_81_gb300 import api
from speculative_decoding_verification_81_gb300 import build as svbuild

FAKE, OTHER = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)  # never dereferenced
MISALIGNED = ctypes.c_void_p(0x10004)
STREAM = types.SimpleNamespace(cuda_stream=0)


@pytest.fixture(scope="module")
def L():
    svbuild.build()
    return sv.lib()


def test_build_block_tables_host_validation(L):
    def call(**kw):
        a = dict(pre=FAKE, new=FAKE, cnt=FAKE, stk=FAKE, fc=FAKE, B=2, ps=0, mp=8, np=64, rows=20,
                 tab=FAKE, rs=FAKE, sm=FAKE, nc=OTHER, nf=OTHER)
        a.update(kw)
        return L.sv_build_block_tables(a["pre"], a["new"], a["cnt"], a["stk"], a["fc"], a["B"], a["ps"],
                                       a["mp"], a["np"], a["rows"], a["tab"], a["rs"], a["sm"], a["nc"],
                                       a["nf"], None, None)
    for name in ("pre", "new", "cnt", "stk", "fc", "tab", "rs", "sm", "nc", "nf"):
        assert call(ps=16, **{name: None}) == sv.SV_ERR_INVALID_ARG, name
    assert call() == sv.SV_ERR_INVALID_ARG                      # page_size 0
    for name in ("B", "mp", "np", "rows"):
        assert call(ps=16, **{name: 0}) == sv.SV_ERR_INVALID_ARG, name
    assert call(ps=16, nc=FAKE) == sv.SV_ERR_INVALID_ARG        # new counts over the old ones
    assert call(ps=16, nf=FAKE) == sv.SV_ERR_INVALID_ARG
    assert call(ps=16, B=4097) == sv.SV_ERR_UNSUPPORTED
    assert call(ps=1 << 28) == sv.SV_ERR_UNSUPPORTED            # max_pages * page_size
    assert call(ps=1 << 20, np=1 << 12) == sv.SV_ERR_UNSUPPORTED  # num_pages * page_size
    assert call(ps=16, rows=1 << 30) == sv.SV_ERR_UNSUPPORTED


def test_release_pages_host_validation(L):
    def call(**kw):
        a = dict(keep=FAKE, cnt=FAKE, tab=FAKE, stk=FAKE, fc=FAKE, B=2, ps=0, mp=8, np=64, nc=OTHER, nf=OTHER)
        a.update(kw)
        return L.sv_release_pages(a["keep"], a["cnt"], a["tab"], a["stk"], a["fc"], a["B"], a["ps"], a["mp"],
                                  a["np"], a["nc"], a["nf"], None, None)
    for name in ("keep", "cnt", "tab", "stk", "fc", "nc", "nf"):
        assert call(ps=16, **{name: None}) == sv.SV_ERR_INVALID_ARG, name
    assert call() == sv.SV_ERR_INVALID_ARG
    assert call(ps=16, nc=FAKE) == sv.SV_ERR_INVALID_ARG
    assert call(ps=16, nf=FAKE) == sv.SV_ERR_INVALID_ARG
    assert call(ps=16, B=5000) == sv.SV_ERR_UNSUPPORTED


def test_append_host_validation(L):
    def call(**kw):
        a = dict(k=FAKE, v=FAKE, dt=sv.SV_BF16, ks=1024, vs=1024, sm=FAKE, rows=4, Hkv=8, D=128, ps=16, np=8,
                 kp=FAKE, vp=FAKE)
        a.update(kw)
        return L.sv_append_kv_paged(a["k"], a["v"], a["dt"], a["ks"], a["vs"], a["sm"], a["rows"], a["Hkv"],
                                    a["D"], a["ps"], a["np"], a["kp"], a["vp"], None, None)
    for name in ("k", "v", "sm", "kp", "vp"):
        assert call(**{name: None}) == sv.SV_ERR_INVALID_ARG, name
    for name in ("k", "v", "kp", "vp"):
        assert call(**{name: MISALIGNED}) == sv.SV_ERR_INVALID_ARG, name
    for name in ("rows", "Hkv", "D", "ps", "np"):
        assert call(**{name: 0}) == sv.SV_ERR_INVALID_ARG, name
    assert call(dt=5) == sv.SV_ERR_INVALID_ARG
    assert call(ks=1016) == sv.SV_ERR_INVALID_ARG               # rows would overlap
    assert call(vs=1028) == sv.SV_ERR_INVALID_ARG               # rows off their 16-byte boundaries
    assert call(dt=sv.SV_F32, vs=1026) == sv.SV_ERR_INVALID_ARG
    assert call(D=100, ks=1024, vs=1024) == sv.SV_ERR_UNSUPPORTED
    assert call(D=512, ks=4096, vs=4096) == sv.SV_ERR_UNSUPPORTED
    assert call(np=1 << 24) == sv.SV_ERR_UNSUPPORTED


def test_append_rows_past_the_kernels_indexes(L):
    # 2^23 heads of 256: 2^31 elements a row
    assert L.sv_append_kv_paged(FAKE, FAKE, sv.SV_BF16, 1 << 31, 1 << 31, FAKE, 1, 1 << 23, 256, 1, 1, FAKE, FAKE,
                                None, None) == sv.SV_ERR_UNSUPPORTED


def test_chunk_attention_host_validation(L):
    def call(**kw):
        a = dict(q=FAKE, qs=4096, k=FAKE, v=FAKE, bt=FAKE, mp=8, np=64, ps=16, pl=FAKE, rs=FAKE, B=2, rows=9, Hq=32,
                 Hkv=8, D=128, scale=0.088, win=0, out=OTHER)
        a.update(kw)
        return L.sv_chunk_attention_paged(a["q"], a["qs"], a["k"], a["v"], a["bt"], a["mp"], a["np"], a["ps"], a["pl"],
                                          a["rs"], a["B"], a["rows"], a["Hq"], a["Hkv"], a["D"], a["scale"], a["win"],
                                          a["out"], None, None, None, 0, None)
    for name in ("q", "k", "v", "bt", "pl", "rs", "out"):
        assert call(**{name: None}) == sv.SV_ERR_INVALID_ARG, name
    for name in ("mp", "np", "ps", "B", "rows", "Hq", "Hkv", "D"):
        assert call(**{name: 0}) == sv.SV_ERR_INVALID_ARG, name
    for name in ("q", "k", "v", "out"):
        assert call(**{name: MISALIGNED}) == sv.SV_ERR_INVALID_ARG, name
    assert call(out=FAKE) == sv.SV_ERR_INVALID_ARG                 # written over its own queries
    assert call(qs=4088) == sv.SV_ERR_INVALID_ARG                  # rows would overlap
    assert call(qs=4100) == sv.SV_ERR_INVALID_ARG                  # rows off their 16-byte boundaries
    assert call(ps=24) == sv.SV_ERR_INVALID_ARG                    # neither a power of two nor a multiple of 128
    assert call(ps=4) == sv.SV_ERR_INVALID_ARG
    assert call(Hq=30) == sv.SV_ERR_INVALID_ARG                    # Hq % Hkv
    assert call(win=-1) == sv.SV_ERR_INVALID_ARG
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == sv.SV_ERR_INVALID_ARG, scale
    assert call(D=96) == sv.SV_ERR_UNSUPPORTED
    assert call(Hq=1032, Hkv=8, qs=1032 * 128) == sv.SV_ERR_UNSUPPORTED   # 129 heads a group
    assert call(B=4097) == sv.SV_ERR_UNSUPPORTED
    assert call(mp=1 << 26) == sv.SV_ERR_UNSUPPORTED               # max_pages * page_size
    assert call(np=1 << 24) == sv.SV_ERR_UNSUPPORTED               # rows of the cache
    assert call(rows=1 << 30) == sv.SV_ERR_UNSUPPORTED
    for kw in (dict(Hq=30, Hkv=8, D=128), dict(Hq=32, Hkv=8, D=96), dict(Hq=256, Hkv=1, D=64), dict(Hq=0, Hkv=1, D=64)):
        assert sv.sv_workspace_size(sv.SV_OP_CHUNK_ATTENTION, 0, 0, **kw) == 0


class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        if name.startswith("__"):
            raise AttributeError(name)

        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(api, "_lib", r)
    monkeypatch.setattr(api, "_on_device", lambda t: True)
    return r


def _i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def _refused(rec, fn, **kw):
    n = len(rec.calls)
    with pytest.raises((ValueError, TypeError)):
        fn(**kw)
    assert len(rec.calls) == n


def _build_kw():
    return dict(prefix_lens=_i32(3), new_lens=_i32(3), page_counts=_i32(3), block_table=_i32(3, 5),
                free_pages=_i32(20), free_count=_i32(1), page_size=16, num_rows=11, row_starts=_i32(4),
                slot_map=_i32(11), new_page_counts=_i32(3), new_free_count=_i32(1), seq_status=_i32(3),
                stream=STREAM)


def test_build_marshalling(rec):
    kw = _build_kw()
    got = api.sv_build_block_tables(**kw)
    name, a = rec.calls[-1]
    assert name == "sv_build_block_tables"
    assert a[5:10] == (3, 16, 5, 20, 11)     # B, page_size, max_pages, num_pages, num_rows
    order = ("prefix_lens", "new_lens", "page_counts", "free_pages", "free_count")
    assert list(a[:5]) == [kw[n].data_ptr() for n in order]
    assert list(a[10:16]) == [kw[n].data_ptr() for n in ("block_table", "row_starts", "slot_map",
                                                         "new_page_counts", "new_free_count", "seq_status")]
    assert [g is kw[n] for g, n in zip(got, ("row_starts", "slot_map", "new_page_counts", "new_free_count"))]


@pytest.mark.parametrize("name,bad", [
    ("prefix_lens", _i32(4)), ("new_lens", _i32(2)), ("page_counts", _i32(1)), ("free_count", _i32(2)),
    ("block_table", _i32(15)), ("free_pages", _i32(4, 5)), ("row_starts", _i32(3)), ("slot_map", _i32(12)),
    ("new_page_counts", _i32(4)), ("new_free_count", _i32(0)), ("seq_status", _i32(4)), ("page_size", 16.0),
    ("num_rows", -1), ("num_rows", True), ("prefix_lens", torch.zeros(3, dtype=torch.int64)),
    ("new_lens", [1, 2, 3]), ("page_counts", _i32(6)[::2]),
])
def test_build_refuses(rec, name, bad):
    kw = _build_kw()
    kw[name] = bad
    _refused(rec, api.sv_build_block_tables, **kw)


def _release_kw():
    return dict(keep_lens=_i32(3), page_counts=_i32(3), block_table=_i32(3, 5), free_pages=_i32(20),
                free_count=_i32(1), page_size=16, new_page_counts=_i32(3), new_free_count=_i32(1),
                seq_status=_i32(3), stream=STREAM)


def test_release_marshalling(rec):
    kw = _release_kw()
    api.sv_release_pages(**kw)
    name, a = rec.calls[-1]
    assert name == "sv_release_pages" and a[5:9] == (3, 16, 5, 20)
    assert list(a[:5]) == [kw[n].data_ptr() for n in ("keep_lens", "page_counts", "block_table", "free_pages",
                                                      "free_count")]


@pytest.mark.parametrize("name,bad", [
    ("keep_lens", _i32(2)), ("page_counts", _i32(4)), ("block_table", _i32(2, 5)), ("free_pages", _i32(2, 2)),
    ("free_count", _i32(3)), ("new_page_counts", _i32(2)), ("new_free_count", _i32(2)), ("seq_status", _i32(1)),
    ("page_size", None),
])
def test_release_refuses(rec, name, bad):
    kw = _release_kw()
    kw[name] = bad
    _refused(rec, api.sv_release_pages, **kw)


def _append_kw(dtype=torch.bfloat16):
    qkv = torch.zeros((6, 9, 8), dtype=dtype)
    return dict(k_new=qkv[:, 5:7], v_new=qkv[:, 7:9], slot_map=_i32(6),
                k_pages=torch.zeros((4, 2, 16, 8), dtype=torch.bfloat16),
                v_pages=torch.zeros((4, 2, 16, 8), dtype=torch.bfloat16), row_status=_i32(6), stream=STREAM)


@pytest.mark.parametrize("dtype,code", [(torch.bfloat16, sv.SV_BF16), (torch.float32, sv.SV_F32)])
def test_append_marshalling(rec, dtype, code):
    kw = _append_kw(dtype)
    api.sv_append_kv_paged(**kw)
    name, a = rec.calls[-1]
    assert name == "sv_append_kv_paged"
    assert a[2:5] == (code, 72, 72) and a[6:11] == (6, 2, 8, 16, 4)  # rows, Hkv, D, page_size, num_pages
    assert a[0] == kw["k_new"].data_ptr() and a[1] == kw["v_new"].data_ptr()


def test_append_refuses(rec):
    bf = torch.bfloat16
    for name, bad in (("k_new", torch.zeros((6, 3, 8), dtype=bf)), ("v_new", torch.zeros((5, 2, 8), dtype=bf)),
                      ("k_new", torch.zeros((6, 2, 8), dtype=torch.float16)),
                      ("v_new", torch.zeros((6, 2, 8), dtype=torch.float32)),
                      ("k_new", torch.zeros((6, 2, 16), dtype=bf)[:, :, ::2]),
                      ("k_new", torch.zeros((2, 6, 8), dtype=bf).transpose(0, 1)),
                      ("slot_map", _i32(7)), ("slot_map", torch.zeros(6)), ("row_status", _i32(5)),
                      ("v_pages", torch.zeros((4, 2, 8, 8), dtype=bf)),
                      ("k_pages", torch.zeros((4, 2, 16, 8)))):
        kw = _append_kw()
        kw[name] = bad
        _refused(rec, api.sv_append_kv_paged, **kw)


def _chunk_kw():
    qkv = torch.zeros((6, 8, 64), dtype=torch.bfloat16)
    pages = torch.zeros((9, 2, 16, 64), dtype=torch.bfloat16)
    return dict(q=qkv[:, :4], k_pages=pages, v_pages=pages.clone(), block_table=_i32(3, 5), prefix_lens=_i32(3),
                row_starts=_i32(4), window=7, out=torch.zeros((6, 4, 64), dtype=torch.bfloat16),
                lse=torch.zeros((6, 4)), seq_status=_i32(3), ws=torch.zeros(256, dtype=torch.uint8), stream=STREAM)


def test_chunk_attention_marshalling(rec):
    kw = _chunk_kw()
    out, lse = api.sv_chunk_attention_paged(**kw)
    name, a = rec.calls[-1]
    assert name == "sv_chunk_attention_paged" and out is kw["out"] and lse is kw["lse"]
    assert a[1] == 512 and a[5:8] == (5, 9, 16)            # row stride; max_pages, num_pages, page_size
    assert a[10:15] == (3, 6, 4, 2, 64)                    # B, num_rows, Hq, Hkv, D
    assert a[15] == pytest.approx(64 ** -0.5) and a[16] == 7
    order = ((0, "q"), (2, "k_pages"), (3, "v_pages"), (4, "block_table"), (8, "prefix_lens"), (9, "row_starts"),
             (17, "out"), (18, "lse"), (19, "seq_status"), (20, "ws"))
    assert all(a[i] == kw[n].data_ptr() for i, n in order) and a[21] == 256
    del kw["lse"]
    assert api.sv_chunk_attention_paged(**kw) is kw["out"]
    assert rec.calls[-1][1][18] is None
    out, lse = api.sv_chunk_attention_paged(**kw, return_lse=True)
    assert lse.shape == (6, 4) and lse.dtype == torch.float32


def test_chunk_attention_refuses(rec):
    bf = torch.bfloat16
    for name, bad in (("q", torch.zeros((6, 4, 128), dtype=bf)), ("q", torch.zeros((6, 4, 64))), ("q", None),
                      ("q", torch.zeros((4, 6, 64), dtype=bf).transpose(0, 1)), ("k_pages", torch.zeros((9, 2, 16), dtype=bf)),
                      ("v_pages", torch.zeros((9, 2, 8, 64), dtype=bf)), ("block_table", _i32(4, 5)),
                      ("block_table", _i32(15)), ("block_table", torch.zeros((3, 5), dtype=torch.int64)),
                      ("prefix_lens", _i32(4)), ("row_starts", _i32(3)), ("window", 2.0), ("window", None),
                      ("out", torch.zeros((6, 4, 32), dtype=bf)), ("lse", torch.zeros((4, 6))),
                      ("lse", torch.zeros((6, 4), dtype=torch.float64)), ("seq_status", _i32(2)),
                      ("ws", torch.zeros(8))):
        kw = _chunk_kw()
        kw[name] = bad
        _refused(rec, api.sv_chunk_attention_paged, **kw)


def test_arrays_on_other_devices_are_refused(rec):
    for fn, kw, name in ((api.sv_build_block_tables, _build_kw(), "new_lens"),
                         (api.sv_release_pages, _release_kw(), "free_pages"),
                         (api.sv_append_kv_paged, _append_kw(), "slot_map"),
                         (api.sv_append_kv_paged, _append_kw(), "k_new"),
                         (api.sv_chunk_attention_paged, _chunk_kw(), "row_starts"),
                         (api.sv_chunk_attention_paged, _chunk_kw(), "q"),
                         (api.sv_chunk_attention_paged, _chunk_kw(), "ws")):
        kw[name] = kw[name].to("meta")
        _refused(rec, fn, **kw)


@pytest.mark.parametrize("current,given", [(1, False), (0, False), (0, True), (1, True)])
def test_launch_makes_the_tensors_device_and_the_stream_current(monkeypatch, current, given):
    """The call's device and the given stream are current while it allocates
    and launches, and what was current before is again afterwards."""
    log = []

    class Context:
        def __init__(self, what):
            self.what = what

        def __enter__(self):
            log.append(("enter", self.what))

        def __exit__(self, *exc):
            log.append(("exit", self.what))

    stream = types.SimpleNamespace(cuda_stream=77)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(torch.cuda, "device", lambda d: Context(d.index))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: Context(s))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=100 + d.index))
    with api._Launch(torch.device("cuda", 1), stream if given else None) as handle:
        assert handle == (77 if given else 101)
        inside = list(log)
    want = ([1] if current != 1 else []) + ([stream] if given else [])
    assert inside == [("enter", w) for w in want]
    assert log[len(inside):] == [("exit", w) for w in reversed(want)]
