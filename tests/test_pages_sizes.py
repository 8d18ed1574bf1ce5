"""Sizes past 32 bits in the paged-cache calls: refused by the binding, not cut
to their low 32 bits on the way to the library (without a GPU; the large
arrays are shapes without memory)."""
import types

import pytest
import torch

from speculative_decoding_verification_81_gb300 import api
from test_pages_binding import Recorder

STREAM = types.SimpleNamespace(cuda_stream=0)
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(api, "_lib", r)
    monkeypatch.setattr(api, "_on_device", lambda t: True)
    return r


def meta(shape, dtype=I32):
    return torch.empty(shape, dtype=dtype, device="meta")


def build(B=3, max_pages=5, num_pages=20, page_size=16, num_rows=11):
    return api.sv_build_block_tables(meta(B), meta(B), meta(B), meta((B, max_pages)), meta(num_pages), meta(1), page_size,
                                     num_rows, slot_map=meta(num_rows), stream=STREAM)


def release(B=3, max_pages=5, num_pages=20, page_size=16):
    return api.sv_release_pages(meta(B), meta(B), meta((B, max_pages)), meta(num_pages), meta(1), page_size, stream=STREAM)


def append(rows=6, hkv=2, d=8, num_pages=4, page_size=16):
    pages = meta((num_pages, hkv, page_size, d), BF)
    return api.sv_append_kv_paged(meta((rows, hkv, d), BF), meta((rows, hkv, d), BF), meta(rows), pages, pages, stream=STREAM)


def chunk(rows=6, hq=4, hkv=2, d=64, num_pages=9, page_size=16, B=3, max_pages=5, window=7):
    pages = meta((num_pages, hkv, page_size, d), BF)
    return api.sv_chunk_attention_paged(meta((rows, hq, d), BF), pages, pages, meta((B, max_pages)), meta(B), meta(B + 1),
                                        window=window, out=meta((rows, hq, d), BF), ws=meta(256, torch.uint8),
                                        stream=STREAM)


@pytest.mark.parametrize("fn,names", [
    (build, ("B", "max_pages", "num_pages", "page_size", "num_rows")),
    (release, ("B", "max_pages", "num_pages", "page_size")),
    (append, ("rows", "hkv", "d", "num_pages", "page_size")),
    (chunk, ("rows", "hq", "hkv", "d", "num_pages", "page_size", "B", "max_pages", "window")),
])
def test_sizes_past_32_bits_are_refused(rec, fn, names):
    fn()
    assert len(rec.calls) == 1
    for name in names:
        for value in (1 << 31, (1 << 32) + 5, (1 << 40) + 16):
            with pytest.raises(ValueError):
                fn(**{name: value})
    assert len(rec.calls) == 1


def test_negative_sizes_past_32_bits_are_refused(rec):
    for call in (lambda: build(page_size=16 - (1 << 32)), lambda: release(page_size=16 - (1 << 32)),
                 lambda: chunk(window=5 - (1 << 32))):
        with pytest.raises(ValueError):
            call()
    assert not rec.calls


def test_sizes_of_31_bits_are_passed_on(rec):
    chunk(window=(1 << 31) - 1)
    assert rec.calls[-1][1][16] == (1 << 31) - 1
