"""A stream of another device than the tensors' is refused before anything is
allocated or launched (stand-ins: no GPU)."""
import types

import pytest
import torch

from speculative_decoding_verification_81_gb300 import api
from test_pages_binding import Recorder, _append_kw, _build_kw, _chunk_kw, _release_kw


def stream_of(device):
    return types.SimpleNamespace(cuda_stream=77, device=torch.device(device))


@pytest.mark.parametrize("name,kw", [("sv_build_block_tables", _build_kw), ("sv_release_pages", _release_kw),
                                     ("sv_append_kv_paged", _append_kw), ("sv_chunk_attention_paged", _chunk_kw)])
def test_a_stream_of_another_device_is_refused(monkeypatch, name, kw):
    rec = Recorder()
    monkeypatch.setattr(api, "_lib", rec)
    monkeypatch.setattr(api, "_on_device", lambda t: True)
    getattr(api, name)(**{**kw(), "stream": stream_of("cpu")})  # the tensors' own
    assert rec.calls[-1][1][-1] == 77
    with pytest.raises(ValueError):
        getattr(api, name)(**{**kw(), "stream": stream_of("cuda:1")})
    assert len(rec.calls) == 1


def test_the_check_comes_before_any_device_is_touched(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: pytest.fail("asked for the device"))
    with pytest.raises(ValueError):
        api._Launch(torch.device("cuda", 0), stream_of("cuda:1"))
