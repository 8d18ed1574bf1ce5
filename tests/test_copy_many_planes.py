"""Copies of pages of more planes than a launch takes: K and V in 4 bits of a model of
many layers are four planes a layer."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv
from speculative_decoding_verification_81_gb300 import api
from test_pages_binding import STREAM, _i32, _refused
from test_pages_binding import rec  # noqa: F401  (a fixture)

u8 = torch.uint8


def planes(n, x=(64, 4)):
    return [torch.zeros((9, 2, 16, x[i % len(x)]), dtype=u8) for i in range(n)]


@pytest.mark.parametrize("n", [1, 63, 64, 65, 128, 320])
@pytest.mark.parametrize("kind", [list, tuple])
def test_launches_of_64_planes(rec, n, kind):  # noqa: F811
    p, copies, status = planes(n), _i32(3, 3), _i32(3)
    api.sv_copy_pages(copies, kind(p), status, stream=STREAM)
    assert [name for name, _ in rec.calls] == ["sv_copy_pages"] * (-(-n // 64))
    at = 0
    for _, a in rec.calls:
        m = a[4]
        assert m == min(64, n - at) and a[0] == copies.data_ptr() and a[8] == status.data_ptr() and a[9] == STREAM.cuda_stream
        assert (a[1], a[5], a[6], a[7]) == (3, 2, 16, 9)
        assert list(a[2]) == [t.data_ptr() for t in p[at:at + m]]
        assert list(a[3]) == [t.shape[3] for t in p[at:at + m]]
        at += m
    assert at == n


def test_a_plane_that_is_refused_leaves_every_plane_alone(rec, monkeypatch):  # noqa: F811
    monkeypatch.setattr(api, "status_string", str)  # (the recorder has none)
    wide = torch.zeros((9, 2, 16, 8192), dtype=u8)
    off = torch.zeros(9 * 2 * 16 * 4 + 4, dtype=u8)[4:].view(9, 2, 16, 4)
    for bad, code in ((planes(1, (6,))[0], sv.SV_ERR_INVALID_ARG), (off, sv.SV_ERR_INVALID_ARG),
                      (torch.zeros((9, 2, 16, 0), dtype=u8), sv.SV_ERR_INVALID_ARG), (wide, sv.SV_ERR_UNSUPPORTED)):
        with pytest.raises(sv.SpecVerifyError) as e:
            api.sv_copy_pages(_i32(3, 3), planes(100) + [bad], stream=STREAM)
        assert e.value.status == code and not rec.calls
    _refused(rec, api.sv_copy_pages, copies=_i32(3, 3), planes=planes(100) + [planes(1)[0][:8]], stream=STREAM)


@pytest.mark.gpu
@pytest.mark.parametrize("layers", [16, 17, 32, 80, 300])
@pytest.mark.parametrize("stream", [False, True])
def test_every_layer_in_one_call(layers, stream):
    rng = np.random.default_rng(layers)
    n, hkv, ps = 9, 2, 8
    cache = []
    for _ in range(layers):
        for _ in range(2):
            cache.append(torch.randint(0, 256, (n, hkv, ps, 32), dtype=u8, device="cuda"))
            cache.append(torch.randn((n, hkv, ps, 2), device="cuda").to(torch.bfloat16))
    ids = rng.permutation(n)
    copies = [[ids[0], ids[1], 5], [-1, -1, 0], [ids[2], ids[3], 8], [ids[4], n, 2]]
    want = [t.clone() for t in cache]
    for w in want:
        w[ids[1], :, :5] = w[ids[0], :, :5]
        w[ids[3]] = w[ids[2]]
    st = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    sv.sv_copy_pages(torch.tensor(copies, dtype=torch.int32, device="cuda"), cache, copy_status=st,
                     **(dict(stream=side) if stream else {}))
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0, 0, sv.SV_ERR_BAD_INPUT]
    assert all(torch.equal(t.view(u8), w.view(u8)) for t, w in zip(cache, want))
