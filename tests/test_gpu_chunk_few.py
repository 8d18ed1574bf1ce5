"""Attention of few rows over the paged cache: the form a call takes for them
(up to 32 sequences, 8 query heads a KV head, room for a cluster of CTAs a row and
KV head) at the sizes where it can go wrong, and the other form on the same
sequences, which a batch of more than 32 sequences takes, most of them empty."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv
from test_gpu_chunk import Case, SMALL, i32, near

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.mark.parametrize("i", range(len(SMALL)))
def test_the_other_form(i):
    lens, kw = SMALL[i]
    Case(lens + [(0, 0)] * 33, seed=i, spare_rows=i % 3, **kw).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("g", range(1, 9))
def test_heads(g, d):
    Case([(100, 1), (0, 1), (333, 2)], hq=2 * g, hkv=2, d=d, page_size=8, seed=g, strided=g % 2 == 0).check()


@pytest.mark.parametrize("past", [0, 1, 6, 7, 8, 9, 14, 15, 16, 17, 127, 128, 129, 255, 256, 511, 512, 1023, 1024])
def test_lengths(past):
    Case([(past, 1)], hq=8, hkv=2, page_size=8 if past % 2 else 16, seed=past).check()


@pytest.mark.parametrize("lens,kw", [
    ([(100, 1)], dict(hq=4, hkv=1)),                         # one CTA a row and head
    ([(200, 1)], dict(hq=4, hkv=1)),                         # two
    ([(500, 1)], dict(hq=32, hkv=8, page_size=128)),         # four
    ([(1000, 1)], dict(hq=14, hkv=2, d=64)),                 # eight
    ([(32000, 1)], dict(hq=8, hkv=1, page_size=256)),        # sixteen, 15 units a warp
    ([(30000, 1)], dict(hq=6, hkv=2, d=64, page_size=8)),
    ([(65400, 1)], dict(hq=2, hkv=1, d=64, page_size=64)),   # all 32 units of a warp
    ([(32750, 1)], dict(hq=32, hkv=8, page_size=8)),
    ([(16000, 1)], dict(hq=32, hkv=8, page_size=384)),
    ([(880, 128)], dict(hq=8, hkv=1)),                       # 128 rows of one sequence, a CTA each
    ([(0, 16)], dict(hq=32, hkv=8)),
    ([(4000, 1), (0, 1)], dict(hq=32, hkv=8, page_size=64)),  # uneven
    ([(0, 0), (5, 1), (0, 0), (70, 2), (0, 0)], dict(hq=8, hkv=2)),
    ([(int(x), 1) for x in np.random.default_rng(1).integers(0, 300, 32)], dict(hq=4, hkv=4, d=64)),
    ([(int(x), 1) for x in np.random.default_rng(2).integers(0, 300, 33)], dict(hq=4, hkv=4, d=64)),  # one too many
])
def test_sizes(lens, kw):
    Case(lens, seed=3, spare_rows=len(lens) % 2, **kw).check()


@pytest.mark.parametrize("window", [1, 2, 7, 8, 9, 15, 16, 17, 100, 1000])
@pytest.mark.parametrize("kw", [dict(hq=8, hkv=2, page_size=8), dict(hq=7, hkv=1, d=64, page_size=128)])
def test_windows(window, kw):
    Case([(3, 1), (700, 3), (1021, 1), (5000, 2)], window=window, seed=window, **kw).check()


def test_offsets_past_32_bits():
    hkv, ps, d = 8, 16, 128
    num_pages = (1 << 25) // (hkv * ps) + 20
    c = Case([(100, 1)], hq=16, hkv=hkv, page_size=ps, seed=9)
    few = c.k.shape[0]
    k = torch.empty((num_pages, hkv, ps, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[-few:], v[-few:] = c.k, c.v
    want = c.want()
    real = (c.table >= 0) & (c.table < few)
    c.table = torch.where(real, c.table + num_pages - few, c.table)
    c.k, c.v = k, v
    near(*c.run(), want)


@pytest.mark.parametrize("empty", [0, 33])
def test_bad_sequences_are_reported_and_left(empty):
    c = Case([(40, 3), (20, 2), (60, 1), (10, 4), (5, 2)] + [(0, 0)] * empty, seed=10)
    o, _, ob, _ = c.want()  # (before the table names a page that does not exist)
    past, starts = list(c.past), list(c.starts)
    past[1] = -1                       # no such length
    past[2] = c.table.shape[1] * 16    # past the table
    c.table[3, 0] = c.k.shape[0]       # a page that does not exist
    starts[5] = len(c.q) + 1           # rows past the batch
    if empty:
        starts[6:] = [12] * empty      # (after it, in order with none)
    st = torch.full((5 + empty,), -7, dtype=torch.int32, device="cuda")
    out = torch.full(c.q.shape, 777.0, dtype=torch.bfloat16, device="cuda")
    sv.sv_chunk_attention_paged(c.q, c.k, c.v, c.table, i32(past), i32(starts), scale=c.scale, out=out,
                                seq_status=st)
    torch.cuda.synchronize()
    bad = sv.SV_ERR_BAD_INPUT
    assert st[:5].tolist() == [0, bad, bad, bad, bad]
    assert (out[3:6] == 777.0).all() and (out[10:] == 777.0).all()
    assert ((out.double() - o).abs() <= ob)[:3].all()


def test_large_scores_and_moving_maximum():
    for seed in range(4):
        Case([(900, 2)], hq=8, hkv=2, seed=seed, q_scale=12.0).check()


def test_rows_of_others_do_not_matter():
    c = Case([(300, 2), (40, 3), (7, 1)], hq=8, hkv=2, seed=20, spare_rows=4)
    want = c.want()
    q = c.q.clone()
    q[6:] = NAN
    q[2:5] = float("inf")
    c.q = q
    out, lse = c.run()
    o, e, ob, eb = want
    for rows in (slice(0, 2), slice(5, 6)):
        assert ((out.double() - o).abs() <= ob)[rows].all() and ((lse.double() - e).abs() <= eb)[rows].all()


def test_captured_repeated_and_on_two_streams():
    """A captured call follows the lengths on the device; repeats and streams change no bit."""
    c = Case([(1500, 1), (700, 1)], hq=32, hkv=8, seed=13)
    past, starts = i32(c.past), i32(c.starts)

    def call(**kw):
        return sv.sv_chunk_attention_paged(c.q, c.k, c.v, c.table, past, starts, scale=c.scale, return_lse=True, **kw)

    want = call()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [call(stream=s) for _ in range(10) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(e, want[1]) for o, e in got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = call()
    for lens in ([1500, 700], [30, 0], [1500, 1], [64, 700]):
        past.copy_(i32(lens))
        c.past = lens
        g.replay()
        torch.cuda.synchronize()
        near(out, lse, c.want())
