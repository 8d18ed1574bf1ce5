"""Chunk attention's uses that its form for few rows and its general form share,
on both: the same sequences alone, and beside enough empty ones that the
general form takes the call.  Which form ran is read from the words in which
each counts its calls in the workspace."""
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv
from test_gpu_chunk import NAN, Case, i32, near
from test_gpu_chunk_giveup import EMPTY, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["few", "general"])
def form(request):
    return request.param


def lens_for(form, lens):
    return lens + EMPTY if form == "general" else lens


def ran(ws):
    general, _, few, _ = ws[:32].view(torch.int64).tolist()
    assert (general > 0) != (few > 0)
    return "general" if general else "few"


def test_pages_shared_by_sequences(form):
    """A prefix's pages in the tables of several sequences, one of them twice."""
    c = Case(lens_for(form, [(64, 20), (64, 1), (64, 3)]), hq=8, hkv=2, seed=21)
    c.table[1:3, :4] = c.table[0, :4]
    c.table[2, 3] = c.table[2, 2]
    ws = workspace(c)
    c.check(ws=ws)
    assert ran(ws) == form


def test_one_page_behind_every_entry(form):
    c = Case(lens_for(form, [(100, 7), (60, 1)]), hq=8, hkv=2, d=64, page_size=8, seed=25)
    one = int(c.table[0, 0])
    c.table[:2] = one
    c.k[one], c.v[one] = torch.randn_like(c.k[one]), torch.randn_like(c.v[one])
    ws = workspace(c)
    c.check(ws=ws)
    assert ran(ws) == form


@pytest.mark.parametrize("scale", [0.7, 1e-6, 30.0])
def test_scale_and_equal_scores(form, scale):
    c = Case(lens_for(form, [(500, 20)]), hq=4, hkv=2, scale=scale, seed=7)
    c.check()
    c.k[~torch.isnan(c.k)] = 0.0  # equal weights: the mean of V
    ws = workspace(c)
    c.check(ws=ws)
    assert ran(ws) == form


@pytest.mark.parametrize("window", [10 ** 6, 2 ** 31 - 1])
def test_a_window_longer_than_the_table_hides_nothing(form, window):
    c = Case(lens_for(form, [(700, 40), (5, 1)]), hq=4, hkv=2, seed=22)
    want = c.run()
    c.window = window
    ws = workspace(c)
    got = c.run(ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ran(ws) == form


def test_single_tokens_agree_with_verification_attention(form):
    c = Case(lens_for(form, [(700, 1), (64, 1), (3, 1)]), hq=32, hkv=8, seed=12)
    ws = workspace(c)
    c.check(ws=ws)
    assert ran(ws) == form
    k, v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    tree = sv.sv_tree_attention_paged(c.q[:3].unsqueeze(1).contiguous(), k, v, c.table[:3].contiguous(), i32(c.past[:3]),
                                      scale=c.scale)
    o, _, ob, _ = c.want()
    assert ((tree.squeeze(1).double() - o).abs() <= ob).all()


def test_a_maximum_that_moves(form):
    """Scores whose maximum grows along the slots, so that sums are rescaled again and again."""
    c = Case(lens_for(form, [(900, 6)]), hq=4, hkv=2, seed=6, q_scale=4.0)
    n = 906
    ramp = torch.linspace(0.1, 4.0, n, device="cuda")
    s = torch.arange(n, device="cuda")
    pg = c.table[0].long()[s // 16]
    c.k[pg, :, s % 16] = (c.k[pg, :, s % 16].float() * ramp[:, None, None]).to(torch.bfloat16)
    ws = workspace(c)
    c.check(ws=ws)
    assert ran(ws) == form


def test_rows_a_little_apart_and_an_output_off_a_wide_boundary(form):
    c = Case(lens_for(form, [(300, 11), (90, 1), (64, 5)]), hq=4, hkv=2, d=64, seed=23)
    want = c.run()
    rows, hq, d = c.q.shape
    buf = torch.zeros(rows * hq * d + 16, dtype=torch.bfloat16, device="cuda")
    off = 8 if buf.data_ptr() % 32 == 0 else 0
    wide = torch.full((rows, hq * d + 8), NAN, dtype=torch.bfloat16, device="cuda")
    wide[:, :hq * d] = c.q.reshape(rows, -1)
    c.q = wide.as_strided((rows, hq, d), (hq * d + 8, d, 1))
    ws = workspace(c)
    got = c.run(out=buf[off:off + rows * hq * d].view(rows, hq, d), ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ran(ws) == form


def test_rows_behind_the_last_sequence_stay_and_repeats_are_equal(form):
    c = Case(lens_for(form, [(1000, 1), (700, 9), (50, 2)]), hq=8, hkv=2, seed=8, spare_rows=5)
    ws = workspace(c)
    a = c.check(ws=ws)  # (its output and log-sum-exp keep what they held in rows of no sequence)
    near(*a, c.want())
    live = slice(0, sum(c.new))
    for _ in range(5):
        b = c.run(ws=ws)
        assert torch.equal(a[0][live], b[0][live]) and torch.equal(a[1][live], b[1][live])
    assert ran(ws) == form
