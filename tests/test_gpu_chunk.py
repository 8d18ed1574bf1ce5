"""Attention of chunks over the paged cache against its definition in 64 bits
(bounds in chunk_ref.py), its refusals, and a run of the paged-cache calls
together as a server makes them."""
import numpy as np
import pytest
import torch

import chunk_ref
import pages_oracle as po
import speculative_decoding_verification_81_gb300 as sv

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Case:
    """A pool with the sequences' pages anywhere in it; slots that no row sees
    hold NaN, and table entries of pages without a seen slot name no page."""

    def __init__(self, lens, hq=8, hkv=2, d=128, page_size=16, window=0, seed=0, scale=None, strided=False,
                 spare_rows=0, q_scale=1.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.past, self.new = [l[0] for l in lens], [l[1] for l in lens]
        self.window, self.page_size = window, page_size
        self.scale = d ** -0.5 if scale is None else scale
        need = [-(-(a + n) // page_size) for a, n in lens]
        max_pages = max(need) + 2
        num_pages = sum(need) + 3
        ids = rng.permutation(num_pages)
        table = np.full((len(lens), max_pages), 10 ** 6, np.int64)
        table[:, 1::2] = -1

        def randn(*shape):
            return torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)

        self.k = torch.full((num_pages, hkv, page_size, d), NAN, dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        used = 0
        for b, (a, n) in enumerate(lens):
            lo = max(0, a - window + 1) if window else 0
            first = lo // page_size if n else need[b]
            for j in range(first, need[b]):
                table[b, j] = ids[used + j]
            used += need[b]
            if n:
                s = torch.arange(lo, a + n, device="cuda")
                pg = i32(table[b])[s // page_size].long()
                self.k[pg, :, s % page_size] = randn(a + n - lo, hkv, d)
                self.v[pg, :, s % page_size] = randn(a + n - lo, hkv, d)
        self.table = i32(table)
        self.starts = np.concatenate([[0], np.cumsum(self.new)])
        rows = int(self.starts[-1]) + spare_rows
        q = randn(max(rows, 1), hq + (2 * hkv if strided else 0), d) * q_scale
        self.q = q[:, :hq] if strided else q

    def run(self, **kw):
        return sv.sv_chunk_attention_paged(self.q, self.k, self.v, self.table, i32(self.past), i32(self.starts),
                                           scale=self.scale, window=self.window, return_lse=True, **kw)

    def want(self):
        return chunk_ref.attention(self.q, self.k, self.v, self.table, self.past, self.new, self.starts, self.scale,
                                   self.window)

    def check(self, **kw):
        st = torch.full((len(self.past),), -7, dtype=torch.int32, device="cuda")
        rows, hq, d = self.q.shape
        out = torch.full((rows, hq, d), 777.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((rows, hq), 777.0, device="cuda")
        self.run(out=out, lse=lse, seq_status=st, **kw)
        torch.cuda.synchronize()
        assert (st == 0).all(), st
        near(out, lse, self.want())
        return out, lse


def near(out, lse, want):
    o, e, ob, eb = want
    have = ~torch.isnan(e)
    assert (lse[~have] == 777.0).all() and (out[~have] == 777.0).all()  # rows of no sequence: as they were
    for name, d, bound in (("out", (out.double() - o).abs()[have], ob[have]),
                           ("lse", (lse.double() - e).abs()[have], eb[have])):
        assert torch.isfinite(d).all()
        assert (d <= bound).all(), f"{name} off by up to {(d / bound).nan_to_num().max().item()} of its bound"


SMALL = [
    # lens (slots before, new rows), then the shape
    ([(0, 1)], {}),
    ([(1, 1)], dict(d=64)),
    ([(127, 1)], dict(hq=32, hkv=8)),
    ([(128, 1)], dict(hq=32, hkv=8)),
    ([(511, 1)], dict(hq=32, hkv=8)),
    ([(4095, 1)], dict(hq=32, hkv=8, page_size=128)),
    ([(0, 2)], {}),
    ([(0, 128)], dict(hq=4, hkv=4)),
    ([(0, 129)], dict(hq=4, hkv=4, d=64)),
    ([(100, 700)], dict(hq=8, hkv=2, page_size=64)),
    ([(1, 257)], dict(hq=16, hkv=16, d=64, page_size=8)),
    ([(300, 33), (0, 0), (5, 1), (0, 64), (64, 65), (1000, 9)], dict(hq=32, hkv=8)),
    ([(37, 1), (500, 1), (0, 1), (128, 1), (255, 1), (256, 1), (900, 1)], dict(hq=8, hkv=1, page_size=256)),
    ([(20, 50), (700, 3)], dict(hq=14, hkv=2, d=64, page_size=32)),      # 7 heads a group: 18 tokens a tile
    ([(10, 5), (200, 11)], dict(hq=128, hkv=1, page_size=128)),          # one token a tile
    ([(130, 6)], dict(hq=100, hkv=1, d=64)),                             # 100 heads a group
    ([(77, 40), (0, 300)], dict(hq=5, hkv=1, page_size=384)),            # 25 tokens a tile, odd pages
    ([(20000, 1)], dict(hq=32, hkv=8, page_size=64)),                    # one token over many CTAs
    ([(9000, 70), (3, 2)], dict(hq=8, hkv=1)),
]


@pytest.mark.parametrize("i", range(len(SMALL)))
def test_chunks(i):
    lens, kw = SMALL[i]
    Case(lens, seed=i, spare_rows=i % 3, strided=i % 2 == 1, **kw).check()


@pytest.mark.parametrize("window", [1, 2, 17, 128, 129, 640])
@pytest.mark.parametrize("lens,kw", [
    ([(0, 300), (1000, 1), (3, 1), (700, 64)], dict(hq=8, hkv=2, page_size=16)),
    ([(2000, 140), (255, 3)], dict(hq=6, hkv=6, d=64, page_size=128)),
])
def test_windows(window, lens, kw):
    Case(lens, window=window, seed=window, **kw).check()


@pytest.mark.parametrize("n,past_hi,kw", [
    (300, 200, dict(hq=32, hkv=8)),        # more sequences than CTAs, each a tile or two
    (1500, 5, dict(hq=2, hkv=1, d=64)),    # more sequences than threads of a CTA
    (33, 3000, dict(hq=8, hkv=8, page_size=128)),
])
def test_many_single_tokens(n, past_hi, kw):
    rng = np.random.default_rng(n)
    Case([(int(x), 1) for x in rng.integers(0, past_hi, n)], seed=n, **kw).check()


def test_mixed_batch():
    rng = np.random.default_rng(5)
    lens = [(int(a), int(b)) for a, b in zip(rng.integers(0, 1500, 40), rng.choice([0, 1, 1, 1, 5, 60, 200], 40))]
    Case(lens, hq=32, hkv=8, page_size=64, seed=5, strided=True).check()


def test_large_scores_and_moving_maximum():
    """Scores of hundreds, whose maximum grows along the slots: O is rescaled again and again."""
    c = Case([(900, 140)], hq=4, hkv=2, seed=6, q_scale=4.0)
    ramp = torch.linspace(0.1, 4.0, 1040, device="cuda").to(torch.bfloat16)
    s = torch.arange(1040, device="cuda")
    pg = c.table[0].long()[s // 16]
    c.k[pg, :, s % 16] = (c.k[pg, :, s % 16].float() * ramp[:, None, None].float()).to(torch.bfloat16)
    c.check()


def test_scale_and_equal_scores():
    c = Case([(500, 20)], hq=4, hkv=2, scale=0.7, seed=7)
    c.k[~torch.isnan(c.k)] = 0.0  # equal weights: the mean of V
    c.check()


def test_repeats_bit_for_bit():
    c = Case([(3000, 1), (700, 300), (50, 9)], hq=32, hkv=8, seed=8)
    a = c.run()
    for _ in range(5):
        b = c.run()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_of_others_do_not_matter():
    """NaN and infinity in the query rows of no sequence, and in a neighbour's
    rows, reach no other row: rows share products but not sums."""
    c = Case([(300, 5), (40, 70), (7, 1), (1000, 1)], hq=8, hkv=2, seed=20, spare_rows=9)
    want = c.want()
    q = c.q.clone()
    q[77:] = NAN
    q[5:75] = float("inf")  # the second sequence's
    c.q = q
    out, lse = c.run()
    o, e, ob, eb = want
    for rows in (slice(0, 5), slice(75, 77)):
        assert ((out.double() - o).abs() <= ob)[rows].all() and ((lse.double() - e).abs() <= eb)[rows].all()


def test_pages_shared_by_sequences():
    """A prefix's pages in the tables of several sequences, one of them twice."""
    c = Case([(64, 20), (64, 1), (64, 3)], hq=8, hkv=2, seed=21)
    c.table[1:, :4] = c.table[0, :4]
    c.table[2, 3] = c.table[2, 2]
    c.check()


@pytest.mark.parametrize("window", [10 ** 6, 2 ** 31 - 1])
def test_a_window_longer_than_the_table_hides_nothing(window):
    c = Case([(700, 40), (5, 1)], hq=4, hkv=2, seed=22)
    want = c.run()
    c.window = window
    got = c.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_alignments_and_strides():
    """An output 16 bytes off a 32-byte boundary, and rows of q a little apart."""
    c = Case([(300, 70), (90, 1), (64, 17)], hq=4, hkv=2, d=64, seed=23)
    want = c.run()
    rows, hq, d = c.q.shape
    buf = torch.zeros(rows * hq * d + 16, dtype=torch.bfloat16, device="cuda")
    off = 8 if buf.data_ptr() % 32 == 0 else 0
    out = buf[off:off + rows * hq * d].view(rows, hq, d)
    wide = torch.full((rows, hq * d + 8), NAN, dtype=torch.bfloat16, device="cuda")
    wide[:, :hq * d] = c.q.reshape(rows, -1)
    c.q = wide.as_strided((rows, hq, d), (hq * d + 8, d, 1))
    got = c.run(out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(sv.SpecVerifyError):  # rows 2 bytes off their 16-byte boundary
        c.q = wide.as_strided((rows, hq, d), (hq * d + 1, d, 1))
        c.run()
    with pytest.raises(sv.SpecVerifyError):  # written over its own queries
        c.q = out
        c.run(out=out)


@pytest.mark.parametrize("lens,kw", [
    ([(30, 2100)], dict(hq=128, hkv=1, d=64)),                 # 1050 items a head: two rounds of the search
    ([(int(x), 1) for x in np.random.default_rng(24).integers(0, 40, 4096)], dict(hq=1, hkv=1, d=64, page_size=8)),
])
def test_many_items(lens, kw):
    Case(lens, seed=24, **kw).check()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements, the sequence's pages at its end."""
    hkv, ps, d = 8, 16, 128
    num_pages = (1 << 25) // (hkv * ps) + 40
    lens = [(300, 70), (200, 1)]
    c = Case(lens, hq=16, hkv=hkv, page_size=ps, seed=9)
    few = c.k.shape[0]
    k = torch.empty((num_pages, hkv, ps, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[-few:], v[-few:] = c.k, c.v
    want = c.want()
    real = (c.table >= 0) & (c.table < few)
    c.table = torch.where(real, c.table + num_pages - few, c.table)
    c.k, c.v = k, v
    out, lse = c.run()
    near(out, lse, want)


def test_bad_sequences_are_reported_and_left():
    c = Case([(40, 3), (20, 2), (60, 1), (10, 4), (5, 2)], seed=10)
    past, starts = list(c.past), list(c.starts)
    past[1] = -1                       # no such length
    past[2] = c.table.shape[1] * 16    # past the table
    c.table[3, 0] = c.k.shape[0]       # a page that does not exist
    starts[5] = len(c.q) + 1           # rows past the batch
    st = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    out = torch.full(c.q.shape, 777.0, dtype=torch.bfloat16, device="cuda")
    sv.sv_chunk_attention_paged(c.q, c.k, c.v, c.table, i32(past), i32(starts), scale=c.scale, out=out,
                                seq_status=st)
    torch.cuda.synchronize()
    bad = sv.SV_ERR_BAD_INPUT
    assert st.tolist() == [0, bad, bad, bad, bad]
    assert (out[3:6] == 777.0).all() and (out[10:] == 777.0).all()
    o, _, ob, _ = chunk_ref.attention(c.q, c.k, c.v, c.table, c.past[:1], c.new[:1], c.starts, c.scale)
    assert ((out.double() - o).abs() <= ob)[:3].all()


def test_nothing_to_do():
    c = Case([(40, 0), (0, 0)], seed=11)
    out = torch.full(c.q.shape, 777.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    torch.cuda.synchronize()
    assert (out == 777.0).all()


def test_single_tokens_agree_with_verification_attention():
    """One token a sequence is sv_tree_attention_paged with one node: both within their bounds."""
    c = Case([(700, 1), (64, 1), (3, 1)], hq=32, hkv=8, seed=12)
    out, _ = c.check()
    k, v = torch.nan_to_num(c.k), torch.nan_to_num(c.v)
    tree = sv.sv_tree_attention_paged(c.q[:3].unsqueeze(1).contiguous(), k, v, c.table, i32(c.past), scale=c.scale)
    o, _, ob, _ = c.want()
    assert ((tree.squeeze(1).double() - o).abs() <= ob).all()


def test_two_streams_and_captured_graphs():
    """Calls on two streams at once, and two graphs replayed at once, each with its own workspace."""
    cases = [Case([(2500, 1), (300, 130)], hq=32, hkv=8, seed=13), Case([(1700, 40), (900, 1)], hq=32, hkv=8, seed=14)]
    want = [c.run() for c in cases]
    past, starts = [i32(c.past) for c in cases], [i32(c.starts) for c in cases]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, c in enumerate(cases):
            got[i].append(sv.sv_chunk_attention_paged(c.q, c.k, c.v, c.table, past[i], starts[i], scale=c.scale,
                                                      return_lse=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, e in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(e, want[i][1])
    graphs, outs = [], []
    for i, c in enumerate(cases):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sv.sv_chunk_attention_paged(c.q, c.k, c.v, c.table, past[i], starts[i], scale=c.scale,
                                                    return_lse=True))
        graphs.append(g)
    for _ in range(10):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])


def test_workspace_too_small_or_too_many_heads():
    c = Case([(10, 1)], seed=15)
    with pytest.raises(sv.SpecVerifyError):
        c.run(ws=torch.zeros(4096, dtype=torch.uint8, device="cuda"))
    q = torch.zeros((1, 129, 128), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((4, 1, 16, 128), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(sv.SpecVerifyError):
        sv.sv_chunk_attention_paged(q, k, k.clone(), c.table, i32([0]), i32([0, 1]))


def test_serving_steps_together():
    """Prompts admitted in chunks beside generating sequences, a rejected tail
    taken back after some steps: tables, rows and attention over several steps,
    each against attention over the K/V history kept apart."""
    rng = np.random.default_rng(31)
    gen = torch.Generator(device="cuda").manual_seed(31)
    B, hq, hkv, d, ps, mp = 5, 8, 2, 128, 16, 24
    num_pages = 64
    k = torch.full((num_pages, hkv, ps, d), NAN, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    stack, free = i32(rng.permutation(num_pages)), i32([num_pages])
    counts, past = i32([0] * B), np.zeros(B, np.int64)
    hist = [[torch.zeros((0, hkv, d), dtype=torch.bfloat16, device="cuda")] * 2 for _ in range(B)]
    for step in range(8):
        new = rng.choice([0, 1, 1, 9, 70], B)
        rows = int(new.sum()) + 2
        qkv = torch.randn((rows, hq + 2 * hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
        q, kn, vn = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st = torch.empty(B, dtype=torch.int32, device="cuda")
        starts, slots, counts, free = sv.sv_build_block_tables(i32(past), i32(new), counts, table, stack, free, ps,
                                                               rows, seq_status=st)
        assert (st == 0).all()
        sv.sv_append_kv_paged(kn, vn, slots, k, v)
        out = sv.sv_chunk_attention_paged(q, k, v, table, i32(past), starts, seq_status=st)
        torch.cuda.synchronize()
        assert (st == 0).all()
        begin = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            r = slice(int(begin[b]), int(begin[b + 1]))
            hist[b] = [torch.cat([h, x[r]]) for h, x in zip(hist[b], (kn, vn))]
        # the history as a cache of one page a sequence
        longest = max(len(h[0]) for h in hist)
        flat = [torch.stack([torch.nn.functional.pad(h[i], (0, 0, 0, 0, 0, longest - len(h[i]))) for h in hist])
                .transpose(1, 2) for i in (0, 1)]
        o, _, ob, _ = chunk_ref.attention(q, flat[0], flat[1], torch.arange(B, device="cuda")[:, None], list(past),
                                          list(new), begin, d ** -0.5)
        have = ~torch.isnan(o)
        assert ((out.double() - o).abs()[have] <= ob[have]).all()
        past = past + new
        back = np.minimum(rng.choice([0, 0, 5], B), past)  # a tail rejected
        past = past - back
        hist = [[h[:n] for h in hb] for hb, n in zip(hist, past)]
        counts, free = sv.sv_release_pages(i32(past), counts, table, stack, free, ps, seq_status=st)
        assert (st == 0).all()
    assert po.pages(past, ps).tolist() == counts.tolist()


@pytest.mark.parametrize("window", [0, 1, 92, 127, 128, 300])
def test_few_items_of_unlike_lengths(window):
    """Items enough for a CTA each, some of them across a tile's end in the middle of a sequence."""
    Case([(0, 1), (5458, 1), (1690, 1), (128, 2), (129, 484)], hq=64, hkv=1, page_size=64, window=window, seed=30).check()
    Case([(400, 300), (700, 170), (0, 90), (20, 3)], hq=12, hkv=4, window=window, seed=31).check()
    Case([(30, 250)] + [(9, 0)] * 40 + [(5, 33), (100, 260)], hq=8, hkv=2, d=64, window=window, seed=32).check()
