"""The cache held in 4 bits on the GPU: rows quantised into the pages (equal to
the format's definition, bit for bit), attention over them in 64 bits (bounds in
quant_ref.py), accepted paths moved, the refusals, and a run of them together."""
import numpy as np
import pytest
import torch

import quant_ref
import speculative_decoding_verification_81_gb300 as sv

pytestmark = pytest.mark.gpu
NAN = float("nan")


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def tree_of(n, rng, width):
    par = np.array([-1] + [max(0, int(rng.integers(max(0, i - width), i))) for i in range(1, n)])
    return par


class Case:
    """A pool with the sequences' pages anywhere in it; slots that no row sees
    hold NaN, and table entries of pages without a seen slot name no page."""

    def __init__(self, lens, hq=8, hkv=2, d=128, page_size=16, window=0, seed=0, scale=None, strided=False,
                 spare_rows=0, tree=0, offset=0.0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.past, self.new = [l[0] for l in lens], [l[1] for l in lens]
        self.window, self.page_size = window, page_size
        self.scale = d ** -0.5 if scale is None else scale
        need = [-(-(a + n) // page_size) for a, n in lens]
        num_pages = sum(need) + 3
        ids = rng.permutation(num_pages)
        table = np.full((len(lens), max(need) + 2), 10 ** 6, np.int64)
        table[:, 1::2] = -1
        self.k, self.v = [], []
        for c in (self.k, self.v):
            c.append(torch.randint(0, 256, (num_pages, hkv, page_size, d // 2), generator=gen, device="cuda", dtype=torch.uint8))
            c.append(torch.full((num_pages, hkv, page_size, 2), NAN, dtype=torch.bfloat16, device="cuda"))
        used = 0
        for b, (a, n) in enumerate(lens):
            lo = max(0, a - window + 1) if window else 0
            for j in range(lo // page_size if n else need[b], need[b]):
                table[b, j] = ids[used + j]
            used += need[b]
            if n:
                s = torch.arange(lo, a + n, device="cuda")
                pg = i32(table[b])[s // page_size].long()
                for c in (self.k, self.v):
                    step = torch.rand((a + n - lo, hkv), generator=gen, device="cuda") * 0.3 + 0.02
                    low = -7.5 * step + torch.randn(step.shape, generator=gen, device="cuda") * 0.5 + offset
                    c[1][pg, :, s % page_size] = torch.stack([step, low], -1).to(torch.bfloat16)
        self.table = i32(table)
        self.starts = np.concatenate([[0], np.cumsum(self.new)])
        rows = int(self.starts[-1]) + spare_rows
        q = torch.randn((max(rows, 1), hq + (2 * hkv if strided else 0), d), generator=gen, device="cuda").to(torch.bfloat16)
        self.q = q[:, :hq]
        self.trees = [tree_of(n, rng, tree) if n else np.zeros(0, np.int64) for n in self.new] if tree else None
        self.parents = None
        if tree:
            flat = np.concatenate([*self.trees, np.full(max(rows, 1) - int(self.starts[-1]), 7)])
            self.parents = i32(flat)

    def run(self, **kw):
        return sv.sv_chunk_attention_quant(self.q, *self.k, *self.v, self.table, i32(self.past), i32(self.starts),
                                           parents=self.parents, scale=self.scale, window=self.window, return_lse=True, **kw)

    def want(self):
        return quant_ref.attention(self.q, self.k, self.v, self.table, self.past, self.new, self.starts, self.scale,
                                   self.window, self.trees)

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
    # roundings are independent of one another: their sum over a row is far below its bound (bf16 output,
    # weights, K, V: four of at most 2^-8, a sixth of that and less in the mean square)
    norm = (out.double() - o)[have].norm() / o[have].norm()
    assert norm < 2.0 ** -8 * 2, norm


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
    ([(2500, 9)] * 7 + [(33, 9)], dict(hq=32, hkv=8)),                   # chains
]


@pytest.mark.parametrize("i", range(len(SMALL)))
def test_chunks(i):
    lens, kw = SMALL[i]
    Case(lens, seed=i, spare_rows=i % 3, strided=i % 2 == 1, **kw).check()


@pytest.mark.parametrize("window", [1, 2, 17, 128, 129, 640])
@pytest.mark.parametrize("lens,kw", [
    ([(0, 300), (1000, 1), (3, 1), (700, 64)], dict(hq=8, hkv=2, page_size=16)),
    ([(2000, 140), (255, 3)], dict(hq=6, hkv=6, d=64, page_size=128)),
    ([(1000, 1), (77, 1)], dict(hq=8, hkv=2, page_size=8)),
])
def test_windows(window, lens, kw):
    Case(lens, window=window, seed=window, **kw).check()


@pytest.mark.parametrize("lens,kw", [
    ([(300, 26), (0, 26), (127, 1), (65, 0), (1000, 26)], dict(hq=32, hkv=8)),
    ([(300, 64), (2000, 64), (100, 63)], dict(hq=32, hkv=8, page_size=64)),   # two Q tiles
    ([(90, 64), (40, 33)], dict(hq=16, hkv=2, page_size=32, d=64)),           # four items of 32 nodes' Q tiles
    ([(90, 5), (40, 3)], dict(hq=128, hkv=1)),                                # a token a Q tile
    ([(500, 3)], dict(hq=8, hkv=2)),                                          # few rows
    ([(3, 2), (0, 4)], dict(hq=4, hkv=2, d=64, page_size=8)),
    ([(120, 20)], dict(hq=8, hkv=8)),                                         # across a K/V tile's end
])
@pytest.mark.parametrize("width", [1, 3, 64])
def test_trees(lens, kw, width):
    Case(lens, seed=len(lens) * 100 + width, tree=width, spare_rows=2, **kw).check()


@pytest.mark.parametrize("n,past_hi,kw", [
    (300, 200, dict(hq=32, hkv=8)),        # more sequences than CTAs, each a tile or two
    (1500, 5, dict(hq=2, hkv=1, d=64)),    # more sequences than threads of a CTA
    (33, 3000, dict(hq=8, hkv=8, page_size=128)),
])
def test_many_single_tokens(n, past_hi, kw):
    rng = np.random.default_rng(n)
    Case([(int(x), 1) for x in rng.integers(0, past_hi, n)], seed=n, **kw).check()


def test_values_far_from_zero():
    """Minima far larger than the steps: what is added to a score is taken off again nowhere."""
    Case([(400, 1)], hq=8, hkv=2, offset=20.0, scale=0.01, seed=3).check()
    Case([(400, 40)], hq=8, hkv=2, offset=20.0, scale=0.01, seed=4).check()


def test_bad_sequences_are_reported_and_touch_no_other():
    c = Case([(50, 3), (20, 4), (30, 2), (9, 1), (300, 5)], tree=2, seed=9)
    want = c.want()
    past, starts, table, par = np.array(c.past), c.starts.copy(), c.table.clone(), c.parents.clone()
    past[0] = -1                       # skipped: its rows stay
    table[1, 1] = -5                   # a page that is none
    par[int(starts[2]) + 1] = 1        # a parent not before its node
    st = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    out = torch.full(c.q.shape, 777.0, dtype=torch.bfloat16, device="cuda")
    sv.sv_chunk_attention_quant(c.q, *c.k, *c.v, table, i32(past), i32(starts), parents=par, out=out, seq_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [6, 6, 6, 0, 0]
    assert (out[:3] == 777.0).all()
    ok = slice(int(starts[3]), int(starts[5]))
    assert ((out.double() - want[0]).abs()[ok] <= want[2][ok]).all()
    c = Case([(50, 65), (20, 4)], tree=2, seed=10)  # more nodes than a tree may have
    c.run(seq_status=st[:2])
    assert st[:2].tolist() == [6, 0]


# ---------------------------------------------------------------- rows

def rows_like(rng, n, hkv, d, kind):
    x = rng.standard_normal((n, hkv, d)).astype(np.float32)
    if kind == "odd":
        x[0] = 0                                   # no range
        x[1 % n, 0] = 3.25
        x[2 % n] *= np.float32(1e-38)              # steps below 2^-126
        x[3 % n] *= np.float32(1e-35)
        x[4 % n, 0, 5] = np.inf
        x[5 % n, -1, 1] = np.nan
        x[6 % n] = np.where(rng.random((hkv, d)) < 0.5, np.float32(3.3e38), np.float32(-3.3e38))  # hi - lo overflows
        x[7 % n] = x[7 % n] * np.float32(1e-3) + 100   # a minimum that bf16 rounds
        x[8 % n] = np.round(x[8 % n] * 4) / 4          # ties
    return x


@pytest.mark.parametrize("n,hkv,d,page_size,wide,strided,kind", [
    (1, 1, 64, 8, False, False, "plain"),
    (37, 8, 128, 16, True, False, "odd"),
    (37, 8, 128, 16, False, True, "odd"),
    (600, 2, 64, 32, True, True, "odd"),
    (1000, 5, 128, 128, False, True, "plain"),
    (13, 3, 64, 384, True, False, "odd"),
])
def test_append(n, hkv, d, page_size, wide, strided, kind):
    rng = np.random.default_rng(n)
    pages = -(-n // page_size) + 3
    slots = rng.permutation(pages * page_size)[:n]
    slots[n // 2::5] = -1
    want_st = np.zeros(n, int)
    if n > 20:
        slots[[3, 11]] = [-2, pages * page_size]
        want_st[[3, 11]] = 6
    x = [torch.from_numpy(rows_like(rng, n, 3 * hkv if strided else hkv, d, kind)) for _ in range(1 if strided else 2)]
    x = [t.to(torch.float32 if wide else torch.bfloat16) for t in x]
    dev = [t.cuda() for t in x]
    kn, vn = (dev[0][:, hkv:2 * hkv], dev[0][:, 2 * hkv:]) if strided else dev
    caches, before = [], []
    for _ in range(2):
        c = [torch.randint(0, 256, (pages, hkv, page_size, d // 2), dtype=torch.uint8, device="cuda"),
             torch.randn((pages, hkv, page_size, 2), device="cuda").to(torch.bfloat16)]
        caches.append(c)
        before.append([t.clone() for t in c])
    st = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    sv.sv_append_kv_quant(kn, vn, i32(slots), *caches[0], *caches[1], row_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == want_st.tolist()
    on = [i for i, s in enumerate(slots) if 0 <= s < pages * page_size]
    s = torch.tensor(slots[on])
    for new, got, old in zip((kn, vn), caches, before):
        codes, step, base = quant_ref.encode(new.float().cpu().numpy()[on])
        want = [old[0].cpu(), old[1].cpu().float()]
        want[0][s // page_size, :, s % page_size] = quant_ref.packed(torch.from_numpy(codes))
        want[1][s // page_size, :, s % page_size] = torch.stack([torch.from_numpy(step), torch.from_numpy(base)], -1)
        assert torch.equal(got[0].cpu(), want[0])
        np.testing.assert_array_equal(got[1].cpu().float().numpy(), want[1].numpy())


def test_values_are_within_half_a_step():
    rng = np.random.default_rng(2)
    x = torch.from_numpy(rng.standard_normal((256, 2, 128)).astype(np.float32)).cuda()
    k = [torch.zeros((16, 2, 16, 64), dtype=torch.uint8, device="cuda"), torch.zeros((16, 2, 16, 2), dtype=torch.bfloat16, device="cuda")]
    v = [t.clone() for t in k]
    sv.sv_append_kv_quant(x, x, i32(np.arange(256)), *k, *v)
    got = quant_ref.values(*k).transpose(1, 2).reshape(256, 2, 128)
    step = (x.amax(-1) - x.amin(-1)).double() / 15
    # half a step of a step rounded by at most 2^-8 of itself, 15 of which may end short of the highest
    # value, and the minimum's rounding
    bound = step * (0.5 * (1 + 2.0 ** -8) + 15 * 2.0 ** -8) + x.amin(-1).abs().double() * 2.0 ** -8
    assert ((got - x.double()).abs().amax(-1) <= bound).all()
    assert torch.equal(k[0], v[0]) and torch.equal(k[1], v[1])


# ---------------------------------------------------------------- accepted paths

@pytest.mark.parametrize("hkv,d,page_size", [(8, 128, 16), (1, 64, 8), (3, 64, 384), (40, 128, 32)])
def test_compact(hkv, d, page_size):
    rng = np.random.default_rng(hkv)
    B, P = 9, 30
    prefix = rng.integers(0, 200, B)
    mp = -(-(200 + P) // page_size) + 1
    pages = B * mp + 2
    table = rng.permutation(pages)[:B * mp].reshape(B, mp)
    acc = rng.integers(0, 12, B)
    path = np.full((B, P), -1)
    for b in range(B):
        path[b, :acc[b] + 1] = np.concatenate([[0], np.sort(rng.permutation(np.arange(1, P))[:acc[b]])])
    acc[1], acc[2] = -1, 3
    path[2, :4] = [0, -40, -30, 5]     # not increasing from 0
    table[3, prefix[3] // page_size] = 10 ** 6 if acc[3] > 0 else table[3, prefix[3] // page_size]
    acc[4] = 29
    path[4] = np.arange(30)            # nothing moves
    cache = [torch.randint(0, 256, (pages, hkv, page_size, d // 2), dtype=torch.uint8, device="cuda"),
             torch.randn((pages, hkv, page_size, 2), device="cuda").to(torch.bfloat16)]
    cache += [torch.randint(0, 256, (pages, hkv, page_size, d // 2), dtype=torch.uint8, device="cuda"),
              torch.randn((pages, hkv, page_size, 2), device="cuda").to(torch.bfloat16)]
    want = [t.clone().cpu() for t in cache]
    lens, status = [], []
    for b in range(B):
        ids = [table[b, s // page_size] for s in range(prefix[b], prefix[b] + acc[b] + 1)]
        ids += [table[b, (prefix[b] + max(0, path[b, d])) // page_size] for d in range(acc[b] + 1)]
        ok = b != 2 and all(0 <= x < pages for x in ids)
        if acc[b] >= 0 and ok:
            for t in want:
                old = t.clone()
                for i in range(1, acc[b] + 1):
                    x, y = prefix[b] + path[b, i], prefix[b] + i
                    t[table[b, y // page_size], :, y % page_size] = old[table[b, x // page_size], :, x % page_size]
        lens.append(prefix[b] + acc[b] + 1 if acc[b] >= 0 and ok else prefix[b])
        status.append(0 if ok else 6)
    st = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    got = sv.sv_compact_kv_quant(*cache, i32(table), i32(prefix), i32(acc), i32(path), seq_status=st)
    torch.cuda.synchronize()
    assert got.tolist() == lens and st.tolist() == status
    for a, w in zip(cache, want):
        assert torch.equal(a.cpu().view(torch.uint8), w.view(torch.uint8))
    assert sv.sv_compact_kv_quant(*cache, i32(table), i32(prefix), i32([2] * B)).tolist() == [
        p + 3 if p + 3 <= mp * page_size else p for p in prefix]  # a chain: nothing moves
