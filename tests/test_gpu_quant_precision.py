"""The attention over pages held in 4 bits at the precision that it states, against
64 bits.

What an output may be off by, as shares of its norm (rows of D independent values):
    its own rounding to bf16   2^-7 / sqrt(12) at most in the mean square (2.26e-3; a step is
                               2^-7 of the lowest value that has it)
    P, V and V's middle in f16 2^-11 / sqrt(3) each at most, 2.8e-4
so 2.31e-3 together, and LIMIT = 2.5e-3 with 2^-24 to spare for the sums.  P is a whole
2^-24 below 2^-14, where the largest P is 2^7 or more: a slot of weight w beside one of
weight 1 has P = 2^7 w or more, off by 2^-25 / (2^7 w) of itself, below 2^-11 down to
w = 2^-21.  The norm of one row and head has fewer values, D = 64 at the least: the mean of
64 squares of a uniform error is off by 0.11 of itself, five times which is 1.25 in the norm.

A log-sum-exp of size x is off by some ten roundings of f32 of sizes up to x and the
scores', independent of one another: 2^-24 sqrt(10 / 3) (x + 6) in the mean square at most,
below 2^-23 (x + 6)."""
import math

import numpy as np
import pytest
import torch

import quant_ref
import speculative_decoding_verification_81_gb300 as sv  # noqa: F401
from test_gpu_quant import Case

pytestmark = pytest.mark.gpu
LIMIT = 2.5e-3


def shares(out, want):
    """Errors' norms over the rows' norms: of all rows, and the largest of a row and head."""
    have = ~torch.isnan(want[..., 0])
    o, d = want[have], out[have].double() - want[have]
    assert torch.isfinite(d).all()
    return (d.norm() / o.norm()).item(), (d.norm(dim=-1) / o.norm(dim=-1)).max().item()


def stated(c):
    (out, lse), (o, e, _, _) = c.run(), c.want()
    of_all, of_one = shares(out, o)
    assert of_all < LIMIT and of_one < 1.25 * LIMIT, (of_all, of_one)
    have = ~torch.isnan(e)
    d, size = (lse.double() - e)[have], e[have].square().mean().sqrt().item()
    rms = d.square().mean().sqrt().item()
    assert rms < 2.0 ** -23 * (size + 6), (rms, size)


EVEN = [
    ([(0, 1)], dict(hq=32, hkv=8)),
    ([(2047, 1), (4095, 1)], dict(hq=32, hkv=8)),
    ([(20000, 1)], dict(hq=32, hkv=8, page_size=64)),
    ([(900, 2)] * 9, dict(hq=32, hkv=8, d=64)),
    ([(300, 3), (41, 1), (1999, 4)], dict(hq=16, hkv=4, page_size=128)),
    ([(2500, 9)] * 7 + [(33, 9)], dict(hq=32, hkv=8)),
    ([(1500, 26), (127, 26), (0, 26)], dict(hq=8, hkv=2, d=64, tree=3)),
    ([(700, 64), (2000, 60)], dict(hq=32, hkv=8, tree=5)),
    ([(0, 700)], dict(hq=8, hkv=2)),
    ([(6000, 200)], dict(hq=8, hkv=8, page_size=384)),
    ([(3000, 300), (100, 1)], dict(hq=14, hkv=2, d=64, window=640)),
]
# The form for few rows goes by the rows of the mean sequence: it meets long ones among single tokens, cut into
# many items, and the other form single tokens beside long prompts.
UNEVEN = [
    ([(300, 1)] * 60 + [(1000, 130)], dict(hq=32, hkv=8)),
    ([(50, 1)] * 90 + [(700, 200), (0, 100)], dict(hq=8, hkv=8)),
    ([(90, 1)] * 40 + [(300, 40)], dict(hq=14, hkv=2, d=64)),
    ([(200, 1)] * 30 + [(500, 40), (90, 26)], dict(hq=8, hkv=2, tree=3)),
    ([(100, 1)] * 50 + [(500, 64), (0, 64), (77, 50)], dict(hq=4, hkv=2, tree=64, d=64)),
    ([(300, 1)] * 60 + [(1000, 130)], dict(hq=32, hkv=8, window=37)),
    ([(50, 1)] * 90 + [(700, 200), (0, 100)], dict(hq=8, hkv=8, window=129, page_size=128)),
    ([(90, 1)] * 40 + [(300, 40)], dict(hq=14, hkv=2, d=64, window=1)),
    ([(700, 1)] * 20 + [(100, 400)], dict(hq=32, hkv=8)),
    ([(700, 1)] * 20 + [(100, 400)], dict(hq=32, hkv=8, window=200)),
]


@pytest.mark.parametrize("i", range(len(EVEN) + len(UNEVEN)))
def test_as_near_as_stated(i):
    lens, kw = (EVEN + UNEVEN)[i]
    stated(Case(lens, seed=200 + i, spare_rows=i % 3, strided=i % 2 == 0, **kw))


@pytest.mark.parametrize("i", range(len(EVEN) + len(UNEVEN)))
def test_every_row_sees_its_slots_and_no_other(i):
    """With q = 0 the weights are even, and with values of 15/16 at dim s mod D of slot s, 0 elsewhere, an
    output counts the seen slots of its residue: one slot more or less is 1 / 157 of it or more here, and
    nothing is rounded but the output, to bf16 (1 / 256 at most), and the division."""
    lens, kw = (EVEN + UNEVEN)[i]
    c = Case(lens, seed=300 + i, **kw)
    c.q.zero_()
    (codes, params), ps, d = c.v, c.page_size, c.q.shape[2]
    one_hot = quant_ref.packed(15 * torch.eye(d, dtype=torch.uint8, device="cuda"))
    for b, (L, n) in enumerate(lens):
        s = torch.arange(max(0, L - c.window + 1) if c.window else 0, L + n, device="cuda")
        pg = c.table[b, s // ps].long()
        codes[pg, :, s % ps] = one_hot[s % d][:, None]
        params[pg, :, s % ps] = torch.tensor([1 / 16, 0], dtype=torch.bfloat16, device="cuda")
    (out, lse), (o, e, _, _) = c.run(), c.want()
    have = ~torch.isnan(e)
    assert ((out.double() - o).abs() <= o.abs() * 2.0 ** -8 + o.abs() * 2.0 ** -20)[have].all()
    assert ((lse.double() - e).abs() <= 2.0 ** -20 * (1 + e))[have].all()


@pytest.mark.parametrize("seed", range(24))
def test_drawn_shapes(seed):
    """Lengths, head layouts, pages, windows and trees drawn over their ranges; the same bits twice."""
    rng = np.random.default_rng(4000 + seed)
    kind = ("single", "short", "chunks", "mixed", "tree")[seed % 5]
    hkv, d = int(rng.choice([1, 2, 3, 8])), int(rng.choice([64, 128]))
    g = int(rng.choice([1, 2, 3, 4, 7, 8, 12, 16, 17, 32, 100, 128]))
    B = int(rng.integers(1, 40)) if hkv * g < 200 else 3
    past = rng.integers(0, int(rng.choice([3, 40, 300, 1500])) + 1, B)
    new = {"single": np.ones(B, int), "short": rng.integers(0, 9, B), "chunks": rng.integers(1, 200, B),
           "tree": rng.integers(0, 65, B), "mixed": np.where(rng.random(B) < 0.7, 1, rng.integers(0, 300, B))}[kind]
    new[0] = max(new[0], 1)
    c = Case(list(zip(past.tolist(), new.tolist())), hq=hkv * g, hkv=hkv, d=d, page_size=int(rng.choice([8, 16, 32, 64, 128, 256, 384])),
             window=0 if kind == "tree" else int(rng.choice([0, 0, 1, 7, 100, 128, 500])), seed=seed, strided=seed % 3 == 0,
             spare_rows=seed % 4, tree=int(rng.integers(1, 8)) if kind == "tree" else 0)
    stated(c)
    n = int(c.starts[-1])  # (rows behind it are no sequence's)
    a, b = c.run(), c.run()
    assert all(torch.equal(x[:n].view(t), y[:n].view(t)) for x, y, t in zip(a, b, (torch.int16, torch.int32)))


# ---------------------------------------------------------------- a slot that has most of the weight

def dominated(lens, at, weight, zero, seed=0, **kw):
    """In each sequence slot `at` has about this weight, and values of 0 under a step of 0 or of its
    own (codes of 8 each): the outputs are the other slots'."""
    c = Case(lens, seed=seed, **kw)
    ps, hkv, d = c.page_size, c.k[0].shape[1], c.q.shape[2]
    rows, hq, _ = c.q.shape
    c.q.mul_(0.25).add_(1.0)
    for params in (c.k[1], c.v[1]):
        step = params[..., 0].float()
        params[..., 1] = (-7.5 * step).to(torch.bfloat16)
    where = [(c.table[b, at // ps].item(), at % ps) for b in range(len(lens))]
    for pg, s in where:
        for codes, params in (c.k, c.v):
            codes[pg, :, s] = 0x88 if codes is c.v[0] else 0
            params[pg, :, s] = 0
        if zero == "codes":
            c.v[1][pg, :, s, 0], c.v[1][pg, :, s, 1] = 0.25, -2.0
        c.k[1][pg, :, s, 1] = -50.0  # (no weight, for the moment)
    lse = c.want()[1]
    for b, (pg, s) in enumerate(where):
        r = slice(int(c.starts[b]), int(c.starts[b + 1]))
        size = (c.scale * c.q[r].double().sum(-1)).reshape(-1, hkv, hq // hkv)
        level = lse[r].reshape(-1, hkv, hq // hkv) + math.log(weight / (1 - weight))
        c.k[1][pg, :, s, 1] = (level / size).mean((0, 2)).to(torch.bfloat16)
    return c


# (as many heads as keep an item on one CTA, or the most of it: a cut item's parts have a maximum each)
@pytest.mark.parametrize("zero", ["step", "codes"])
@pytest.mark.parametrize("lens,at,kw", [
    ([(16384, 40)], 0, dict(hq=64, hkv=64)),
    ([(16384, 130)], 0, dict(hq=64, hkv=64)),
    ([(16384, 130)], 9000, dict(hq=64, hkv=64, page_size=128)),
    ([(12000, 70), (9000, 33)], 3, dict(hq=160, hkv=40, d=64, page_size=64)),
    ([(16384, 1)], 0, dict(hq=32, hkv=8)),
    ([(16384, 1)] * 4, 0, dict(hq=128, hkv=128)),
    ([(16384, 1)] * 4, 9000, dict(hq=128, hkv=128, d=64)),
    ([(12000, 4), (16000, 3)], 1, dict(hq=240, hkv=60, page_size=128)),
])
def test_one_slot_has_most_of_the_weight(lens, at, kw, zero):
    c = dominated(lens, at, 0.99, zero, seed=len(lens) + at, **kw)
    of_all, _ = shares(c.run()[0], c.want()[0])
    assert of_all < LIMIT, of_all


# ---------------------------------------------------------------- scores at the ends of f32

@pytest.mark.parametrize("lens,kw", [([(0, 1)], {}), ([(40, 1)], dict(d=64)), ([(300, 2)], dict(hq=8, hkv=4)),
                                     ([(100, 30)], {})])
@pytest.mark.parametrize("size", [-1.5, -0.875, 0.875, 1.5])
def test_scores_near_the_ends_of_the_range(lens, kw, size):
    """Scores past 2^126 in log2 units: in f32 they are whole multiples of 2^103, and the weights have no
    bound, since exp of an error of that size has none.  What holds for any weights: an output is among
    the values that its row sees, but for the roundings to f16 and bf16 (2^-11 twice and 2^-8 of the
    largest of them), and the log-sum-exp is the score."""
    c = Case(lens, seed=31, scale=1.0, **kw)
    (_, hq, d), ps, hkv, n = c.q.shape, c.page_size, c.k[0].shape[1], sum(lens[0])
    c.q.fill_(size * 2.0 ** 60)
    c.k[0].zero_()
    c.k[1][..., 0], c.k[1][..., 1] = 0.0, 2.0 ** 66 / d
    out, lse = c.run()
    s = torch.arange(n, device="cuda")
    pg = c.table[0, s // ps].long()
    v = quant_ref.values(c.v[0][pg, :, s % ps], c.v[1][pg, :, s % ps]).repeat_interleave(hq // hkv, 1)
    room = v.abs().amax(0) * 2.0 ** -7
    assert (out.double() >= v.amin(0) - room).all() and (out.double() <= v.amax(0) + room).all()
    score = size * 2.0 ** 126
    assert ((lse.double() - score).abs() < abs(score) * 2.0 ** -21).all()
