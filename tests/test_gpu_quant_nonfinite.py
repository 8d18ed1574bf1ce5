"""Rows of a cache held in 4 bits that read as NaN (sv_append_kv_quant makes them of rows
with a value that is not finite): every row of queries that sees one is NaN, and no other
row is touched, whatever shares a tile or an item with it."""
import numpy as np
import pytest
import torch

import quant_ref
import speculative_decoding_verification_81_gb300 as sv
from test_gpu_quant import Case, i32

pytestmark = pytest.mark.gpu
NAN = float("nan")

CASES = {
    "chains": ([(900, 4), (30, 3), (127, 4)], dict(hq=32, hkv=8)),
    "long chains": ([(900, 12), (121, 14)], dict(hq=8, hkv=8, d=64)),
    "trees, few rows": ([(200, 4), (125, 4)], dict(hq=8, hkv=2, tree=4)),
    "trees": ([(300, 26), (0, 26), (120, 26)], dict(hq=32, hkv=8, tree=3)),
    "trees of two tiles": ([(300, 64), (100, 50)], dict(hq=32, hkv=8, tree=64, d=64)),
    "a prompt": ([(100, 300)], dict(hq=8, hkv=2)),
    "a window": ([(100, 300), (900, 1)], dict(hq=8, hkv=2, window=50)),
    "few rows in a window": ([(300, 8), (900, 1)], dict(hq=8, hkv=4, window=5)),
    "a prompt beside single tokens": ([(50, 1)] * 60 + [(100, 123)], dict(hq=32, hkv=8)),
}


def sees(c, b):
    """[rows, slots] of sequence b."""
    L, n = c.past[b], c.new[b]
    pos, slot = L + np.arange(n)[:, None], np.arange(L + n)
    m = slot <= pos
    if c.window:
        m &= slot > pos - c.window
    if c.trees is not None:
        m[:, L:] = quant_ref.ancestors(c.trees[b])
    return m


@pytest.mark.parametrize("which", ["K", "V", "both"])
@pytest.mark.parametrize("name", CASES)
def test_it_reaches_the_rows_that_see_it_alone(name, which):
    lens, kw = CASES[name]
    c = Case(lens, seed=21, **kw)
    out, e, ob, eb = c.want()
    rng = np.random.default_rng(22)
    hkv, ps = c.k[0].shape[1:3]
    rows, hq, _ = c.q.shape
    hit = torch.zeros((rows, hq), dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.new):
        for i in sorted({n - 1, n // 2, n // 3}):
            s, h = c.past[b] + i, int(rng.integers(hkv))
            kn, vn = (torch.randn((1, hkv, c.q.shape[2]), device="cuda") for _ in range(2))
            if which != "V":
                kn[0, h, 3] = NAN
            if which != "K":
                vn[0, h, 7] = float("inf")
            old = [t[c.table[b, s // ps].item(), :, s % ps].clone() for t in (*c.k, *c.v)]
            sv.sv_append_kv_quant(kn, vn, i32([c.table[b, s // ps].item() * ps + s % ps]), *c.k, *c.v)
            for t, o, mine in zip((*c.k, *c.v), old, (which != "V",) * 2 + (which != "K",) * 2):
                keep = torch.ones(hkv, dtype=torch.bool, device="cuda")
                keep[h] = not mine
                t[c.table[b, s // ps].item(), keep, s % ps] = o[keep]
            r = int(c.starts[b]) + np.flatnonzero(sees(c, b)[:, s])
            hit[r, h * (hq // hkv):(h + 1) * (hq // hkv)] = True
    got, lse = c.run()
    assert torch.isnan(got[hit]).all()
    if which != "V":
        assert not torch.isfinite(lse[hit]).any()
    assert 0 < hit.sum() < hit.numel()
    assert ((got.double() - out).abs() <= ob)[~hit].all() and ((lse.double() - e).abs() <= eb)[~hit].all()
