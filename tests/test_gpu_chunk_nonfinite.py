"""A query row that is not finite shows as such in its own output and
log-sum-exp, however the work is cut, and in no other row.

With q = NaN every score of the row is NaN: out and lse are NaN.  With an
infinite element a score is infinite or NaN: a weight exp(x - max) is then NaN
(inf - inf) or, where every score is -inf, the weights are 0 / 0: out is NaN
either way, and lse is not finite."""
import pytest
import torch

from test_gpu_chunk import Case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
EMPTY = [(0, 0)] * 33  # more sequences than the form for few rows takes

# lens, shape, rows that stop being finite
FORMS = {
    "few rows": ([(300, 2), (40, 3), (0, 1)], dict(hq=8, hkv=2), (0, 3, 5)),
    "few rows, many CTAs": ([(9000, 1)], dict(hq=6, hkv=2, d=64), (0,)),
    "whole items": ([(5, 1)] * 40 + [(0, 1)], dict(hq=8, hkv=2), (0, 7, 40)),
    "cut items of few rows": ([(20000, 1)] + EMPTY, dict(hq=32, hkv=8, page_size=64), (0,)),
    "cut items of many rows": ([(9000, 70)], dict(hq=8, hkv=1), (0, 31, 64, 69)),
    "cut items of two tiles": ([(6000, 150)], dict(hq=4, hkv=2, d=64), (0, 63, 64, 149)),
}


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("value,whole", [(NAN, False), (NAN, True), (INF, False), (-INF, False), (INF, True)])
def test_a_query_row_that_is_not_finite(form, window, value, whole):
    lens, kw, rows = FORMS[form]
    c = Case(lens, window=window, seed=40, **kw)
    out, lse = c.run()
    q = c.q.clone()
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    for i, r in enumerate(rows):
        h = (3 * i + 1) % lse.shape[1]  # one head of the row, its neighbours stay
        q[r, h, slice(None) if whole else 5] = value
        hit[r, h] = True
    c.q = q
    got, ge = c.run()
    torch.cuda.synchronize()
    assert torch.isnan(got[hit]).all()
    assert not torch.isfinite(ge[hit]).any()
    if value != value:
        assert torch.isnan(ge[hit]).all()
    assert torch.equal(got[~hit], out[~hit]) and torch.equal(ge[~hit], lse[~hit])
