"""The cache held in 4 bits and the attention over it from their definitions,
in 64 bits, with the bounds that the kernels' roundings allow.

Bounds, beside those of chunk_ref.py (P in 16 bits among them), for one output
element with weights w_j, A = sum_j w_j |v_j|, S = sum_j w_j 8 step_j and
Q = max_j scale * sum_d |q_d k_jd|: values of K and V rounded to bf16 would each be
off by at most 2^-8 of themselves, scores by at most 2^-8 Q, the weights by as much
relative, in the numerator and in the sum, 2 Q 2^-8 A (and its square, for exp), and V
2^-8 A; w_j step_j in 16 bits before it meets codes - 8, of 8 at most, 2^-8 S; scores
from sums of codes that a larger part is taken off again, whose f32 sums are off by at
most Q' 2^-16, Q' = scale * sum_d |q_d| (143 step + |minimum|).  The kernels stay
below: K's codes are exact, P and V (or P and its step) in f16, off by 2^-11.
"""
import numpy as np
import torch

ORDER = (0, 2, 4, 6, 1, 3, 5, 7)


def codes_of(packed):
    """[..., D / 2] bytes -> [..., D] codes."""
    out = torch.empty((*packed.shape[:-1], packed.shape[-1] * 2), dtype=torch.uint8, device=packed.device)
    for i, dim in enumerate(ORDER):
        out[..., dim::8] = (packed[..., i // 2::4] >> (4 * (i % 2))) & 15
    return out


def packed(codes):
    out = torch.zeros((*codes.shape[:-1], codes.shape[-1] // 2), dtype=torch.uint8, device=codes.device)
    for i, dim in enumerate(ORDER):
        out[..., i // 2::4] |= codes[..., dim::8] << (4 * (i % 2))
    return out


def values(packed_codes, params):
    return params[..., 1:].double() + params[..., :1].double() * codes_of(packed_codes).double()


def encode(rows):
    """Rows [..., D] f32 (numpy) -> (codes [..., D] uint8, step, minimum as f32 values of bf16 numbers)."""
    with np.errstate(all="ignore"):
        lo, hi = rows.min(-1), rows.max(-1)
        step = torch.from_numpy(np.asarray((hi - lo) * np.float32(1 / 15), np.float32)).to(torch.bfloat16).float().numpy()
        base = torch.from_numpy(np.asarray(lo, np.float32)).to(torch.bfloat16).float().numpy()
        bad = ~np.isfinite(rows).all(-1) | ~np.isfinite(step) | ~np.isfinite(base)
        step = np.where(bad | (step < np.float32(2.0 ** -126)), np.float32(0), step)
        base = np.where(bad, np.float32("nan"), base)
        inv = np.float32(1) / step
        c = np.rint(((rows - base[..., None]).astype(np.float32) * inv[..., None]).astype(np.float32))
    c = np.where((step == 0)[..., None], 0, np.clip(c, 0, 15))
    return np.nan_to_num(c).astype(np.uint8), step.astype(np.float32), base.astype(np.float32)


def ancestors(parents):
    n = len(parents)
    a = np.eye(n, dtype=bool)
    for i in range(1, n):
        a[i] |= a[parents[i]]
    return a


def attention(q, k, v, table, past, new, starts, scale, window=0, parents=None, chunk=256):
    """k, v: (packed codes, params).  Returns (out, lse, out bound, lse bound) in
    float64, NaN rows where no sequence has them."""
    rows, hq, d = q.shape
    hkv, ps = k[0].shape[1:3]
    g = hq // hkv
    out = torch.full((rows, hq, d), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((rows, hq), float("nan"), dtype=torch.float64, device=q.device)
    ob, lb = out.clone(), lse.clone()
    e = 2.0 ** -8
    for b, (L, n) in enumerate(zip(past, new)):
        above = torch.tensor(ancestors(parents[b]), device=q.device) if parents is not None else None
        for i in range(0, n, chunk):
            m = min(chunk, n - i)
            r = starts[b] + i
            lo = max(0, L + i - window + 1) if window else 0
            slot = torch.arange(lo, L + i + m, device=q.device)
            pg = table[b].long()[slot // ps]
            kk, vv, size, mag = [], [], [], []
            for codes, params in (k, v):
                c, p = codes[pg, :, slot % ps].transpose(0, 1), params[pg, :, slot % ps].transpose(0, 1)
                (kk if not kk else vv).append(values(c, p).repeat_interleave(g, 0))
                size.append(p[..., 0].double().repeat_interleave(g, 0))
                mag.append((143 * p[..., 0].double() + p[..., 1].double().abs()).repeat_interleave(g, 0))
            kk, vv = kk[0], vv[0]
            qq = q[r:r + m].double().transpose(0, 1)
            x = scale * qq @ kk.transpose(1, 2)
            p = L + i + torch.arange(m, device=q.device)[:, None]
            sees = slot <= p
            if window:
                sees &= slot > p - window
            if above is not None:
                sees = torch.cat([sees[:, :L], above[i:i + m, :i + m]], 1)
            z = x.masked_fill(~sees, -float("inf"))
            s = torch.logsumexp(z, -1)
            w = torch.exp(z - s[..., None])
            o = w @ vv
            a = w @ vv.abs()
            st = 8 * (w @ size[1][..., None])
            qk = (scale * qq.abs() @ kk.abs().transpose(1, 2)).masked_fill(~sees, 0).amax(-1)
            qf = (scale * qq.abs().sum(-1)[..., None] * mag[0][:, None]).masked_fill(~sees, 0).amax(-1)
            nn = float(len(slot))
            score = torch.maximum(e * qk, 2.0 ** -16 * qf) + 2.0 ** -16 * qk
            rel = e + torch.expm1(2 * score) + 2.0 ** -20 * (1 + qk) + 2 * nn * 2.0 ** -23
            out[r:r + m], lse[r:r + m] = o.transpose(0, 1), s.T
            ob[r:r + m] = (o.abs() * e + (a * (rel[..., None] + e) + st * e) * (1 + e)).transpose(0, 1)
            lb[r:r + m] = (score + 2.0 ** -20 * (1 + qk) + nn * 2.0 ** -23 + 2.0 ** -22 * s.abs()).T
    return out, lse, ob, lb
