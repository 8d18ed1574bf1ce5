"""Attention of packed chunks over a paged cache from its definition, in 64
bits, with the bounds that the kernel's roundings allow.

Bounds, for one output element o = sum_j w_j v_j (w: softmax weights, n slots
seen), A = sum_j w_j |v_j| and Q = max_j scale * sum_d |q_d k_jd|:
  - the bf16 output: at most half a step, 2^-8 |o|;
  - P in bf16: each w_j off by at most 2^-8 of itself, 2^-8 A in all;
  - scores: 128 products summed in f32, each addition off by at most 2^-23
    (a truncating adder), so at most Q 2^-16 absolute, as much relative error
    of the weights, in the numerator and in the sum: 2 Q 2^-16 A;
  - the exponential (2^-22) and the scaled difference to the maximum: below
    2^-20 (1 + Q) A;
  - sums over n slots in f32, numerator and row sum: 2 n 2^-23 A.
  For the log-sum-exp: Q 2^-16 + 2^-20 (1 + Q) + n 2^-23, and 2^-22 |lse|
  for its own roundings.
"""
import torch


def gather(pages, table_row, slots):
    """[Hkv, slots, D] float64 of logical slots."""
    ps = pages.shape[2]
    s = torch.as_tensor(slots, device=pages.device)
    pg = table_row.long()[s // ps]
    return pages[pg, :, s % ps].double().transpose(0, 1)


def attention(q, k_pages, v_pages, table, past, new, starts, scale, window=0, chunk=256):
    """Returns (out, lse, out bound, lse bound) in float64, NaN rows where no sequence has them."""
    rows, hq, d = q.shape
    hkv = k_pages.shape[1]
    g = hq // hkv
    out = torch.full((rows, hq, d), float("nan"), dtype=torch.float64, device=q.device)
    lse = torch.full((rows, hq), float("nan"), dtype=torch.float64, device=q.device)
    ob, lb = out.clone(), lse.clone()
    for b, (L, n) in enumerate(zip(past, new)):
        for i in range(0, n, chunk):
            m = min(chunk, n - i)
            r = starts[b] + i
            lo = max(0, L + i - window + 1) if window else 0
            slot = torch.arange(lo, L + i + m, device=q.device)
            k, v = (gather(x, table[b], slot).repeat_interleave(g, 0) for x in (k_pages, v_pages))
            qq = q[r:r + m].double().transpose(0, 1)             # [hq, m, d]
            x = scale * qq @ k.transpose(1, 2)
            p = L + i + torch.arange(m, device=q.device)[:, None]
            sees = slot <= p
            if window:
                sees &= slot > p - window
            z = x.masked_fill(~sees, -float("inf"))
            e = torch.logsumexp(z, -1)
            w = torch.exp(z - e[..., None])
            o = w @ v
            a = w @ v.abs()
            qk = (scale * qq.abs() @ k.abs().transpose(1, 2)).masked_fill(~sees, 0).amax(-1)
            nn = float(len(slot))
            rel = 2.0 ** -8 + 2 * qk * 2.0 ** -16 + 2.0 ** -20 * (1 + qk) + 2 * nn * 2.0 ** -23
            out[r:r + m], lse[r:r + m] = o.transpose(0, 1), e.T
            ob[r:r + m] = (o.abs() * 2.0 ** -8 + a * rel[..., None] * (1 + 2.0 ** -8)).transpose(0, 1)
            lb[r:r + m] = (qk * 2.0 ** -16 + 2.0 ** -20 * (1 + qk) + nn * 2.0 ** -23 + 2.0 ** -22 * e.abs()).T
    return out, lse, ob, lb
