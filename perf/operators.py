"""The paged-cache operators that surround a verification step, as they are measured: page tables and slot maps
from request lengths, pages given back, new K/V rows written to the cache, and the attention of chunks of new
tokens over it.  `run` computes them in plain torch operations, or through the library where `own` is true."""
import math

import numpy as np
import torch

own = False

#: The serving shape of the repository's bench: 32 query heads over 8 KV heads of dimension 128.
_HEADS = {"hq": 32, "hkv": 8, "d": 128}


# ---------------------------------------------------------------- the cases

def _attention(name, *, singles=0, single_lo=1, single_hi=1, chunks=0, new_lo=1, new_hi=1, past_lo=0, past_hi=0,
               page=16, window=0, lse=False, strided=False, lens=0, **heads):
    return {"name": name, "op": "attention", "singles": singles, "single_lo": single_lo, "single_hi": single_hi,
            "chunks": chunks, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo, "past_hi": past_hi,
            "page": page, "window": window, "lse": lse, "strided": strided, "lens": lens, **{**_HEADS, **heads}}


def _tables(name, op, batch, new_hi, past_hi, page, tight=False, lens=0):
    return {"name": name, "op": op, "batch": batch, "new_hi": new_hi, "past_hi": past_hi, "page": page,
            "tight": tight, "lens": lens}


def _append(name, rows, page, wide, strided=False, lens=0, hkv=8, d=128):
    return {"name": name, "op": "append", "rows": rows, "page": page, "wide": wide, "strided": strided, "lens": lens,
            "hkv": hkv, "d": d}


def listed():
    return [
        # one request generating alone: the smallest call, where the launch is what it costs
        _attention("one token, 511 before it", singles=1, single_lo=511, single_hi=511),
        # a decoding batch of the bench's size and lengths: bound by the cache's bytes
        _attention("32 tokens, each after 2048 to 4096", singles=32, single_lo=2048, single_hi=4096, lse=True, lens=1),
        # continuous batching: prompt chunks admitted beside requests that generate
        _attention("48 tokens beside 2 chunks", singles=48, single_lo=500, single_hi=4096, chunks=2, new_lo=400,
                   new_hi=512, past_lo=0, past_hi=8192, page=64, strided=True, lens=2),
        # a whole prompt into an empty cache: bound by the tensor cores
        _attention("a prompt of 8192", chunks=1, new_lo=8192, new_hi=8192, page=128, strided=True),
        # a late chunk of a long prompt
        _attention("a chunk of 4096 after 28672", chunks=1, new_lo=4096, new_hi=4096, past_lo=28672, past_hi=28672,
                   page=64, lens=4),
        # ragged prompts of a model with small heads, one KV head a query head and a sliding window
        _attention("6 prompts, window of 1024", chunks=6, new_lo=200, new_hi=1500, past_lo=0, past_hi=4000, page=32,
                   window=1024, lse=True, lens=5, hq=16, hkv=16, d=64),
        # the tables of a verification step of 9 positions for 8 requests
        _tables("tables for 8 requests", "tables", 8, 9, 4096, 16),
        # the tables of a whole node's requests, prompt chunks among them, with too few free pages for all
        _tables("tables for 2048 requests", "tables", 2048, 64, 8192, 16, tight=True, lens=1),
        # the tails that a verification step rejected
        _tables("pages of 8 requests back", "release", 8, 64, 4096, 16),
        _tables("pages of 2048 requests back", "release", 2048, 256, 8192, 16, lens=1),
        # the K/V rows of one decoding step, as a rotary embedding in 32 bits leaves them
        _append("32 rows from 32 bits", 32, 16, True),
        # the K/V rows of a prompt chunk, parts of the rows of one fused projection
        _append("8192 rows of a fused projection", 8192, 64, False, strided=True),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "tables", "release", "append"])
    page, lens = rng.choice([8, 16, 32, 64, 128, 256]), rng.randrange(1 << 30)
    if kind in ("tables", "release"):
        return _tables("", kind, _log_between(rng, 1, 2048), _log_between(rng, 1, 256), _log_between(rng, 1, 8192), page,
                       rng.random() < 0.3, lens)
    if kind == "append":
        wide = rng.random() < 0.5
        return _append("", _log_between(rng, 1, 8192 if not wide else 4096), page, wide, rng.random() < 0.5, lens,
                       rng.choice([1, 2, 5, 8]), rng.choice([64, 80, 128]))
    heads = rng.choice([(32, 8, 128), (32, 8, 128), (16, 16, 64), (14, 2, 64), (8, 1, 128), (12, 4, 128)])
    singles, chunks = rng.choice([(1, 0), (1, 1), (0, 1), (0, 1)])
    singles *= _log_between(rng, 1, 64)
    single_hi = _log_between(rng, 1, 8192)
    new_hi = _log_between(rng, 2, 4096)
    past_hi = _log_between(rng, 1, 16384)
    chunks *= _log_between(rng, 1, max(1, min(8, 4096 // new_hi)))
    return _attention("", singles=singles, single_lo=max(1, single_hi // 3), single_hi=single_hi, chunks=chunks,
                      new_lo=max(1, new_hi // 2), new_hi=new_hi, past_lo=past_hi // 2, past_hi=past_hi, page=page,
                      window=rng.choice([0, 0, 0, _log_between(rng, 1, 4096)]), lse=rng.random() < 0.5,
                      strided=rng.random() < 0.5, lens=lens, hq=heads[0], hkv=heads[1], d=heads[2])


# ---------------------------------------------------------------- lengths, as a scheduler knows them on the host

def _attention_lens(case):
    """(tokens before, new tokens) of every request, single tokens among the chunks."""
    r = np.random.default_rng([17, case["lens"]])
    past = list(r.integers(case["single_lo"], case["single_hi"] + 1, case["singles"]))
    new = [1] * case["singles"]
    past += list(r.integers(case["past_lo"], case["past_hi"] + 1, case["chunks"]))
    new += list(r.integers(case["new_lo"], case["new_hi"] + 1, case["chunks"]))
    order = r.permutation(len(new))
    return [int(past[i]) for i in order], [int(new[i]) for i in order]


def _table_lens(case):
    """(tokens before, new or rejected tokens) of every request."""
    r = np.random.default_rng([18, case["lens"]])
    past = r.integers(0, case["past_hi"] + 1, case["batch"])
    new = r.integers(0, case["new_hi"] + 1, case["batch"])
    return past, new


def _visible(past, n, window):
    """Pairs of a new token and a slot that it sees."""
    p = np.arange(past, past + n, dtype=np.int64) + 1
    return int((np.minimum(p, window) if window else p).sum())


def work(case):
    if case["op"] == "attention":
        past, new = _attention_lens(case)
        hq, hkv, d, w = case["hq"], case["hkv"], case["d"], case["window"]
        rows = sum(new)
        slots = sum(p + n - (max(0, p - w + 1) if w else 0) for p, n in zip(past, new))
        return {"bytes": rows * hq * d * 4 + slots * hkv * d * 4 + (rows * hq * 4 if case["lse"] else 0),
                "flops": 4 * d * hq * sum(_visible(p, n, w) for p, n in zip(past, new))}
    if case["op"] == "append":
        return {"bytes": 2 * case["rows"] * case["hkv"] * case["d"] * ((4 if case["wide"] else 2) + 2) + 4 * case["rows"],
                "flops": 0}
    past, new = _table_lens(case)
    pages = -(-(past + new) // case["page"]) - -(-past // case["page"])
    if case["op"] == "release":
        return {"bytes": int(16 * case["batch"] + 8 * pages.sum()), "flops": 0}
    return {"bytes": int(24 * case["batch"] + 8 * pages.sum() + 4 * new.sum()), "flops": 0}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "append": _prepare_append, "tables": _prepare_tables,
            "release": _prepare_tables}[case["op"]](case, gen, seed)


def _bf16(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _int32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _paging(held, page, spare, seed):
    """A pool in use for a while: every request's pages anywhere in it, in a table with room for growth."""
    held = np.asarray(held)
    used = int(held.sum())
    order = np.random.default_rng([19, seed]).permutation(used + spare)
    table = np.full((len(held), int(held.max()) + 1 + spare // len(held)), -1, np.int64)
    table[np.arange(table.shape[1]) < held[:, None]] = order[:used]
    return table, order


def _prepare_attention(case, gen, seed):
    past, new = _attention_lens(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    pages = [-(-(p + n) // page) for p, n in zip(past, new)]
    table, order = _paging(pages, page, 3, seed)
    rows = sum(new)
    if case["strided"]:  # the query part of the rows of one fused projection
        q = _bf16(gen, rows, hq + 2 * hkv, d)[:, :hq]
    else:
        q = _bf16(gen, rows, hq, d)
    return {"op": "attention", "q": q, "k": _bf16(gen, len(order), hkv, page, d), "v": _bf16(gen, len(order), hkv, page, d),
            "table": _int32(table), "prefix": _int32(past), "starts": _int32(np.cumsum([0] + new)),
            "past": past, "new": new, "page": page, "window": case["window"], "lse": case["lse"]}


def _prepare_append(case, gen, seed):
    rows, hkv, d, page = case["rows"], case["hkv"], case["d"], case["page"]
    slots_in_use = -(-rows // page) + 8
    slots = np.random.default_rng([20, seed]).permutation(slots_in_use)[:-(-rows // page), None] * page + np.arange(page)
    slots = slots.reshape(-1)[:rows].copy()
    slots[rows - rows // 16:] = -1  # the rows that pad the batch
    dtype = torch.float32 if case["wide"] else torch.bfloat16
    if case["strided"]:  # a query head for each KV head, then the keys and the values
        qkv = torch.randn((rows, 3 * hkv, d), generator=gen, device="cuda", dtype=dtype)
        k, v = qkv[:, hkv:2 * hkv], qkv[:, 2 * hkv:]
    else:
        k, v = (torch.randn((rows, hkv, d), generator=gen, device="cuda", dtype=dtype) for _ in range(2))
    return {"op": "append", "k_new": k, "v_new": v, "slots": _int32(slots),
            "k": _bf16(gen, slots_in_use, hkv, page, d), "v": _bf16(gen, slots_in_use, hkv, page, d)}


def _prepare_tables(case, gen, seed):
    past, new = _table_lens(case)
    page, r = case["page"], np.random.default_rng([21, seed])
    if case["op"] == "release":  # every request holds the pages of its rejected tokens too
        held = -(-(past + new) // page)
        table, order = _paging(held, page, 64, seed)
        free = len(order) - int(held.sum())
        keep = past
    else:  # some hold a page that an earlier, shortened step left them
        need = -(-(past + new) // page) - -(-past // page)
        held = -(-past // page) + (r.random(len(past)) < 0.2)
        spare = max(1, int(need.sum() * (0.7 if case["tight"] else 1.2)))
        table, order = _paging(held, page, spare, seed)
        wider = np.full((len(past), int((-(-(past + new) // page)).max()) + 2), -1, np.int64)
        wider[:, :min(table.shape[1], wider.shape[1])] = table[:, :wider.shape[1]]
        table, free, keep = wider, spare, None
    stack = np.full(len(order), -1, np.int64)
    stack[:free] = order[len(order) - free:]
    return {"op": case["op"], "prefix": _int32(past), "new": _int32(new), "keep": _int32(past if keep is None else keep),
            "held": _int32(held), "table": _int32(table), "stack": _int32(stack), "free": _int32([free]), "page": page,
            "rows": int(new.sum()) + 5}  # a batch padded to a size that the program keeps


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"attention": _plain_attention, "append": _plain_append, "tables": _plain_tables,
            "release": _plain_release}[state["op"]](state)


def _run_own(s):
    import speculative_decoding_verification_81_gb300 as sv

    if s["op"] == "attention":
        out = sv.sv_chunk_attention_paged(s["q"], s["k"], s["v"], s["table"], s["prefix"], s["starts"],
                                          window=s["window"], return_lse=s["lse"])
        return list(out) if s["lse"] else [out]
    if s["op"] == "append":
        sv.sv_append_kv_paged(s["k_new"], s["v_new"], s["slots"], s["k"], s["v"])
        return [s["k"], s["v"]]
    if s["op"] == "tables":
        starts, slots, held, free = sv.sv_build_block_tables(s["prefix"], s["new"], s["held"], s["table"], s["stack"],
                                                             s["free"], s["page"], s["rows"])
        return [s["table"], starts, slots, held, free]
    held, free = sv.sv_release_pages(s["keep"], s["held"], s["table"], s["stack"], s["free"], s["page"])
    return [s["stack"], held, free]


def _attend(q, k, v, first, window):
    """q [b, n, hq, d] at positions first[b] .. first[b] + n - 1 over k, v [b, hkv, slots, d], in 32 bits."""
    b, n, hq, d = q.shape
    hkv, slots = k.shape[1:3]
    g = hq // hkv
    rows = q.float().view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    scores = (rows @ k.float().transpose(2, 3)) * (1.0 / math.sqrt(d))
    at = (first[:, None] + torch.arange(n, device=q.device))[:, :, None]
    slot = torch.arange(slots, device=q.device)
    hidden = slot > at
    if window:
        hidden |= slot <= at - window
    scores = scores.view(b, hkv, g, n, slots).masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = (scores - top).exp_()
    total = weights.sum(-1, keepdim=True)
    values = torch.where(hidden.all(1)[:, None, :, None], 0.0, v.float())  # a slot that no row sees may hold anything
    out = (weights.view(b, hkv, g * n, slots) @ values).view(b, hkv, g, n, d) / total
    lse = (top + total.log()).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d), lse.permute(0, 3, 1, 2).reshape(b, n, hq)


def _plain_attention(s):
    page, (rows, hq, d) = s["page"], s["q"].shape
    hkv = s["k"].shape[1]
    out = torch.empty((rows, hq, d), device="cuda", dtype=torch.bfloat16)
    lse = torch.empty((rows, hq), device="cuda", dtype=torch.float32)
    starts = np.cumsum([0] + s["new"])
    one = [b for b, n in enumerate(s["new"]) if n == 1]
    for group in ([one] if one else []) + [[b] for b, n in enumerate(s["new"]) if n > 1]:
        n, longest = s["new"][group[0]], max(s["past"][b] + s["new"][b] for b in group)
        picked = torch.tensor(group, device="cuda")
        table = s["table"][picked, :-(-longest // page)].clamp_min(0).long()
        k, v = (x[table].transpose(1, 2).reshape(len(group), hkv, -1, d) for x in (s["k"], s["v"]))
        at = torch.tensor(starts[group], device="cuda")[:, None] + torch.arange(n, device="cuda")
        o, e = _attend(s["q"][at], k, v, s["prefix"][picked].long(), s["window"])
        out[at], lse[at] = o.to(torch.bfloat16), e
    return [out, lse] if s["lse"] else [out]


def _plain_append(s):
    page, slots = s["k"].shape[2], s["slots"].long()
    row = torch.arange(len(slots), device="cuda")
    kept = slots >= 0
    row = torch.where(kept, row, kept.int().argmax())  # a row that pads the batch writes the first one again
    slots = slots[row]
    s["k"][slots // page, :, slots % page] = s["k_new"][row].to(torch.bfloat16)
    s["v"][slots // page, :, slots % page] = s["v_new"][row].to(torch.bfloat16)
    return [s["k"], s["v"]]


def _plain_tables(s):
    page, table = s["page"], s["table"]
    prefix, new, held, free = s["prefix"].long(), s["new"].long(), s["held"].long(), s["free"].long()
    ends = new.clamp_min(0).cumsum(0)
    starts = torch.cat([ends.new_zeros(1), ends])
    total = (prefix + new + page - 1) // page
    valid = ((prefix >= 0) & (new >= 0) & (total <= table.shape[1]) & (held <= table.shape[1])
             & (held >= (prefix + page - 1) // page) & (ends <= s["rows"]))
    need = torch.where(valid, (total - held).clamp_min(0), 0)
    upto = need.cumsum(0)
    served = valid & ((need == 0) | (upto <= free))
    column = torch.arange(table.shape[1], device="cuda")[None]
    added = (column >= held[:, None]) & (column < (held + need)[:, None])
    taken = free - 1 - ((upto - need)[:, None] + column - held[:, None])
    fresh = s["stack"][taken.clamp(0, len(s["stack"]) - 1)]
    table.copy_(torch.where(added, torch.where(served[:, None], fresh, -1), table))
    row = torch.arange(s["rows"], device="cuda")
    owner = torch.searchsorted(ends, row, right=True).clamp_max(len(new) - 1)
    at = prefix[owner] + row - starts[owner]
    live = served[owner] & (row < ends[-1])
    of = table[owner, (at // page).clamp(0, table.shape[1] - 1)]
    slots = torch.where(live, of * page + at % page, -1)
    counts = torch.where(served, held + need, held)
    left = free - torch.where(served & (need > 0), upto, 0).amax()
    return [table] + [x.to(torch.int32) for x in (starts, slots, counts, left)]


def _plain_release(s):
    page, stack = s["page"], s["stack"]
    keep, held, free = s["keep"].long(), s["held"].long(), s["free"].long()
    kept = (keep + page - 1) // page
    back = held - kept
    upto = back.cumsum(0)
    entry = torch.arange(len(stack), device="cuda") - free
    owner = torch.searchsorted(upto, entry, right=True).clamp_max(len(held) - 1)
    column = kept[owner] + entry - (upto - back)[owner]
    pushed = (entry >= 0) & (entry < upto[-1])
    stack.copy_(torch.where(pushed, s["table"][owner, column.clamp(0, s["table"].shape[1] - 1)], stack))
    return [stack, kept.to(torch.int32), (free + upto[-1]).to(torch.int32)]


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "append":
        return _exact_append(s)
    return (_exact_tables if case["op"] == "tables" else _exact_release)({k: v.tolist() if torch.is_tensor(v) else v
                                                                           for k, v in s.items()})


def _exact_attention(s):
    page, (rows, hq, d) = s["page"], s["q"].shape
    group = hq // s["k"].shape[1]
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, hq), dtype=torch.float64, device="cuda")
    row = 0
    for b, (past, n) in enumerate(zip(s["past"], s["new"])):
        slot = torch.arange(past + n, device="cuda")
        pages, offset = s["table"][b].long()[slot // page], slot % page
        for i in range(0, n, 1024):
            m = min(1024, n - i)
            p = past + i + torch.arange(m, device="cuda")[:, None]
            lo = max(0, past + i - s["window"] + 1) if s["window"] else 0
            hi = past + i + m
            sees = slot[lo:hi] <= p
            if s["window"]:
                sees &= slot[lo:hi] > p - s["window"]
            for h in range(hq):
                k = s["k"][pages[lo:hi], h // group, offset[lo:hi]].double()
                v = s["v"][pages[lo:hi], h // group, offset[lo:hi]].double()
                x = torch.einsum("id,jd->ij", s["q"][row + i:row + i + m, h].double(), k) / math.sqrt(d)
                x = torch.where(sees, x, torch.full_like(x, -math.inf))
                z = torch.logsumexp(x, 1)
                out[row + i:row + i + m, h] = torch.exp(x - z[:, None]) @ v
                lse[row + i:row + i + m, h] = z
        row += n
    return [out, lse] if s["lse"] else [out]


def _exact_append(s):
    slots = s["slots"].tolist()
    page = s["k"].shape[2]
    outs = []
    for pages, rows in ((s["k"], s["k_new"]), (s["v"], s["v_new"])):
        flat = pages.double().transpose(1, 2).reshape(-1, pages.shape[1], pages.shape[3])
        where = [i for i, x in enumerate(slots) if x >= 0]
        flat[[slots[i] for i in where]] = rows.double()[where]
        outs.append(flat.view(-1, page, *flat.shape[1:]).transpose(1, 2).contiguous())
    return outs


def _exact_tables(s):
    page, table, rows, free = s["page"], s["table"], s["rows"], s["free"][0]
    starts, slots, counts, asked, taken = [0], [-1] * rows, [], 0, 0
    for b, (past, n, held) in enumerate(zip(s["prefix"], s["new"], s["held"])):
        pages, begin = -(-(past + n) // page), starts[-1]
        starts.append(begin + n)
        need = max(0, pages - held)
        asked += need
        served = need == 0 or asked <= free
        for j in range(need):
            table[b][held + j] = s["stack"][free - 1 - (asked - need + j)] if served else -1
        counts.append(held + need if served else held)
        if served:
            taken = asked if need else taken
            for i in range(n):
                slots[begin + i] = table[b][(past + i) // page] * page + (past + i) % page
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (table, starts, slots, counts, [free - taken])]


def _exact_release(s):
    page, stack, top, counts = s["page"], s["stack"], s["free"][0], []
    for b, (keep, held) in enumerate(zip(s["keep"], s["held"])):
        counts.append(-(-keep // page))
        for j in range(counts[-1], held):
            stack[top] = s["table"][b][j]
            top += 1
    return [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (stack, counts, [top])]
