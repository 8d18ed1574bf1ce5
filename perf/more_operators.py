"""A paged cache held in 4 bits and requests that share its pages, as they are measured: new K/V rows quantised
into the pages, attention of single tokens, chains, trees and prompt chunks over them, the rows of an accepted path
moved together, requests forked, and shared pages given back.  `run` computes them in plain torch operations, or
through the library where `own` is true.

A row of a slot and KV head is D codes of 4 bits and two bf16 numbers (scale, minimum); value = minimum + scale * code.
A word of 8 dims holds dims 0, 2, 4, 6, 1, 3, 5, 7 from its lowest four bits up."""
import math

import numpy as np
import torch

own = False

#: The serving shape of the repository's bench: 32 query heads over 8 KV heads of dimension 128.
_HEADS = {"hq": 32, "hkv": 8, "d": 128}
_ORDER = [0, 2, 4, 6, 1, 3, 5, 7]


# ---------------------------------------------------------------- the cases

def _attention(name, *, seqs=0, seq_lo=1, seq_hi=1, nodes=1, tree=False, chunks=0, new_lo=1, new_hi=1, past_lo=0,
               past_hi=0, page=16, window=0, lse=False, strided=False, lens=0, **heads):
    """`seqs` requests of `nodes` rows each (single tokens, chains or trees) and `chunks` parts of prompts."""
    return {"name": name, "op": "attention", "seqs": seqs, "seq_lo": seq_lo, "seq_hi": seq_hi, "nodes": nodes,
            "tree": tree, "chunks": chunks, "new_lo": new_lo, "new_hi": new_hi, "past_lo": past_lo,
            "past_hi": past_hi, "page": page, "window": window, "lse": lse, "strided": strided, "lens": lens,
            **{**_HEADS, **heads}}


def _append(name, rows, page, wide, strided=False, hkv=8, d=128):
    return {"name": name, "op": "append", "rows": rows, "page": page, "wide": wide, "strided": strided, "hkv": hkv, "d": d}


def _compact(name, batch, nodes, past_hi, page, lens=0, hkv=8, d=128):
    return {"name": name, "op": "compact", "batch": batch, "nodes": nodes, "past_hi": past_hi, "page": page, "lens": lens,
            "hkv": hkv, "d": d}


def _fork(name, batch, forks, past_hi, page, tight=False, lens=0, hkv=8, d=128):
    return {"name": name, "op": "fork", "batch": batch, "forks": forks, "past_hi": past_hi, "page": page, "tight": tight,
            "lens": lens, "hkv": hkv, "d": d}


def _release(name, batch, branches, past_hi, new_hi, page, lens=0):
    return {"name": name, "op": "release", "batch": batch, "branches": branches, "past_hi": past_hi, "new_hi": new_hi,
            "page": page, "lens": lens}


def listed():
    return [
        # one request generating alone
        _attention("one token, 2047 before it", seqs=1, seq_lo=2047, seq_hi=2047),
        # the bench's verification step: the last token and 8 drafts of each of 32 requests
        _attention("chains of 9 for 32 requests", seqs=32, seq_lo=2048, seq_hi=4096, nodes=9, lse=True, lens=1),
        # draft trees of a model with small heads, queries as a part of a fused projection
        _attention("trees of 26, small heads", seqs=16, seq_lo=1000, seq_hi=3000, nodes=26, tree=True, page=64,
                   strided=True, lens=2, d=64),
        # a late chunk of a long prompt: bound by the tensor cores
        _attention("a chunk of 2048 after 14336", chunks=1, new_lo=2048, new_hi=2048, past_lo=14336, past_hi=14336,
                   page=128, strided=True, lens=3),
        # the rows of one decoding step, as a rotary embedding in 32 bits leaves them
        _append("32 rows in 32 bits", 32, 16, True),
        # the rows of a prompt chunk, parts of the rows of one fused projection
        _append("8192 rows of a projection", 8192, 64, False, strided=True),
        # accepted paths of draft trees
        _compact("paths of 4 trees", 4, 26, 2048, 16),
        _compact("paths of 1024 trees", 1024, 60, 600, 32, lens=1),
        # four continuations of one prompt
        _fork("4 forks of one request", 5, 4, 700, 16),
        # best-of-n sampling on a whole node, with too few free pages for all of the forks
        _fork("1024 forks of 128 requests", 1152, 1024, 8192, 16, tight=True, lens=1),
        # requests that end beside others that go on, pages of their prompts still held by some
        _release("8 branches back", 8, 4, 4096, 64, 16),
        _release("2048 branches back", 2048, 8, 2048, 256, 16, lens=1),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "attention", "append", "compact", "fork", "release"])
    page, lens = rng.choice([8, 16, 32, 64, 128, 256]), rng.randrange(1 << 30)
    hkv, d = rng.choice([1, 2, 5, 8]), rng.choice([64, 128])
    if kind == "append":
        wide = rng.random() < 0.5
        return _append("", _log_between(rng, 1, 8192 if not wide else 4096), page, wide, rng.random() < 0.5, hkv, d)
    if kind == "compact":
        return _compact("", _log_between(rng, 1, 512), rng.randrange(2, 65), _log_between(rng, 1, 900), page, lens, hkv, d)
    if kind == "fork":
        forks = _log_between(rng, 1, 512)
        return _fork("", forks + _log_between(rng, 1, 128), forks, _log_between(rng, 1, 4096), page, rng.random() < 0.3,
                     lens, hkv, d)
    if kind == "release":
        return _release("", _log_between(rng, 1, 2048), rng.randrange(1, 9), _log_between(rng, 1, 2048),
                        _log_between(rng, 1, 256), page, lens)
    heads = dict(zip(("hq", "hkv", "d"), rng.choice([(32, 8, 128), (32, 8, 128), (32, 8, 64), (16, 16, 64), (14, 2, 64),
                                                     (8, 1, 128), (12, 4, 128)])))
    common = {"page": page, "lse": rng.random() < 0.5, "strided": rng.random() < 0.5, "lens": lens, **heads}
    form = rng.choice(["single", "chain", "tree", "chunk", "mixed"])
    if form == "chunk":
        new_hi, past_hi = _log_between(rng, 2, 2048), _log_between(rng, 1, 12288)
        return _attention("", chunks=_log_between(rng, 1, max(1, min(8, 2048 // new_hi))), new_lo=max(1, new_hi // 2),
                          new_hi=new_hi, past_lo=past_hi // 2, past_hi=past_hi,
                          window=rng.choice([0, 0, _log_between(rng, 1, 4096)]), **common)
    seq_hi = _log_between(rng, 1, 4096)
    many = {"seqs": _log_between(rng, 1, 64), "seq_lo": seq_hi // 3, "seq_hi": seq_hi, **common}
    if form == "single":
        return _attention("", window=rng.choice([0, 0, 0, _log_between(rng, 1, 4096)]), **many)
    if form == "mixed":
        new_hi = _log_between(rng, 2, 512)
        return _attention("", chunks=rng.randrange(1, 4), new_lo=max(1, new_hi // 2), new_hi=new_hi, past_hi=2048, **many)
    many["seqs"] = min(many["seqs"], 32)
    return _attention("", nodes=rng.randrange(2, 65 if form == "tree" else 17), tree=form == "tree", **many)


# ---------------------------------------------------------------- lengths and structure, as a scheduler knows them on the host

def _attention_lens(case):
    """(tokens before, new rows) of every request."""
    r = np.random.default_rng([27, case["lens"]])
    past = list(r.integers(case["seq_lo"], case["seq_hi"] + 1, case["seqs"]))
    new = [case["nodes"]] * case["seqs"]
    past += list(r.integers(case["past_lo"], case["past_hi"] + 1, case["chunks"]))
    new += list(r.integers(case["new_lo"], case["new_hi"] + 1, case["chunks"]))
    order = r.permutation(len(new))
    return [int(past[i]) for i in order], [int(new[i]) for i in order]


def _trees(case, seqs):
    """Parent arrays, each parent before its children: a few wide levels, as drafts of the likeliest tokens have them."""
    r = np.random.default_rng([28, case["lens"], seqs])
    n = case["nodes"]
    parents = np.zeros((seqs, n), np.int64)
    for i in range(1, n):
        parents[:, i] = np.minimum((i - 1) // 3 + r.integers(0, 2, seqs), i - 1)
    parents[:, 0] = -1
    return parents


def _ancestors(parents):
    """[n, n] truth values: node j is i or above it."""
    n = len(parents)
    above = np.eye(n, dtype=bool)
    for i in range(1, n):
        above[i] |= above[parents[i]]
    return above


def _visible(past, n, window):
    """Pairs of a new row and a slot that it sees."""
    p = np.arange(past, past + n, dtype=np.int64) + 1
    return int((np.minimum(p, window) if window else p).sum())


def _paths(case):
    """(prefix lengths, accepted lengths, paths): a node of a path is at its place already or behind the path's end."""
    r = np.random.default_rng([29, case["lens"]])
    b, n = case["batch"], case["nodes"]
    prefix = r.integers(0, case["past_hi"] + 1, b)
    accepted = r.integers(0, max(1, min(8, n // 2)) + 1, b)
    paths = np.full((b, n), -1)
    for i, a in enumerate(accepted):
        stay = r.integers(0, a + 1)  # nodes 0 .. stay are where they belong
        later = np.sort(r.permutation(np.arange(a + 1, n))[:a - stay])
        accepted[i] = a = stay + len(later)
        paths[i, :a + 1] = np.concatenate([np.arange(stay + 1), later])
    return prefix, accepted, paths


def _fork_plan(case):
    """(lengths of all requests, sources, targets, lengths at the fork); targets hold nothing before it."""
    r = np.random.default_rng([30, case["lens"]])
    b, f = case["batch"], case["forks"]
    order = r.permutation(b)
    targets, holders = order[:f], order[f:]
    lens = np.zeros(b, np.int64)
    lens[holders] = r.integers(case["past_hi"] // 2, case["past_hi"] + 1, len(holders))
    sources = r.choice(holders, f)
    at = lens[sources] - (r.random(f) < 0.25) * r.integers(0, lens[sources] + 1)
    return lens, sources, targets, at


def _release_plan(case):
    """(tokens shared with a group's first request, tokens held, tokens kept) of every request."""
    r = np.random.default_rng([31, case["lens"]])
    b, g = case["batch"], case["branches"]
    shared = r.integers(0, case["past_hi"] + 1, -(-b // g)).repeat(g)[:b] // case["page"] * case["page"]
    held = shared + r.integers(0, case["new_hi"] + 1, b)
    keep = np.where(r.random(b) < 0.6, 0, held - r.integers(0, np.minimum(held - shared, 8) + 1))
    return shared, held, keep


def _pages(tokens, page):
    return -(-tokens // page)


def work(case):
    if case["op"] == "attention":
        past, new = _attention_lens(case)
        hq, hkv, d, w = case["hq"], case["hkv"], case["d"], case["window"]
        rows = sum(new)
        slots = sum(p + n - (max(0, p - w + 1) if w else 0) for p, n in zip(past, new))
        pairs = sum(_visible(p, n, w) for p, n in zip(past, new))
        if case["tree"]:
            pairs = sum(p * n + int(_ancestors(t).sum()) for p, n, t in zip(past, new, _trees(case, len(new))))
        return {"bytes": rows * hq * d * 4 + slots * hkv * (d + 8) + (rows * hq * 4 if case["lse"] else 0),
                "flops": 4 * d * hq * pairs}
    row = case.get("d", 0) // 2 + 4  # codes and parameters of a row
    if case["op"] == "append":
        return {"bytes": 2 * case["rows"] * case["hkv"] * (case["d"] * (4 if case["wide"] else 2) + row) + 4 * case["rows"],
                "flops": 0}
    if case["op"] == "compact":
        _, accepted, paths = _paths(case)
        moved = int(((paths >= 0) & (paths != np.arange(case["nodes"]))).sum())
        return {"bytes": 4 * moved * case["hkv"] * row + 4 * int(accepted.sum()) + 12 * case["batch"], "flops": 0}
    page = case["page"]
    if case["op"] == "fork":
        lens, _, _, at = _fork_plan(case)
        pool = int(_pages(lens, page).sum()) + case["forks"]
        return {"bytes": int(8 * (at // page).sum() + 4 * (at % page).sum() * case["hkv"] * row + 8 * pool
                             + 40 * case["forks"] + 8 * case["batch"]), "flops": 0}
    shared, held, keep = _release_plan(case)
    back = int((_pages(held, page) - _pages(keep, page)).sum())
    pool = int((_pages(held, page) - shared // page).sum() + (shared[::case["branches"]] // page).sum()) + 16
    return {"bytes": 12 * back + 8 * pool + 16 * case["batch"], "flops": 0}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"attention": _prepare_attention, "append": _prepare_append, "compact": _prepare_compact,
            "fork": _prepare_fork, "release": _prepare_release}[case["op"]](case, gen, seed)


def _int32(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def _quantised(rows):
    """Codes and parameters of rows [..., d] in 32 bits."""
    lo, hi = rows.amin(-1, keepdim=True), rows.amax(-1, keepdim=True)
    scale = ((hi - lo) * (1.0 / 15.0)).to(torch.bfloat16).float()
    scale = torch.where(scale < 2.0 ** -126, 0.0, scale)
    low = lo.to(torch.bfloat16).float()
    codes = torch.where(scale > 0, torch.round((rows - low) * (1.0 / scale)), 0.0).clamp_(0, 15).to(torch.uint8)
    codes = codes.view(*codes.shape[:-1], -1, 8)[..., _ORDER]
    codes = (codes[..., 0::2] | codes[..., 1::2] << 4).flatten(-2)
    return codes, torch.cat([scale, low], -1).to(torch.bfloat16)


def _values(codes, params):
    """The rows that codes [..., d / 2] and parameters stand for, in 32 bits."""
    parts = torch.stack([codes & 15, codes >> 4], -1).view(*codes.shape[:-1], -1, 8).float()
    whole = torch.empty_like(parts)
    whole[..., _ORDER] = parts
    params = params.float()
    return params[..., 1:] + params[..., :1] * whole.flatten(-2)


def _cache(gen, pages, hkv, page, d):
    """Pages of K or V rows, their heads and dims of unlike size as a model's are."""
    size = torch.rand((1, hkv, 1, d), generator=gen, device="cuda") * 1.5 + 0.25
    parts = [_quantised(torch.randn((n, hkv, page, d), generator=gen, device="cuda") * size)
             for n in [min(4096, pages - i) for i in range(0, pages, 4096)]]
    return [torch.cat(x) for x in zip(*parts)]


def _paging(held, page, spare, seed):
    """A pool in use for a while: every request's pages anywhere in it, in a table with room for growth."""
    held = np.asarray(held)
    used = int(held.sum())
    order = np.random.default_rng([32, seed]).permutation(used + spare)
    table = np.full((len(held), int(held.max()) + 2), -1, np.int64)
    table[np.arange(table.shape[1]) < held[:, None]] = order[:used]
    return table, order


def _prepare_attention(case, gen, seed):
    past, new = _attention_lens(case)
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    table, order = _paging([_pages(p + n, page) for p, n in zip(past, new)], page, 3, seed)
    rows = sum(new)
    q = torch.randn((rows, hq + (2 * hkv if case["strided"] else 0), d), generator=gen, device="cuda").to(torch.bfloat16)
    trees = _trees(case, len(new)) if case["tree"] else None
    return {"op": "attention", "q": q[:, :hq], "k": _cache(gen, len(order), hkv, page, d),
            "v": _cache(gen, len(order), hkv, page, d), "table": _int32(table), "prefix": _int32(past),
            "starts": _int32(np.cumsum([0] + new)), "past": past, "new": new, "page": page, "window": case["window"],
            "lse": case["lse"], "parents": None if trees is None else _int32(trees.reshape(-1)),
            "depth": 0 if trees is None else int(max(_ancestors(t).sum(1).max() for t in trees))}


def _prepare_append(case, gen, seed):
    rows, hkv, d, page = case["rows"], case["hkv"], case["d"], case["page"]
    count = _pages(rows, page) + 8
    slots = np.random.default_rng([33, seed]).permutation(count)[:_pages(rows, page), None] * page + np.arange(page)
    slots = slots.reshape(-1)[:rows].copy()
    slots[rows - rows // 16:] = -1  # the rows that pad the batch
    dtype = torch.float32 if case["wide"] else torch.bfloat16
    # (strided: a query head for each KV head, then the keys and the values)
    qkv = [torch.randn((rows, (3 if case["strided"] else 1) * hkv, d), generator=gen, device="cuda").to(dtype)
           for _ in range(1 if case["strided"] else 2)]
    k, v = (qkv[0][:, hkv:2 * hkv], qkv[0][:, 2 * hkv:]) if case["strided"] else qkv
    return {"op": "append", "k_new": k, "v_new": v, "slots": _int32(slots), "k": _cache(gen, count, hkv, page, d),
            "v": _cache(gen, count, hkv, page, d)}


def _prepare_compact(case, gen, seed):
    prefix, accepted, paths = _paths(case)
    page = case["page"]
    table, order = _paging(_pages(prefix + case["nodes"], page), page, 2, seed)
    return {"op": "compact", "k": _cache(gen, len(order), case["hkv"], page, case["d"]),
            "v": _cache(gen, len(order), case["hkv"], page, case["d"]), "table": _int32(table), "prefix": _int32(prefix),
            "accepted": _int32(accepted), "paths": _int32(paths)}


def _prepare_fork(case, gen, seed):
    lens, sources, targets, at = _fork_plan(case)
    page = case["page"]
    held = _pages(lens, page)
    need = int((at % page != 0).sum())
    spare = max(1, int(need * 0.7) if case["tight"] else case["forks"])
    table, order = _paging(held, page, spare, seed)
    stack = np.full(len(order), -1, np.int64)
    stack[:spare] = order[len(order) - spare:]
    shares = np.zeros(len(order), np.int64)
    shares[order[:len(order) - spare]] = np.random.default_rng([34, seed]).integers(0, 2, len(order) - spare)
    return {"op": "fork", "k": _cache(gen, len(order), case["hkv"], page, case["d"]),
            "v": _cache(gen, len(order), case["hkv"], page, case["d"]), "table": _int32(table), "sources": _int32(sources),
            "targets": _int32(targets), "at": _int32(at), "held": _int32(held), "stack": _int32(stack),
            "free": _int32([spare]), "shares": _int32(shares), "page": page}


def _prepare_release(case, gen, seed):
    shared, held, keep = _release_plan(case)
    page, g, r = case["page"], case["branches"], np.random.default_rng([35, seed])
    common, total = shared // page, _pages(held, page)
    pool = int((total - common).sum() + common[::g].sum()) + 16
    order = list(r.permutation(pool))
    table = np.full((len(held), int(total.max()) + 1), -1, np.int64)
    shares = np.zeros(pool, np.int64)
    for b in range(len(held)):
        if b % g == 0:
            first = [order.pop() for _ in range(common[b])]
        shares[first] += b % g > 0
        table[b, :total[b]] = first + [order.pop() for _ in range(total[b] - common[b])]
    stack = np.full(pool, -1, np.int64)
    stack[:16] = order
    return {"op": "release", "keep": _int32(keep), "held": _int32(total), "table": _int32(table), "stack": _int32(stack),
            "free": _int32([16]), "shares": _int32(shares), "page": page}


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"attention": _plain_attention, "append": _plain_append, "compact": _plain_compact, "fork": _plain_fork,
            "release": _plain_release}[state["op"]](state)


def _run_own(s):
    import speculative_decoding_verification_81_gb300 as sv

    if s["op"] == "attention":
        out = sv.sv_chunk_attention_quant(s["q"], *s["k"], *s["v"], s["table"], s["prefix"], s["starts"],
                                          parents=s["parents"], window=s["window"], return_lse=s["lse"])
        return list(out) if s["lse"] else [out]
    if s["op"] == "append":
        sv.sv_append_kv_quant(s["k_new"], s["v_new"], s["slots"], *s["k"], *s["v"])
        return [*s["k"], *s["v"]]
    if s["op"] == "compact":
        lens = sv.sv_compact_kv_quant(*s["k"], *s["v"], s["table"], s["prefix"], s["accepted"], s["paths"])
        return [*s["k"], *s["v"], lens]
    if s["op"] == "fork":
        copies, counts, free, shares = sv.sv_fork_tables(s["sources"], s["targets"], s["at"], s["held"], s["table"],
                                                         s["stack"], s["free"], s["shares"], s["page"])
        sv.sv_copy_pages(copies, [*s["k"], *s["v"]])
        return [s["table"], copies, counts, free, shares, *s["k"], *s["v"]]
    counts, free, shares = sv.sv_release_shared_pages(s["keep"], s["held"], s["table"], s["stack"], s["free"], s["shares"],
                                                      s["page"])
    return [s["stack"], counts, free, shares]


def _attend(q, k, v, hidden):
    """q [b, n, hq, d] over k, v [b, hkv, slots, d] in 32 bits; hidden [b, n, slots]."""
    b, n, hq, d = q.shape
    hkv, slots = k.shape[1:3]
    g = hq // hkv
    rows = q.float().view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    scores = (rows @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    scores = scores.view(b, hkv, g, n, slots).masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = (scores - top).exp_()
    total = weights.sum(-1, keepdim=True)
    seen = torch.where(hidden.all(1)[:, None, :, None], 0.0, v)  # a slot that no row sees may hold anything
    out = (weights.view(b, hkv, g * n, slots) @ seen).view(b, hkv, g, n, d) / total
    lse = (top + total.log()).squeeze(-1)
    return out.permute(0, 3, 1, 2, 4).reshape(b, n, hq, d), lse.permute(0, 3, 1, 2).reshape(b, n, hq)


def _plain_attention(s):
    page, (rows, hq, d) = s["page"], s["q"].shape
    hkv = s["k"][0].shape[1]
    out = torch.empty((rows, hq, d), device="cuda", dtype=torch.bfloat16)
    lse = torch.empty((rows, hq), device="cuda", dtype=torch.float32)
    starts = np.cumsum([0] + s["new"])
    one = [b for b, n in enumerate(s["new"]) if n == 1]
    for group in [one[i:i + 16] for i in range(0, len(one), 16)] + [[b] for b, n in enumerate(s["new"]) if n > 1]:
        n, longest = s["new"][group[0]], max(s["past"][b] + s["new"][b] for b in group)
        picked = torch.tensor(group, device="cuda")
        table = s["table"][picked, :_pages(longest, page)].clamp_min(0).long()
        k, v = (_values(*(x[table].transpose(1, 2).reshape(len(group), hkv, -1, x.shape[3]) for x in c))
                for c in (s["k"], s["v"]))
        first, row = s["prefix"][picked].long()[:, None], torch.arange(n, device="cuda")
        slot = torch.arange(k.shape[2], device="cuda")
        hidden = slot > (first + row)[:, :, None]
        if s["window"]:
            hidden |= slot <= (first + row)[:, :, None] - s["window"]
        at = torch.tensor(starts[group], device="cuda")[:, None] + row
        if s["parents"] is not None:
            above, node = torch.zeros((len(group), n, k.shape[2]), dtype=torch.bool, device="cuda"), row.expand(len(group), n)
            parents = s["parents"][at].long()
            for _ in range(s["depth"]):
                above |= (slot == (first + node)[:, :, None]) & (node >= 0)[:, :, None]
                node = torch.where(node >= 0, parents.gather(1, node.clamp_min(0)), -1)
            hidden = ~(above | (slot < first)[:, None])
        o, e = _attend(s["q"][at], k, v, hidden)
        out[at], lse[at] = o.to(torch.bfloat16), e
    return [out, lse] if s["lse"] else [out]


def _plain_append(s):
    page, slots = s["k"][0].shape[2], s["slots"].long()
    row = torch.arange(len(slots), device="cuda")
    kept = slots >= 0
    row = torch.where(kept, row, kept.int().argmax())  # a row that pads the batch writes the first one again
    slots = slots[row]
    for new, cache in ((s["k_new"], s["k"]), (s["v_new"], s["v"])):
        for x, y in zip(cache, _quantised(new[row].float())):
            x[slots // page, :, slots % page] = y
    return [*s["k"], *s["v"]]


def _plain_compact(s):
    page, prefix, accepted = s["k"][0].shape[2], s["prefix"].long(), s["accepted"].long()
    d = torch.arange(s["paths"].shape[1], device="cuda")
    on = d <= accepted[:, None]
    source, target = (prefix[:, None] + torch.where(on, x, 0) for x in (s["paths"].long(), d))
    pages_from, pages_to = (s["table"].long().gather(1, x // page) for x in (source, target))
    for x in (*s["k"], *s["v"]):
        x[pages_to, :, target % page] = x[pages_from, :, source % page]
    return [*s["k"], *s["v"], (prefix + accepted + 1).to(torch.int32)]


def _plain_fork(s):
    page, table = s["page"], s["table"]
    sources, targets, at, held, free = (s[x].long() for x in ("sources", "targets", "at", "held", "free"))
    full, part = at // page, at % page
    valid = (at >= 0) & (full + (part > 0) <= held[sources]) & (held[targets] == 0) & (sources != targets)
    need = (valid & (part > 0)).long()
    upto = need.cumsum(0)
    served = valid & ((need == 0) | (upto <= free))
    fresh = s["stack"].long()[(free - upto).clamp(0, len(s["stack"]) - 1)]
    column = torch.arange(table.shape[1], device="cuda")
    old = table[sources]
    shared = served[:, None] & (column < full[:, None])
    new = torch.where(shared, old, table[targets])
    last = column == full[:, None]
    given = last & (served & (need > 0))[:, None]
    table[targets] = torch.where(given, fresh[:, None].to(torch.int32), new)
    shares = s["shares"].long().index_add(0, torch.where(shared, old, 0).flatten().long(), shared.flatten().long())
    copied = served & (need > 0)
    origin = old.gather(1, full.clamp_max(table.shape[1] - 1)[:, None])[:, 0].long()
    copies = torch.stack([torch.where(copied, origin, -1), torch.where(copied, fresh, -1), torch.where(copied, part, 0)], 1)
    counts = held.index_copy(0, targets, torch.where(served, full + need, held[targets]))
    left = free - torch.where(copied, upto, 0).amax()
    slot = torch.arange(page, device="cuda")
    first = copied.int().argmax()  # (a fork without a copy makes the first one's again)
    source, target, rows = (torch.where(copied, x, x[first]) for x in (origin, fresh, part))
    some = copied.any()
    for x in (*s["k"], *s["v"]):
        move = (some & (slot < rows[:, None]))[:, None, :, None]
        x[target] = torch.where(move, x[source], x[target])
    return [table, copies.to(torch.int32), counts.to(torch.int32), left.to(torch.int32), shares.to(torch.int32),
            *s["k"], *s["v"]]


def _plain_release(s):
    page, stack, table = s["page"], s["stack"], s["table"]
    keep, held, free, shares = (s[x].long() for x in ("keep", "held", "free", "shares"))
    kept = _pages(keep, page)
    column = torch.arange(table.shape[1], device="cuda")
    back = ((column >= kept[:, None]) & (column < held[:, None])).flatten()
    entry = torch.arange(back.numel(), device="cuda")
    page_of = torch.where(back, table.flatten().long(), len(stack))  # (one place more, for the entries that stay)
    times = torch.zeros(len(stack) + 1, dtype=torch.long, device="cuda").index_add(0, page_of, back.long())[:-1]
    last = torch.full((len(stack) + 1,), -1, dtype=torch.long, device="cuda").scatter_reduce(0, page_of, entry, "amax")[:-1]
    last = torch.where(times > shares, last, -1)
    pushed = torch.cat([last, last.new_full((1,), -1)])[page_of] == entry
    pushed &= back
    at = torch.arange(len(stack), device="cuda")
    taken = torch.searchsorted(pushed.long().cumsum(0), at - free + 1).clamp_max(back.numel() - 1)
    count = pushed.sum()
    stack.copy_(torch.where((at >= free) & (at < free + count), page_of[taken].to(torch.int32), stack))
    return [stack, kept.to(torch.int32), (free + count).to(torch.int32), (shares - times).clamp_min(0).to(torch.int32)]


# ---------------------------------------------------------------- in 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    host = {k: v.cpu() if torch.is_tensor(v) else [x.cpu() for x in v] if isinstance(v, list) else v for k, v in s.items()}
    return {"append": _exact_append, "compact": _exact_compact, "fork": _exact_fork, "release": _exact_release}[case["op"]](host)


def _read64(codes, params):
    """Rows that packed codes stand for, in 64 bits."""
    out = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device=codes.device)
    for i, dim in enumerate((0, 2, 4, 6, 1, 3, 5, 7)):
        out[..., dim::8] = (codes[..., i // 2::4] >> 4 * (i % 2)) & 15
    return params[..., 1:].double() + params[..., :1].double() * out


def _exact_attention(s):
    page, (rows, hq, d) = s["page"], s["q"].shape
    group = hq // s["k"][0].shape[1]
    out = torch.zeros((rows, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((rows, hq), dtype=torch.float64, device="cuda")
    row = 0
    for past, n, table in zip(s["past"], s["new"], s["table"].long()):
        slot = torch.arange(past + n, device="cuda")
        pages, offset = table[slot // page], slot % page
        if s["parents"] is not None:
            above = torch.tensor(_ancestors(s["parents"][row:row + n].tolist()), device="cuda")
        for h in range(hq):
            if h % group == 0:
                k, v = (_read64(c[0][pages, h // group, offset], c[1][pages, h // group, offset]) for c in (s["k"], s["v"]))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                p = past + i + torch.arange(m, device="cuda")[:, None]
                sees = slot <= p
                if s["window"]:
                    sees &= slot > p - s["window"]
                if s["parents"] is not None:
                    sees[:, past:] = above[i:i + m]
                x = s["q"][row + i:row + i + m, h].double() @ k.T / math.sqrt(d)
                x = torch.where(sees, x, -math.inf)
                z = torch.logsumexp(x, 1)
                out[row + i:row + i + m, h] = torch.exp(x - z[:, None]) @ v
                lse[row + i:row + i + m, h] = z
        row += n
    return [out, lse] if s["lse"] else [out]


def _exact_append(s):
    page, outs = s["k"][0].shape[2], []
    where = [i for i, x in enumerate(s["slots"].tolist()) if x >= 0]
    slots = s["slots"].numpy()[where]
    for new, (codes, params) in ((s["k_new"], s["k"]), (s["v_new"], s["v"])):
        x = new[where].float().numpy()  # the format's own arithmetic is in 32 bits
        lo, hi = x.min(-1), x.max(-1)
        scale = torch.from_numpy((hi - lo) * np.float32(1.0 / 15.0)).to(torch.bfloat16)
        low = torch.from_numpy(lo).to(torch.bfloat16)
        step, base = scale.float().numpy(), low.float().numpy()
        c = np.rint((x - base[..., None]) * (np.float32(1) / step)[..., None]).clip(0, 15).astype(np.uint8)
        packed = np.zeros((*c.shape[:-1], c.shape[-1] // 2), np.uint8)
        for i, dim in enumerate((0, 2, 4, 6, 1, 3, 5, 7)):
            packed[..., i // 2::4] |= c[..., dim::8] << (4 * (i % 2))
        codes[slots // page, :, slots % page] = torch.from_numpy(packed)
        params[slots // page, :, slots % page] = torch.stack([scale, low], -1)
        outs += [codes, params]
    return outs


def _exact_compact(s):
    page, lens = s["k"][0].shape[2], []
    for b, (prefix, accepted) in enumerate(zip(s["prefix"].tolist(), s["accepted"].tolist())):
        table = s["table"][b].tolist()
        for d in range(accepted + 1):
            i, j = prefix + int(s["paths"][b, d]), prefix + d
            if i != j:
                for x in (*s["k"], *s["v"]):
                    x[table[j // page], :, j % page] = x[table[i // page], :, i % page]
        lens.append(prefix + accepted + 1)
    return [*s["k"], *s["v"], torch.tensor(lens, dtype=torch.int32)]


def _exact_fork(s):
    page, table, stack, shares = s["page"], s["table"].clone(), s["stack"].tolist(), s["shares"].clone()
    counts, free, asked, taken, copies = s["held"].clone(), int(s["free"]), 0, 0, []
    for source, target, at in zip(s["sources"].tolist(), s["targets"].tolist(), s["at"].tolist()):
        full, part = divmod(at, page)
        asked += part > 0
        copy = [-1, -1, 0]
        if part == 0 or asked <= free:
            table[target, :full] = s["table"][source, :full]
            shares[s["table"][source, :full].long()] += 1
            counts[target] = full + (part > 0)
            if part:
                copy = [int(s["table"][source, full]), stack[free - asked], part]
                table[target, full] = copy[1]
                taken = asked
                for x in (*s["k"], *s["v"]):
                    x[copy[1], :, :part] = x[copy[0], :, :part]
        copies.append(copy)
    return [table, torch.tensor(copies, dtype=torch.int32), counts, torch.tensor([free - taken], dtype=torch.int32), shares,
            *s["k"], *s["v"]]


def _exact_release(s):
    page, stack, shares, top = s["page"], s["stack"].tolist(), s["shares"].tolist(), int(s["free"])
    keep, held, table = s["keep"].tolist(), s["held"].tolist(), s["table"].tolist()
    back = [p for b in range(len(keep)) for p in table[b][_pages(keep[b], page):held[b]]]
    last = {p: i for i, p in enumerate(back)}
    for i, p in enumerate(back):
        if shares[p] > 0 and last[p] != i:
            shares[p] -= 1
        elif last[p] == i:  # its last holder in this call: another one may be left
            if shares[p] > 0:
                shares[p] -= 1
            else:
                stack[top] = p
                top += 1
    return [torch.tensor(x, dtype=torch.int32) for x in (stack, [_pages(k, page) for k in keep], [top], shares)]
