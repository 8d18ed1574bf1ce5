"""The calls of a cache held in 4 bits and of requests that share pages as a server
makes them: one after another over the same pages, captured and replayed, on other
streams, forms of the attention taking turns in one workspace, caches past 2^32
bytes, query rows that are not finite."""
import numpy as np
import pytest
import torch

import quant_ref
import speculative_decoding_verification_81_gb300 as sv
from test_gpu_chunk import Case as Bf16Case
from test_gpu_quant import Case, i32, near

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


# ---------------------------------------------------------------- a run of them

@pytest.mark.parametrize("hq,hkv,d,ps", [(8, 2, 128, 16), (4, 4, 64, 8), (16, 2, 64, 128)])
def test_a_request_forked_drafted_and_given_back(hq, hkv, d, ps):
    """A prompt, two branches of it, a draft tree on each of the three, the accepted paths, a token
    more, and everything given back.  The cache is read back for the reference, so that only the
    attention's own roundings count; the tables and counts are whole numbers."""
    gen = torch.Generator(device="cuda").manual_seed(d + ps)
    rng = np.random.default_rng(ps)
    B, mp, n_pages, prompt = 3, 600 // ps + 3, 3 * (600 // ps) + 20, 421
    k = [torch.full((n_pages, hkv, ps, d // 2), 0x5a, dtype=torch.uint8, device="cuda"),
         torch.full((n_pages, hkv, ps, 2), NAN, dtype=torch.bfloat16, device="cuda")]
    v = [t.clone() for t in k]
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    stack, free = i32(rng.permutation(n_pages)), i32([n_pages])
    counts, shares, lens = i32([0] * B), i32([0] * n_pages), i32([0] * B)

    def step(new, trees=None):
        nonlocal counts, free
        rows = sum(new)
        starts, slots, counts, free = sv.sv_build_block_tables(lens, i32(new), counts, table, stack, free, ps, rows)
        qkv = torch.randn((rows, hq + 2 * hkv, d), generator=gen, device="cuda").to(torch.bfloat16)
        sv.sv_append_kv_quant(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], slots, *k, *v)
        parents = None if trees is None else i32(np.concatenate(trees))
        out, lse = sv.sv_chunk_attention_quant(qkv[:, :hq], *k, *v, table, lens, starts, parents=parents, return_lse=True)
        near(out, lse, quant_ref.attention(qkv[:, :hq], k, v, table, lens.tolist(), new, starts.tolist(), d ** -0.5, 0, trees))

    step([prompt, 0, 0])
    lens = i32([prompt, 0, 0])
    at = [prompt, prompt - 5]
    copies, counts, free, shares = sv.sv_fork_tables(i32([0, 0]), i32([1, 2]), i32(at), counts, table, stack, free, shares, ps)
    sv.sv_copy_pages(copies, [*k, *v])
    lens = i32([prompt, *at])
    assert shares.sum().item() == sum(n // ps for n in at)
    nodes = 11
    trees = [np.array([-1] + [int(rng.integers(0, i)) for i in range(1, nodes)]) for _ in range(B)]
    step([nodes] * B, trees)
    paths, accepted = np.full((B, nodes), -1), []
    for b, tree in enumerate(trees):
        path = [int(rng.integers(1, nodes))]
        while path[0] > 0:
            path.insert(0, int(tree[path[0]]))
        accepted.append(len(path) - 1)
        paths[b, :len(path)] = path
    old = [quant_ref.values(*c) for c in (k, v)]
    lens_before = lens.tolist()
    lens = sv.sv_compact_kv_quant(*k, *v, table, lens, i32(accepted), i32(paths))
    assert lens.tolist() == [a + n + 1 for a, n in zip(lens_before, accepted)]
    for b in range(B):
        for i in range(accepted[b] + 1):
            x, y = lens_before[b] + paths[b, i], lens_before[b] + i
            for c, o in zip((k, v), old):
                now = quant_ref.values(*c)[table[b, y // ps].item(), :, y % ps]
                assert torch.equal(now, o[table[b, x // ps].item(), :, x % ps])
    step([1] * B)
    counts, free, shares = sv.sv_release_shared_pages(i32([0] * B), counts, table, stack, free, shares, ps)
    assert counts.tolist() == [0] * B and free.item() == n_pages and not shares.any()
    assert sorted(stack.tolist()) == list(range(n_pages))


# ---------------------------------------------------------------- captured, on other streams, in turns

CASES = {
    "single tokens": ([(700, 1), (3, 1), (1500, 1)], dict(hq=32, hkv=8)),
    "one long token": ([(20000, 1)], dict(hq=8, hkv=8)),
    "chains": ([(900, 9)] * 5, dict(hq=32, hkv=8)),
    "trees": ([(300, 26)] * 3, dict(hq=8, hkv=2, tree=3)),
    "a prompt": ([(500, 300), (0, 1)], dict(hq=8, hkv=1)),
    "many single tokens": ([(i % 90, 1) for i in range(400)], dict(hq=32, hkv=8)),
}


def fixed(c):
    """The case's call with its arrays already on the GPU."""
    past, starts = i32(c.past), i32(c.starts)
    return lambda **kw: sv.sv_chunk_attention_quant(c.q, *c.k, *c.v, c.table, past, starts, parents=c.parents, scale=c.scale,
                                                    return_lse=True, **kw)


def test_forms_take_turns_in_one_workspace():
    """Every call of a kind has one answer, bit for bit, whatever ran before it in the workspace, which
    the calls over the bf16 cache share."""
    cases = {name: Case(lens, seed=3, **kw) for name, (lens, kw) in CASES.items()}
    for name in ("single tokens", "a prompt", "many single tokens"):
        lens, kw = CASES[name]
        cases[f"{name}, bf16"] = Bf16Case(lens, seed=3, **kw)
    first = {name: [t.clone() for t in c.run()] for name, c in cases.items()}
    rng = np.random.default_rng(4)
    for name in rng.choice(list(cases), 60):
        assert same(cases[name].run(), first[name]), name


@pytest.mark.parametrize("seed", range(8))
def test_items_of_one_and_of_two_tiles_in_turn(seed):
    """Chunks whose rows fill one or two of the kernel's tiles of queries, beside single tokens, each call
    on pages that no cache holds: within the bounds, and the same bits every time."""
    rng = np.random.default_rng(100 + seed)
    page_size, d = int(rng.choice([16, 32, 64])), 128 if seed % 4 else 64
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for i in range(4):
        lens = [(int(rng.integers(0, 2000)), int(rng.integers(30, 400))) for _ in range(rng.integers(3, 7))]
        lens += [(int(rng.integers(1, 40)), 1) for _ in range(rng.integers(0, 30))]
        c = Case([lens[j] for j in rng.permutation(len(lens))], hq=32, hkv=8, d=d, page_size=page_size, seed=int(rng.integers(1000)))
        run = fixed(c)
        flush.fill_(i)
        first = run()
        near(*first, c.want())
        for _ in range(6):
            flush.fill_(i + 1)
            assert same(run(), first)


@pytest.mark.parametrize("name", CASES)
def test_captured_and_replayed(name):
    lens, kw = CASES[name]
    c = Case(lens, seed=5, **kw)
    want, run = c.check(), fixed(c)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    graphs = []
    for _ in range(2):  # (each graph has a workspace of its own)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(out=out, lse=lse)
            run(out=out, lse=lse)
        graphs.append(g)
    for g in (graphs[0], graphs[1], graphs[0]):
        out.fill_(1.0)
        lse.fill_(1.0)
        g.replay()
        run()
        torch.cuda.synchronize()
        assert same((out, lse), want)


def test_tables_and_rows_captured():
    rng = np.random.default_rng(6)
    B, ps, mp = 2100, 16, 30
    held = rng.integers(1, mp + 1, B)
    ids = rng.permutation(int(held.sum()) + 7)
    table = np.full((B, mp), -1)
    table[np.arange(mp) < held[:, None]] = ids[:held.sum()]
    stack = np.full(len(ids), -3)
    stack[:7] = ids[held.sum():]
    args = [i32(rng.integers(0, 2, B) * held * ps), i32(held), i32(table), i32(stack), i32([7]), i32([0] * len(ids))]
    want = sv.sv_release_shared_pages(*args[:3], s0 := i32(stack), *args[4:], ps)
    rows, hkv, d = 40, 3, 64
    kn, vn = (torch.randn((rows, hkv, d), device="cuda") for _ in range(2))
    planes = [torch.zeros((6, hkv, 8, x), dtype=t, device="cuda") for x, t in ((d // 2, torch.uint8), (2, torch.bfloat16)) * 2]
    slots = i32(rng.permutation(48)[:rows])
    sv.sv_append_kv_quant(kn, vn, slots, *planes)
    again = [torch.zeros_like(t) for t in planes]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sv.sv_release_shared_pages(*args, ps)
        sv.sv_append_kv_quant(kn, vn, slots, *again)
    for _ in range(2):
        args[3].copy_(i32(stack))
        g.replay()
        torch.cuda.synchronize()
        assert same(got, want) and torch.equal(args[3], s0) and same(again, planes)


@pytest.mark.parametrize("given", [True, False])
def test_another_stream(given):
    side = torch.cuda.Stream()
    for name in ("single tokens", "trees"):
        lens, kw = CASES[name]
        c = Case(lens, seed=7, **kw)
        want, run = c.check(), fixed(c)
        torch.cuda.synchronize()
        if given:
            got = [run(stream=side) for _ in range(3)]
        else:
            with torch.cuda.stream(side):
                got = [run() for _ in range(3)]
        side.synchronize()
        assert all(same(x, want) for x in got)


# ---------------------------------------------------------------- the ends of the ranges

def test_a_cache_past_32_bits_of_bytes():
    """Pages at the end of codes of 4.5 GB: rows written, read by each form, moved and copied there."""
    hkv, d, ps = 8, 128, 128
    n_pages = (9 << 29) // (hkv * ps * d // 2)
    codes = [torch.empty((n_pages, hkv, ps, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    params = [torch.empty((n_pages, hkv, ps, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = [codes[0], params[0]], [codes[1], params[1]]
    assert codes[0].numel() > 1 << 32
    ids = [n_pages - 1, 0, n_pages - 2, n_pages // 2 + 1, n_pages - 3]
    table = i32([ids[:4]])
    past, new = 380, 40
    gen = torch.Generator(device="cuda").manual_seed(8)
    kn, vn = (torch.randn((past + new, hkv, d), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = i32([ids[s // ps] * ps + s % ps for s in range(past + new)])
    st = torch.full((past + new,), -7, dtype=torch.int32, device="cuda")
    sv.sv_append_kv_quant(kn, vn, slots, *k, *v, row_status=st)
    assert not st.any()
    small = [[t[ids] for t in c] for c in (k, v)]   # the same pages, few of them
    q = torch.randn((new, 32, d), generator=gen, device="cuda").to(torch.bfloat16)
    for rows in (1, 9, new):
        got = sv.sv_chunk_attention_quant(q[:rows], *k, *v, table, i32([past]), i32([0, rows]), return_lse=True)
        want = sv.sv_chunk_attention_quant(q[:rows], *small[0], *small[1], i32([[0, 1, 2, 3]]), i32([past]), i32([0, rows]),
                                           return_lse=True)
        assert same(got, want), rows
    sv.sv_copy_pages(i32([[ids[0], ids[4], ps]]), [*k, *v])
    assert all(torch.equal(bits(t[ids[0]]), bits(t[ids[4]])) for t in (*k, *v))
    path = i32([[0, 20, 39]])
    assert sv.sv_compact_kv_quant(*k, *v, table, i32([past]), i32([2]), path).tolist() == [past + 3]
    sv.sv_compact_kv_quant(*small[0], *small[1], i32([[0, 1, 2, 3]]), i32([past]), i32([2]), path)
    for big, few in zip((*k, *v), (*small[0], *small[1])):
        assert torch.equal(bits(big[ids[:4]]), bits(few[:4]))


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("value,whole", [(NAN, False), (NAN, True), (INF, False), (-INF, True)])
def test_a_query_row_that_is_not_finite(name, value, whole):
    """It shows in its own out and lse, and in no other row's: of those not a bit changes."""
    lens, kw = CASES[name]
    c = Case(lens, seed=9, **kw)
    want = c.run()
    out, lse = (t.clone() for t in want)
    hit = torch.zeros(lse.shape, dtype=torch.bool, device="cuda")
    for i, r in enumerate(range(0, out.shape[0], max(1, out.shape[0] // 4))):
        h = (3 * i + 1) % lse.shape[1]
        c.q[r, h, slice(None) if whole else 5] = value
        hit[r, h] = True
    o, e = c.run()
    assert torch.isnan(o[hit]).all() and not torch.isfinite(e[hit]).any()
    assert torch.equal(bits(o[~hit]), bits(out[~hit])) and torch.equal(bits(e[~hit]), bits(lse[~hit]))


def test_rows_of_V_of_many_sizes():
    """Slots whose values lie 2^60 and more apart: each output within its bound, which is of the size
    of the values that the row has weight on."""
    for lens, kw in (([(700, 1)], dict(hq=8, hkv=1)), ([(700, 40)], dict(hq=8, hkv=1))):
        c = Case(lens, seed=11, **kw)
        for size in (0.0, 2.0 ** -90, 2.0 ** 40):
            d = Case(lens, seed=11, **kw)
            d.v[1].nan_to_num_().mul_(size)
            if size:
                d.check()
            else:  # (an error relative to nothing has no size: zeros, and the lse within its bound)
                (out, lse), (_, e, _, eb) = d.run(), d.want()
                assert not out.any() and ((lse.double() - e).abs() <= eb).all()
        # one sequence, tiles of very different sizes
        scale = torch.tensor([2.0 ** (20 * (i % 3) - 20) for i in range(c.v[1].shape[0])], device="cuda")
        c.v[1].mul_(scale[:, None, None, None].to(torch.bfloat16))
        c.check()
