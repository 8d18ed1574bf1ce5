"""Forked requests, copies of pages and shared pages given back, on the GPU against their
definitions taken one fork and one entry at a time (whole numbers and copied bits: equal)."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv

pytestmark = pytest.mark.gpu
OK, BAD, NO_PAGES = sv.SV_OK, sv.SV_ERR_BAD_INPUT, sv.SV_ERR_NO_PAGES


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def pages(n, ps):
    return -(-n // ps)


def fork(src, tgt, lens, counts, table, stack, free, shares, ps):
    """The call, fork by fork."""
    B, mp = table.shape
    n_pages = len(stack)
    pool = 0 <= free <= n_pages
    table, out_shares, out = table.copy(), np.maximum(shares, 0), counts.copy()
    owner, copies, status, asked, taken = {}, [], [], 0, 0
    for f, t in enumerate(tgt):
        if 0 <= t < B:
            owner.setdefault(t, f)
    old = table.copy()
    for f, (s, t, n) in enumerate(zip(src, tgt, lens)):
        copies.append([-1, -1, 0])
        if not (0 <= s < B and 0 <= t < B and s != t and n >= 0 and counts[t] == 0 and owner[t] == f
                and pages(n, ps) <= counts[s] <= mp):
            status.append(BAD)
            continue
        full, part = divmod(n, ps)
        asked += part > 0
        if part and not (pool and asked <= free):
            status.append(NO_PAGES if pool else BAD)
            continue
        status.append(OK)
        out[t] = pages(n, ps)
        for j in range(full):
            p = table[t, j] = old[s, j]
            if 0 <= p < n_pages:
                out_shares[p] += 1
            else:
                status[f] = BAD
        if part:
            taken = asked
            copies[f] = [old[s, full], stack[free - asked], part]
            table[t, full] = copies[f][1]
            if not (0 <= copies[f][0] < n_pages and 0 <= copies[f][1] < n_pages):
                status[f] = BAD
    return table, np.array(copies).reshape(-1, 3), out, free - taken, out_shares, status


def release(keep, counts, table, stack, free, shares, ps):
    B, mp = table.shape
    n_pages = len(stack)
    pool = 0 <= free <= n_pages
    stack, out, status, entries = list(stack), counts.copy(), [OK] * B, []
    for b in range(B):
        k = pages(keep[b], ps)
        if keep[b] < 0 or counts[b] < k or counts[b] > mp or (not pool and counts[b] > k):
            status[b] = BAD
            continue
        out[b] = k
        entries += [(b, table[b, j]) for j in range(k, counts[b])]
    times, last = {}, {}
    for i, (b, p) in enumerate(entries):
        times[p], last[p] = times.get(p, 0) + 1, i
    new = np.maximum(shares, 0)
    top = free
    for i, (b, p) in enumerate(entries):
        if not 0 <= p < n_pages:
            status[b] = BAD
            continue
        if shares[p] > 0:
            new[p] = max(0, shares[p] - times[p])
            if times[p] <= shares[p] or last[p] != i:
                continue
        if top < n_pages:
            stack[top] = p
            top += 1
        else:
            status[b] = BAD
    return stack, out, top, new, status


def run_fork(src, tgt, lens, counts, table, stack, free, shares, ps):
    want = fork(src, tgt, lens, counts, table, stack, free, shares, ps)
    t, st = i32(table), torch.full((len(src),), -7, dtype=torch.int32, device="cuda")
    got = sv.sv_fork_tables(i32(src), i32(tgt), i32(lens), i32(counts), t, i32(stack), i32([free]), i32(shares), ps,
                            fork_status=st)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(t.cpu().numpy(), want[0])
    for g, w, name in zip(got, (want[1], want[2], [want[3]], want[4]), ("copies", "counts", "free", "shares")):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    assert st.tolist() == want[5]
    return want, got


def run_release(keep, counts, table, stack, free, shares, ps):
    want = release(keep, counts, table, stack, free, shares, ps)
    s, st = i32(stack), torch.full((len(keep),), -7, dtype=torch.int32, device="cuda")
    got = sv.sv_release_shared_pages(i32(keep), i32(counts), i32(table), s, i32([free]), i32(shares), ps, seq_status=st)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(s.cpu().numpy(), want[0])
    for g, w, name in zip(got, (want[1], [want[2]], want[3]), ("counts", "free", "shares")):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    assert st.tolist() == want[4]
    return want, got


def pool(rng, lens, ps, spare, mp=None):
    held = pages(np.asarray(lens), ps)
    ids = rng.permutation(int(held.sum()) + spare)
    mp = int(held.max()) + 2 if mp is None else mp
    table = rng.integers(-9, -1, (len(lens), mp))
    table[np.arange(mp) < held[:, None]] = ids[:held.sum()]
    stack = np.full(len(ids), -3)
    stack[:spare] = ids[held.sum():]
    shares = np.zeros(len(ids), np.int64)
    shares[ids[:held.sum()]] = rng.integers(-1, 3, held.sum())
    return held, table, stack, shares


@pytest.mark.parametrize("B,F,past_hi,ps,share,seed", [
    (2, 1, 0, 16, 1.0, 1),
    (2, 1, 40, 16, 1.0, 2),
    (9, 8, 900, 16, 1.0, 3),
    (70, 64, 300, 8, 0.5, 4),          # the pool runs out half way
    (4096, 4000, 60, 16, 0.9, 5),      # the most sequences
    (5, 4, 200000, 16, 1.0, 6),        # long ones
    (700, 650, 500, 24, 1.0, 7),
    (40, 30, 77, 1, 1.0, 8),           # nothing to copy
])
def test_fork(B, F, past_hi, ps, share, seed):
    rng = np.random.default_rng(seed)
    order = rng.permutation(B)
    tgt, holders = order[:F], order[F:]
    lens = np.zeros(B, np.int64)
    lens[holders] = rng.integers(past_hi // 2, past_hi + 1, len(holders))
    src = rng.choice(holders, F)
    at = np.where(rng.random(F) < 0.3, rng.integers(0, lens[src] + 1), lens[src])
    need = int((at % ps != 0).sum())
    held, table, stack, shares = pool(rng, lens, ps, max(1, int(need * share)))
    run_fork(src, tgt, at, held, table, stack, max(1, int(need * share)), shares, ps)


def test_bad_forks():
    """Each kind of bad fork is reported and takes nothing; its neighbours are served."""
    rng = np.random.default_rng(11)
    ps = 16
    held, table, stack, shares = pool(rng, [50, 0, 33, 0, 0, 0, 0, 40, 0], ps, 6, mp=6)
    #      ok  taken ok  same too long neg  out of range     not empty  ok (bad page)  first of two, second
    src = [0, 0, 2, 3, 2, 0, 9, -1, 0, 0, 7, 0, 2]
    tgt = [1, 1, 3, 3, 4, 4, 5, 5, 9, 7, 6, 8, 8]
    lens = [50, 32, 33, 0, 49, -1, 3, 3, 3, 3, 40, 17, 17]
    table[7, 1] = 10 ** 6
    want, _ = run_fork(src, tgt, lens, held, table, stack, 6, shares, ps)
    assert want[5] == [OK, BAD, OK, BAD, BAD, BAD, BAD, BAD, BAD, BAD, BAD, OK, BAD]
    for free in (-1, len(stack) + 1):
        run_fork(src, tgt, lens, held, table, stack, free, shares, ps)
    held[0] = 9  # more pages than the table has
    run_fork(src, tgt, lens, held, table, stack, 6, shares, ps)


@pytest.mark.parametrize("B,g,past_hi,new_hi,ps,seed", [
    (1, 1, 0, 0, 16, 1),
    (1, 1, 500, 0, 16, 2),
    (8, 4, 900, 64, 16, 3),
    (100, 5, 3000, 300, 8, 4),
    (4096, 8, 100, 64, 16, 5),
    (3, 3, 200000, 1, 16, 6),
    (513, 2, 50, 50, 1, 7),
    (3000, 4, 300, 40, 8, 8),   # a table of more entries than one cluster takes
    (4096, 2, 40, 100, 8, 9),
])
def test_release_shared(B, g, past_hi, new_hi, ps, seed):
    rng = np.random.default_rng(seed)
    common = np.repeat(rng.integers(0, past_hi + 1, pages(B, g)), g)[:B] // ps
    held = pages(common * ps + rng.integers(0, new_hi + 1, B), ps)
    keep = np.where(rng.random(B) < 0.6, 0, held * ps - rng.integers(0, np.minimum(held * ps, 9) + 1))
    n_pages = int((held - common).sum() + common[::g].sum()) + 5
    ids = list(rng.permutation(n_pages))
    table, shares = rng.integers(-9, -1, (B, int(held.max()) + 1)), np.zeros(n_pages, np.int64)
    for b in range(B):
        if b % g == 0:
            first = [ids.pop() for _ in range(common[b])]
        shares[first] += b % g > 0
        table[b, :held[b]] = first + [ids.pop() for _ in range(held[b] - common[b])]
    stack = np.full(n_pages, -3)
    stack[:5] = ids
    run_release(keep, held, table, stack, 5, shares, ps)


def test_bad_releases():
    rng = np.random.default_rng(5)
    ps = 16
    held, table, stack, shares = pool(rng, [50, 33, 64, 20, 16, 90], ps, 4, mp=7)
    stack_free = 4
    shares[:] = 0
    keep = [10, -1, 80, 0, 16, 90]
    run_release(keep, held, table, stack, stack_free, shares, ps)
    table[0, 2] = -1
    table[3, 0] = 10 ** 6
    run_release(keep, held, table, stack, stack_free, shares, ps)
    table[0, 2] = table[0, 1]                     # one page twice: as many times on the stack
    run_release(keep, held, table, stack, len(stack) - 2, shares, ps)  # and too little room there
    for free in (-1, len(stack) + 1):
        run_release(keep, held, table, stack, free, shares, ps)
    held[5] = 8
    run_release(keep, held, table, stack, stack_free, shares, ps)


def test_a_page_given_back_more_often_than_it_is_shared():
    table = np.array([[0, 1], [0, 2], [0, 3], [0, 4]])
    want, _ = run_release([0, 0, 0, 0], np.array([2, 2, 2, 2]), table, np.full(8, -1), 0, np.array([1, 0, 0, 0, 0, 0, 0, 0]), 4)
    assert want[0][:5] == [1, 2, 3, 0, 4] and want[2] == 5


@pytest.mark.parametrize("hkv,ps", [(8, 16), (1, 8), (3, 384), (2, 1)])
def test_copy_pages(hkv, ps):
    rng = np.random.default_rng(hkv)
    n = 23
    planes = [torch.randint(0, 256, (n, hkv, ps, x), dtype=torch.uint8, device="cuda") for x in (64, 4, 256, 20, 48, 4096)]
    planes.append(torch.randn((n, hkv, ps, 2), device="cuda").to(torch.bfloat16))
    planes.append(torch.randn((n, hkv, ps, 128), device="cuda").to(torch.bfloat16))
    ids = rng.permutation(n)
    copies = [[ids[i], ids[i + 8], rng.integers(0, ps + 1)] for i in range(8)]
    copies += [[-1, -1, 5], [ids[0], n, 1], [-2, ids[17], 1], [ids[0], ids[18], ps + 1], [ids[1], ids[19], -1], [ids[2], ids[2], 1]]
    want = [p.clone() for p in planes]
    for a, b, m in copies[:8]:
        for w in want:
            w[b, :, :m] = w[a, :, :m].clone()
    st = torch.full((len(copies),), -7, dtype=torch.int32, device="cuda")
    sv.sv_copy_pages(i32(copies), planes, copy_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0] * 9 + [6] * 5
    for p, w in zip(planes, want):
        assert torch.equal(p.view(torch.uint8), w.view(torch.uint8))
