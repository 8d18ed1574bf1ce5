"""Page tables, slot maps, pages given back and new K/V rows, on the GPU
against their definitions (all whole numbers or copied bits: equal, not close)."""
import numpy as np
import pytest
import torch

import pages_oracle as po
import speculative_decoding_verification_81_gb300 as sv
from speculative_decoding_verification_81_gb300 import workloads as W
from gpu_util import dev, host

pytestmark = pytest.mark.gpu
CODE = {"OK": sv.SV_OK, "NO_PAGES": sv.SV_ERR_NO_PAGES, "BAD_INPUT": sv.SV_ERR_BAD_INPUT}


def i32(a):
    return dev(np.asarray(a, np.int32))


def pool(rng, held, max_pages, spare):
    held = np.asarray(held)
    used = int(held.sum())
    ids = rng.permutation(used + spare)
    table = rng.integers(-5, 3, (len(held), max_pages))  # entries past the held ones: anything
    table[np.arange(max_pages) < held[:, None]] = ids[:used]
    stack = np.full(used + spare, -9)
    stack[:spare] = ids[used:]
    return table, stack, spare


def check_build(prefix, new, held, table, stack, free, page_size, num_rows, stream=None):
    want = po.build(prefix, new, held, table, stack, free, page_size, num_rows)
    t, st = i32(table), torch.full((len(held),), -7, dtype=torch.int32, device="cuda")
    fp = i32(stack)
    got = sv.sv_build_block_tables(i32(prefix), i32(new), i32(held), t, fp, i32([free]), page_size,
                                   num_rows, seq_status=st, stream=stream)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(t), want[0])
    for g, w, name in zip(got, (want[1], want[2], want[3], [want[4]]),
                          ("row_starts", "slot_map", "counts", "free")):
        np.testing.assert_array_equal(host(g), w, err_msg=name)
    assert host(st).tolist() == [CODE[s] for s in want[5]]
    np.testing.assert_array_equal(host(fp), stack)
    return want, got


@pytest.mark.parametrize("B,page_size,past_hi,new_hi,share,seed", [
    (1, 16, 0, 1, 1.0, 1),
    (1, 1, 5, 7, 1.0, 2),
    (8, 16, 4096, 9, 1.0, 3),
    (33, 8, 300, 40, 0.5, 4),       # the pool runs out half way
    (513, 128, 5000, 300, 0.9, 5),  # more sequences than threads
    (4096, 16, 200, 3, 0.97, 6),
    (7, 24, 100, 5000, 1.0, 7),     # many rows a sequence, an odd page size
    (40, 16, 0, 0, 1.0, 8),         # nothing new, nothing held
])
def test_build_tables(B, page_size, past_hi, new_hi, share, seed):
    rng = np.random.default_rng(seed)
    past = rng.integers(0, past_hi + 1, B)
    new = rng.integers(0, new_hi + 1, B)
    held = po.pages(past, page_size) + (rng.random(B) < 0.25)
    need = np.maximum(po.pages(past + new, page_size) - held, 0)
    max_pages = int(max(held.max(), po.pages(past + new, page_size).max())) + 1
    table, stack, free = pool(rng, held, max_pages, max(1, int(need.sum() * share)))
    check_build(past, new, held, table, stack, free, page_size, int(new.sum()) + 3)


def test_build_tables_bad_sequences():
    """Each kind of bad sequence is reported and takes nothing; its neighbours are served."""
    rng = np.random.default_rng(11)
    ps, mp = 16, 6
    #        ok  L<0  n<0  too long  held<prefix  held>max  ok   past the rows  held<0
    past = [20, -1, 30, 90, 40, 10, 0, 5, 0]
    new = [30, 4, -2, 7, 3, 2, 40, 60, 1]
    held = [2, 1, 2, 6, 2, 7, 0, 1, -1]
    table, stack, free = pool(rng, np.clip(held, 0, mp), mp, 12)
    want, _ = check_build(past, new, held, table, stack, free, ps, 100)
    assert want[5] == ["OK"] + ["BAD_INPUT"] * 5 + ["OK", "BAD_INPUT", "BAD_INPUT"]


def test_build_tables_bad_page_ids():
    rng = np.random.default_rng(12)
    past, new, held = [20, 20, 0], [20, 20, 40], [2, 2, 0]
    table, stack, free = pool(rng, held, 4, 8)
    table[1, 1] = len(stack)       # a held page that new rows fall into
    stack[free - 3] = -4           # the second page handed to sequence 2
    want, _ = check_build(past, new, held, table, stack, free, 16, 80)
    assert want[5] == ["OK", "BAD_INPUT", "BAD_INPUT"]


@pytest.mark.parametrize("free", [-1, 9])
def test_build_tables_bad_free_count(free):
    rng = np.random.default_rng(13)
    table, stack, _ = pool(rng, [1, 1], 4, 6)
    want, _ = check_build([5, 5], [2, 30], [1, 1], table, stack, free, 16, 32)
    assert want[5] == ["OK", "BAD_INPUT"] and want[4] == free


def test_build_tables_lengths_past_32_bits():
    """Row counts whose sum passes 2^31: the later sequences are refused, nothing wraps."""
    ps = 1 << 20
    past, new = [0] * 6, [(1 << 29) + 1] * 6
    held = [0] * 6
    table = np.full((6, 600), -1)
    stack = np.arange(1500)
    check_build(past, new, held, table, stack, 1500, ps, 64)


@pytest.mark.parametrize("B,page_size,past_hi,tail_hi,seed", [
    (1, 16, 40, 64, 1), (8, 16, 4096, 64, 2), (600, 8, 300, 90, 3), (4096, 32, 64, 64, 4), (5, 1, 30, 9, 5),
])
def test_release_pages(B, page_size, past_hi, tail_hi, seed):
    rng = np.random.default_rng(seed)
    keep = rng.integers(0, past_hi + 1, B)
    keep[rng.random(B) < 0.2] = 0  # sequences that end
    held = po.pages(keep + rng.integers(0, tail_hi + 1, B), page_size)
    table, stack, free = pool(rng, held, max(1, int(held.max())), 5)
    want = po.release(keep, held, table, stack, free, page_size)
    st = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    fp, t = i32(stack), i32(table)
    counts, left = sv.sv_release_pages(i32(keep), i32(held), t, fp, i32([free]), page_size, seq_status=st)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(fp), want[0])
    np.testing.assert_array_equal(host(counts), want[1])
    assert host(left).tolist() == [want[2]]
    assert host(st).tolist() == [CODE[s] for s in want[3]]
    np.testing.assert_array_equal(host(t), table)


@pytest.mark.parametrize("free", [4, 9, 13, -2, 40])
def test_release_pages_refusals(free):
    """Bad lengths, and a stack with too little room (a page in two tables)."""
    keep, held = [10, -1, 40, 0, 5, 0], [3, 2, 2, 4, 7, 0]
    table = np.arange(36).reshape(6, 6) % 17
    stack = np.arange(17)
    want = po.release(keep, held, table, stack, free, 16)
    st = torch.full((6,), -7, dtype=torch.int32, device="cuda")
    fp = i32(stack)
    counts, left = sv.sv_release_pages(i32(keep), i32(held), i32(table), fp, i32([free]), 16, seq_status=st)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(fp), want[0])
    np.testing.assert_array_equal(host(counts), want[1])
    assert host(left).tolist() == [want[2]]
    assert host(st).tolist() == [CODE[s] for s in want[3]]


@pytest.mark.parametrize("rows,hkv,d,page_size,wide,strided,seed", [
    (1, 1, 8, 1, False, False, 1), (32, 8, 128, 16, True, False, 2), (37, 5, 80, 8, False, True, 3),
    (1000, 2, 64, 128, True, True, 4), (3, 8, 256, 24, False, False, 5), (2, 40, 256, 16, True, False, 6),
])
def test_append_rows(rows, hkv, d, page_size, wide, strided, seed):
    rng = np.random.default_rng(seed)
    num_pages = rows // page_size + 3
    slots = rng.permutation(num_pages * page_size)[:rows]
    slots[rng.random(rows) < 0.2] = -1
    if rows > 2:
        slots[1] = num_pages * page_size  # past the last page
        slots[2] = -2
    wk = rng.standard_normal((rows, (3 if strided else 1) * hkv, d)).astype(np.float32)
    wv = rng.standard_normal((rows, (3 if strided else 1) * hkv, d)).astype(np.float32)
    if wide:
        wk[0, 0, :3] = [np.inf, -np.inf, 1 + 2.0 ** -8]  # the last: a tie, to even
    k0 = rng.integers(0, 1 << 15, (num_pages, hkv, page_size, d)).astype(np.uint16)
    v0 = rng.integers(0, 1 << 15, (num_pages, hkv, page_size, d)).astype(np.uint16)
    src_k, src_v = (wk, wv) if wide else (W.f32_to_bf16_bits(wk), W.f32_to_bf16_bits(wv))
    cut = (lambda t: t[:, hkv:2 * hkv]) if strided else (lambda t: t)
    want_k, want_v = k0.copy(), v0.copy()
    for r, s in enumerate(slots):
        if 0 <= s < num_pages * page_size:
            want_k[s // page_size, :, s % page_size] = cut(W.f32_to_bf16_bits(wk))[r]
            want_v[s // page_size, :, s % page_size] = cut(W.f32_to_bf16_bits(wv))[r]
    kd, vd = dev(k0), dev(v0)
    st = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    sv.sv_append_kv_paged(cut(dev(src_k)), cut(dev(src_v)), i32(slots), kd, vd, row_status=st)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(host(kd), want_k)
    np.testing.assert_array_equal(host(vd), want_v)
    bad = (slots < -1) | (slots >= num_pages * page_size)
    np.testing.assert_array_equal(host(st), np.where(bad, sv.SV_ERR_BAD_INPUT, sv.SV_OK))


def test_append_past_32_bits():
    """Slots at the end of a pool of more than 2^32 elements."""
    hkv, ps, d = 8, 16, 128
    num_pages = (1 << 25) // (hkv * ps) + 3
    k = torch.empty((num_pages, hkv, ps, d), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k[-2:], v[-2:] = 0, 0
    rows = torch.randn((5, hkv, d), device="cuda").to(torch.bfloat16)
    slots = [num_pages * ps - 1, (num_pages - 1) * ps, num_pages * ps - 5, (num_pages - 2) * ps + 3, -1]
    sv.sv_append_kv_paged(rows, rows * 2, i32(slots), k, v)
    torch.cuda.synchronize()
    for r, s in enumerate(slots[:4]):
        assert torch.equal(k[s // ps, :, s % ps], rows[r]) and torch.equal(v[s // ps, :, s % ps], rows[r] * 2)
    assert (k[-2:] != 0).any(-1).sum() == 4 * hkv


def test_tables_across_steps_keep_every_page_once():
    """Build, shorten and give back over many steps: the pages in the tables
    and on the stack are always the whole pool, each once."""
    rng = np.random.default_rng(21)
    B, ps, mp, num_pages = 19, 8, 12, 150
    held, past = np.zeros(B, np.int64), np.zeros(B, np.int64)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    stack, free = i32(rng.permutation(num_pages)), i32([num_pages])
    counts = i32(held)
    for _ in range(25):
        new = rng.integers(0, 20, B)
        new = np.minimum(new, mp * ps - past)
        st = torch.empty(B, dtype=torch.int32, device="cuda")
        starts, slots, counts, free = sv.sv_build_block_tables(i32(past), i32(new), counts, table, stack, free,
                                                               ps, int(new.sum()) + 1, seq_status=st)
        served = host(st) == sv.SV_OK
        s = host(slots)
        assert len(set(s[s >= 0])) == (s >= 0).sum()
        past = np.where(served, past + rng.integers(0, 20, B) % (new + 1), past)
        past[rng.random(B) < 0.1] = 0
        counts, free = sv.sv_release_pages(i32(past), counts, table, stack, free, ps, seq_status=st)
        assert (host(st) == sv.SV_OK).all()
        c, t, f = host(counts), host(table), int(host(free)[0])
        np.testing.assert_array_equal(c, po.pages(past, ps))
        ids = np.concatenate([t[b, :c[b]] for b in range(B)] + [host(stack)[:f]])
        np.testing.assert_array_equal(np.sort(ids), np.arange(num_pages))


def test_tables_captured_and_on_another_stream():
    rng = np.random.default_rng(22)
    past, new = rng.integers(0, 200, 20), rng.integers(0, 30, 20)
    held = po.pages(past, 16)
    table, stack, free = pool(rng, held, 20, 60)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        t, args = i32(table), [i32(past), i32(new), i32(held)]
        fp, fc = i32(stack), i32([free])
        rows = int(new.sum()) + 2
    s.synchronize()
    _, want = check_build(past, new, held, table, stack, free, 16, rows, stream=s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = sv.sv_build_block_tables(*args, t, fp, fc, 16, rows)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        np.testing.assert_array_equal(host(a), host(b))


def test_tables_from_two_threads_at_once():
    """Calls whose shared memory is past the default limit by different amounts, from two host threads."""
    import threading
    failed = []

    def calls(B):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                past = torch.arange(B, dtype=torch.int32, device="cuda") % 5
                new, held = torch.ones_like(past), (past + 3) // 4
                table = torch.zeros(B, 2, dtype=torch.int32, device="cuda")
                stack = torch.arange(B, dtype=torch.int32, device="cuda")
                free = torch.tensor([B], dtype=torch.int32, device="cuda")
            for _ in range(200):
                r = sv.sv_build_block_tables(past, new, held, table, stack, free, 4, B, stream=stream)
            stream.synchronize()
            need = ((torch.arange(B) % 5 + 4) // 4 - (torch.arange(B) % 5 + 3) // 4).sum().item()
            assert host(r[3])[0] == B - need
        except Exception as e:
            failed.append(e)
    threads = [threading.Thread(target=calls, args=(B,)) for B in (4096, 2100)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
