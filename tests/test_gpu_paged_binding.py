"""The paged-cache calls' two ways to the library -- the extension that takes
their plain form, and the interpreted checks that take the rest -- give the
same results, and what the extension does not take is refused by the other."""
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def tables():
    return dict(prefix_lens=i32([3, 0, 40]), new_lens=i32([2, 5, 30]), page_counts=i32([1, 0, 3]),
                block_table=i32([[4, -1, -1, -1, -1], [-1] * 5, [1, 0, 2, -1, -1]]),
                free_pages=i32([9, 8, 7, 6, 5, 3, -1, -1, -1, -1]), free_count=i32([6]), page_size=16, num_rows=40)


def cache():
    gen = torch.Generator(device="cuda").manual_seed(3)
    return [torch.randn((10, 2, 16, 64), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]


def spied(monkeypatch):
    """Whether the extension made the call."""
    real, seen = sv.api._native(), []

    class Spy:
        def __getattr__(self, name):
            def fn(*a):
                r = getattr(real, name)(*a)
                seen.append(r is not None)
                return r
            return fn
    monkeypatch.setattr(sv.api, "_native", lambda: Spy())
    return seen


def test_extension_is_built_and_bound():
    assert sv.api._native() is not None


def test_tables_both_ways(monkeypatch):
    seen, here = spied(monkeypatch), torch.cuda.current_stream()
    a, b = tables(), tables()
    sa, sb = i32([-7] * 3), i32([-7] * 3)
    ra = sv.sv_build_block_tables(**a, seq_status=sa)
    rb = sv.sv_build_block_tables(**b, seq_status=sb, stream=here)
    assert seen == [True]
    for x, y in zip([*ra, sa, a["block_table"]], [*rb, sb, b["block_table"]]):
        assert torch.equal(x, y)
    keep = i32([3, 2, 40])
    ga = sv.sv_release_pages(keep, ra[2], a["block_table"], a["free_pages"], ra[3], 16)
    gb = sv.sv_release_pages(keep, rb[2], b["block_table"], b["free_pages"], rb[3], 16, stream=here)
    assert seen == [True, True]
    for x, y in zip([*ga, a["free_pages"]], [*gb, b["free_pages"]]):
        assert torch.equal(x, y)


def test_rows_and_attention_both_ways(monkeypatch):
    seen, here = spied(monkeypatch), torch.cuda.current_stream()
    gen = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn((7, 8, 64), generator=gen, device="cuda").to(torch.bfloat16)
    slots = i32([5, 6, -1, 70, 16, 17, 18])
    (ka, va), (kb, vb) = cache(), cache()
    sv.sv_append_kv_paged(qkv[:, 4:6], qkv[:, 6:], slots, ka, va)
    sv.sv_append_kv_paged(qkv[:, 4:6], qkv[:, 6:], slots, kb, vb, stream=here)
    assert seen == [True] and torch.equal(ka, kb) and torch.equal(va, vb)
    args = (qkv[:, :4], ka, va, i32([[0, 1], [4, 2]]), i32([5, 20]), i32([0, 3, 7]))
    want = sv.sv_chunk_attention_paged(*args, window=9, return_lse=True, stream=here)
    got = sv.sv_chunk_attention_paged(*args, window=9, return_lse=True)
    out = sv.sv_chunk_attention_paged(*args, window=9)
    assert seen == [True] * 3
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(out, want[0])


def test_refusals_come_from_the_checks():
    a = tables()
    for name, bad in (("prefix_lens", i32([1, 2])), ("new_lens", torch.zeros(3, device="cuda")), ("page_size", -16),
                      ("free_count", torch.zeros(1, dtype=torch.int32)), ("num_rows", 0), ("page_counts", None),
                      ("block_table", a["block_table"].t())):
        with pytest.raises((TypeError, ValueError, sv.SpecVerifyError)):
            sv.sv_build_block_tables(**{**a, name: bad})
    k, v = cache()
    rows = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    for kn, vn, slots in ((rows, rows.half(), i32([0] * 4)), (rows[:, :1], rows, i32([0] * 4)), (rows, rows, i32([0] * 5)),
                          (rows.transpose(0, 1), rows, i32([0] * 4))):
        with pytest.raises((TypeError, ValueError)):
            sv.sv_append_kv_paged(kn, vn, slots, k, v)
    q, t, p, s = rows, i32([[0, 1]]), i32([4]), i32([0, 4])
    for kw in (dict(q=q[:, :, :32]), dict(q=q.float()), dict(block_table=t.long()), dict(prefix_lens=s),
               dict(row_starts=p), dict(window=-1), dict(window=1.5), dict(scale=0.0), dict(k_pages=k[:, :, :8]),
               dict(v_pages=v.transpose(2, 3)), dict(seq_status=s)):
        call = dict(q=q, k_pages=k, v_pages=v, block_table=t, prefix_lens=p, row_starts=s)
        with pytest.raises((TypeError, ValueError, sv.SpecVerifyError)):
            sv.sv_chunk_attention_paged(**{**call, **kw})
