"""Refusals of the attention and cache calls: every invalid argument gives its status before any HIP call, and the
binding refuses tensors that do not fit."""

import math

import pytest
import torch

from quantized_weight_linear_amd import nq

A, MIS = 0x10000, 0x10002       # fake device addresses, never followed: aligned, misaligned


@pytest.fixture(scope="module")
def L():
    return nq.lib()


def changed(f, good, changes):
    for name, value, status in changes:
        args = dict(good)
        assert name in args
        args[name] = value
        assert f(*args.values()) == status, (name, value)


def test_prompt_refusals(L):
    good = dict(q=A, qs=1536, k=A, ks=256, v=A, vs=256, cu_q=A, cu_k=A, B=2, Tq=9, Tk=9, Hq=6, Hkv=1, D=256, scale=0.1, out=0,
                o=A, lse=None, stream=None)
    S, N, R, AL = nq.NQ_ERR_SHAPE, nq.NQ_ERR_NULL, nq.NQ_ERR_RANGE, nq.NQ_ERR_ALIGN
    changed(L.nq_attn_prompt, good, [
        ("D", 96, S), ("D", 512, S), ("Hkv", 4, S),
        ("Hkv", 0, S), ("Hq", 0, S), ("B", -1, S), ("Tq", -1, S), ("Tk", -1, S), ("qs", 1528, S), ("qs", 1537, S), ("ks", 255, S),
        ("vs", 248, S), ("qs", 1 << 24, S), ("Tq", 1 << 31, S), ("out", 2, nq.NQ_ERR_FORMAT), ("scale", 0.0, R),
        ("scale", -1.0, R), ("scale", math.inf, R), ("scale", math.nan, R), ("q", None, N), ("k", None, N), ("v", None, N),
        ("cu_q", None, N), ("cu_k", None, N), ("o", None, N), ("q", MIS, AL), ("k", MIS, AL), ("o", MIS, AL), ("lse", MIS, AL),
        ("cu_k", MIS, AL)])
    assert L.nq_attn_prompt(*dict(good, Tq=0, q=None, o=None).values()) == nq.NQ_OK
    assert L.nq_attn_prompt(*dict(good, B=0, cu_q=None).values()) == nq.NQ_OK


def test_tree_refusals(L):
    good = dict(fmt=1, q=A, qs=1536, kp=A, vp=A, ks=A, vs=A, table=A, width=8, lens=A, cu=A, mask=A, B=2, max_q=4, T=6, Hq=6,
                Hkv=1, D=256, page=64, pages=9, max_len=100, scale=0.1, out=1, o=A, lse=A, ws=None, wb=0, stream=None)
    S, N, AL = nq.NQ_ERR_SHAPE, nq.NQ_ERR_NULL, nq.NQ_ERR_ALIGN
    changed(L.nq_attn_tree, good, [
        ("fmt", 2, nq.NQ_ERR_FORMAT), ("out", 5, nq.NQ_ERR_FORMAT), ("max_q", 0, S), ("max_q", 65, S), ("page", 8, S),
        ("page", 48, S), ("page", 8192, S), ("width", -1, S), ("width", 1 << 25, S), ("pages", -1, S), ("max_len", -1, S),
        ("wb", -1, S), ("D", 32, S), ("Hkv", 4, S), ("qs", 1000, S), ("T", -1, S), ("B", -1, S), ("scale", 0.0, nq.NQ_ERR_RANGE),
        ("q", None, N), ("kp", None, N), ("vp", None, N), ("ks", None, N), ("vs", None, N), ("table", None, N), ("lens", None, N),
        ("cu", None, N), ("mask", None, N), ("o", None, N), ("kp", MIS, AL), ("table", MIS, AL), ("ws", MIS, AL), ("lse", MIS, AL)])
    assert L.nq_attn_tree(*dict(good, T=0, q=None).values()) == nq.NQ_OK
    a = dict(good, T=3, B=0)
    assert L.nq_attn_tree(*a.values()) == nq.NQ_OK
    assert L.nq_attn_tree_workspace_bytes(1, 0, 6, 1, 256, 100) == 0
    assert L.nq_attn_tree_workspace_bytes(1, 1, 6, 1, 256, 1) == 0            # nothing to split
    assert L.nq_attn_tree_workspace_bytes(1, 1, 24, 4, 256, 100000) > 0


def test_cache_refusals(L):
    S, N, AL, F = nq.NQ_ERR_SHAPE, nq.NQ_ERR_NULL, nq.NQ_ERR_ALIGN, nq.NQ_ERR_FORMAT
    good = dict(fmt=1, k=A, ks=256, v=A, vs=256, k_scale=A, v_scale=A, table=A, width=8, lens=A, cu=A, B=2, T=5, Hkv=1, D=256,
                page=64, pages=9, kp=A, vp=A, stream=None)
    changed(L.nq_kv_append, good, [
        ("fmt", -1, F), ("T", -1, S), ("D", 100, S), ("Hkv", 0, S), ("ks", 200, S), ("page", 63, S), ("k", None, N), ("v", None, N),
        ("k_scale", None, N), ("v_scale", None, N), ("table", None, N), ("lens", None, N), ("cu", None, N), ("kp", None, N),
        ("vp", None, N), ("k", MIS, AL), ("vp", MIS, AL)])
    assert L.nq_kv_append(*dict(good, T=0, k=None).values()) == nq.NQ_OK
    good = dict(refs=A, pages=9, table=A, width=8, lens=A, new=A, B=2, page=16, free=A, short=A, stream=None)
    changed(L.nq_kv_reserve, good, [
        ("B", 8193, S), ("B", -1, S), ("page", 15, S), ("pages", -1, S), ("refs", None, N), ("table", None, N), ("lens", None, N),
        ("new", None, N), ("free", None, N), ("short", None, N), ("short", MIS, AL)])
    good = dict(refs=A, pages=9, table=A, width=8, keep=A, B=2, page=16, stream=None)
    changed(L.nq_kv_release, good, [("page", 0, S), ("width", -1, S), ("refs", None, N), ("table", None, N), ("keep", None, N),
                                    ("table", MIS, AL)])
    assert L.nq_kv_release(*dict(good, B=0, table=None).values()) == nq.NQ_OK
    good = dict(refs=A, pages=9, table=A, width=8, lens=A, B=2, parents=A, children=3, page=16, child=A, copies=A, free=A, short=A,
                stream=None)
    changed(L.nq_kv_fork, good, [("children", -1, S), ("page", 24, S), ("refs", None, N), ("table", None, N), ("lens", None, N),
                                 ("parents", None, N), ("child", None, N), ("copies", None, N), ("free", None, N),
                                 ("short", None, N), ("copies", MIS, AL)])
    assert L.nq_kv_fork(*dict(good, children=0, parents=None).values()) == nq.NQ_OK
    good = dict(pool=A, planes=2, plane_bytes=9 * 4096, page_bytes=4096, pages=9, copies=A, n=3, stream=None)
    changed(L.nq_kv_copy_pages, good, [("planes", -1, S), ("planes", 65536, S), ("page_bytes", 4104, S), ("plane_bytes", 8 * 4096, S),
                                       ("n", -1, S), ("pool", None, N), ("copies", None, N), ("pool", MIS, AL)])
    assert L.nq_kv_copy_pages(*dict(good, n=0, copies=None).values()) == nq.NQ_OK
    good = dict(pool=A, planes=2, plane_bytes=9 * 16 * 512, Hkv=1, page=16, row=512, pages=9, table=A, width=8, lens=A, accept=A,
                cu=A, B=2, accepted=4, stream=None)
    changed(L.nq_kv_compact, good, [("row", 520, S), ("row", 8, S), ("row", 1024, S), ("Hkv", 0, S), ("plane_bytes", 16, S),
                                    ("accepted", -1, S), ("page", 20, S), ("pool", None, N), ("table", None, N), ("lens", None, N),
                                    ("accept", None, N), ("cu", None, N), ("pool", MIS, AL)])
    assert L.nq_kv_compact(*dict(good, accepted=0, accept=None).values()) == nq.NQ_OK


@pytest.mark.parametrize("width", [1 << 27, 1 << 57, 1 << 59, (1 << 63) - 1])
def test_tables_beyond_all_sizes(L, width):
    """Widths whose product with the page size passes 2^30 tokens, 64 bits included."""
    S = nq.NQ_ERR_SHAPE
    assert L.nq_kv_release(A, 9, A, width, A, 2, 16, None) == S
    assert L.nq_kv_reserve(A, 9, A, width, A, A, 2, 16, A, A, None) == S
    assert L.nq_attn_tree(0, A, 1536, A, A, None, None, A, width, A, A, A, 2, 4, 6, 6, 1, 256, 32, 9, 100, 0.1, 1, A, None, None, 0,
                          None) == S
    assert L.nq_kv_copy_pages(A, 2, 9 * 4096, 4096, 9, A, width << 4 & (1 << 63) - 1 | 1 << 47, None) == S


def test_binding_refuses_tensors_that_do_not_fit():
    q, k = torch.zeros((4, 6, 64), dtype=torch.bfloat16), torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cu, o = torch.tensor([0, 4], dtype=torch.int32), torch.zeros((4, 6, 64))
    bad = [
        lambda: nq.nq_attn_prompt(q.float(), k, k, cu, cu, 0.1, o),
        lambda: nq.nq_attn_prompt(q, k.transpose(0, 1).contiguous().transpose(0, 1), k, cu, cu, 0.1, o),   # heads apart
        lambda: nq.nq_attn_prompt(q, k, k[:3], cu, cu, 0.1, o),
        lambda: nq.nq_attn_prompt(q, k, k, cu.long(), cu, 0.1, o),
        lambda: nq.nq_attn_prompt(q, k, k, cu, cu[:1], 0.1, o),
        lambda: nq.nq_attn_prompt(q, k, k, cu, cu, 0.1, o[:3]),
        lambda: nq.nq_attn_prompt(q, k, k, cu, cu, 0.1, o, torch.zeros((4, 5))),
        lambda: nq.nq_attn_prompt(q, k, k, cu, cu, 0.1, o, torch.zeros((4, 6), dtype=torch.float64)),
    ]
    pages = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    table, lens, mask = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)

    def tree(fmt=nq.NQ_KV_BF16, kp=pages, vp=pages, table=table, lens=lens, mask=mask, o=o):
        nq.nq_attn_tree(fmt, q, kp, vp, None, None, table, lens, cu, mask, 4, 10, 0.1, o)

    bad += [lambda: tree(fmt=nq.NQ_KV_E4M3), lambda: tree(vp=pages[:2]), lambda: tree(kp=pages.view(3, 2, 64, 16)),
            lambda: tree(table=table.long()), lambda: tree(table=table[0]), lambda: tree(lens=lens[:0]),
            lambda: tree(mask=mask[:3]), lambda: tree(mask=mask.int()), lambda: tree(o=o[:2]),
            lambda: nq.nq_kv_copy_pages(pages, table), lambda: nq.nq_kv_copy_pages(pages[None], table.float()),
            lambda: nq.nq_kv_fork(lens, table, lens, lens, 16, table[:, :1].contiguous(), table, lens, lens),
            lambda: nq.nq_kv_reserve(lens, table, lens[:0], lens, 16, lens, lens)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(nq.NQError) as e:
        nq.nq_attn_prompt(q, k, k, cu, cu, 0.0, o)
    assert e.value.status == nq.NQ_ERR_RANGE


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the addresses are not real: a launch has to fail")
def test_small_arrays_need_no_more_than_their_elements_alignment(L):
    """Scales, offsets, lengths, tables, counts and pairs at 4 bytes, masks at 8: the checks pass, the launch fails."""
    S4, S8, HIP = A + 4, A + 8, nq.NQ_ERR_HIP
    for x in (S4, S8, A + 12):
        assert L.nq_attn_prompt(A, 1536, A, 256, A, 256, x, x, 2, 9, 9, 6, 1, 256, 0.1, 0, A, x, None) == HIP
        assert L.nq_kv_append(1, A, 256, A, 256, x, x, x, 8, x, x, 2, 5, 1, 256, 64, 9, A, A, None) == HIP
        assert L.nq_attn_tree(1, A, 1536, A, A, x, x, x, 8, x, x, S8, 2, 4, 6, 6, 1, 256, 64, 9, 100, 0.1, 1, A, x, None, 0,
                              None) == HIP
        assert L.nq_kv_reserve(x, 9, x, 8, x, x, 2, 16, x, x, None) == HIP
        assert L.nq_kv_release(x, 9, x, 8, x, 2, 16, None) == HIP
        assert L.nq_kv_fork(x, 9, x, 8, x, 2, x, 3, 16, x, x, x, x, None) == HIP
        assert L.nq_kv_copy_pages(A, 2, 9 * 4096, 4096, 9, x, 3, None) == HIP
        assert L.nq_kv_compact(A, 2, 9 * 16 * 512, 1, 16, 512, 9, x, 8, x, x, x, 2, 4, None) == HIP
    assert L.nq_attn_tree(1, A, 1536, A, A, A, A, A, 8, A, A, S4, 2, 4, 6, 6, 1, 256, 64, 9, 100, 0.1, 1, A, A, None, 0,
                          None) == nq.NQ_ERR_ALIGN


@pytest.mark.parametrize("hq,hkv,d", [(24, 4, 256), (32, 8, 128), (40, 8, 128), (8, 1, 256), (14, 2, 64), (20, 20, 64), (128, 1, 64)])
def test_tree_workspace_of_the_largest_call_serves_smaller_ones(L, hq, hkv, d):
    """The size never falls as the batch, the drafted tokens or the length grow."""
    size = lambda b, q, n: L.nq_attn_tree_workspace_bytes(b, q, hq, hkv, d, n)  # noqa: E731
    batches, lengths = (1, 2, 5, 16, 31, 32, 33, 64, 65, 129, 300), (0, 700, 769, 3000, 32768, 131000, 1 << 20)
    for n in lengths:
        for b in batches:
            sizes = [size(b, q, n) for q in range(1, 65)]
            assert sizes == sorted(sizes)
    for q in (1, 4, 17, 33, 64):
        for n in lengths:
            sizes = [size(b, q, n) for b in batches]
            assert sizes == sorted(sizes)
        for b in batches:
            sizes = [size(b, q, n) for n in lengths]
            assert sizes == sorted(sizes)


@pytest.mark.parametrize("name", ["B", "Tq", "Tk"])
def test_prompt_sizes_near_32_bits(L, name):
    """Sizes whose last tile, or last look through the sequences, would pass 32 bits."""
    good = dict(q=A, qs=64, k=A, ks=64, v=A, vs=64, cu_q=A, cu_k=A, B=1, Tq=1, Tk=1, Hq=1, Hkv=1, D=64, scale=0.1, out=0, o=A, lse=None,
                stream=None)
    for n in ((1 << 31) - 1, (1 << 31) - 1023):
        assert L.nq_attn_prompt(*dict(good, **{name: n}).values()) == nq.NQ_ERR_SHAPE


@pytest.mark.parametrize("b", [1, 5, 300, 100000])
def test_tree_lengths_beyond_all_tables(L, b):
    """A length above what a table can hold (2^30 tokens) asks for the workspace of that, not for less."""
    top = L.nq_attn_tree_workspace_bytes(b, 4, 24, 4, 256, 1 << 30)
    assert top > 0
    for n in ((1 << 30) + 1, 1 << 40, 1 << 57, 1 << 62, (1 << 63) - 1):
        assert L.nq_attn_tree_workspace_bytes(b, 4, 24, 4, 256, n) == top
