"""Refusals of the norm, the block-scaled FP8 product, the rotated append and the cache with a scale a row: every invalid
argument gives its status before any HIP call, and the binding refuses tensors that do not fit."""

import math

import pytest
import torch

from quantized_weight_linear_amd import nq

A, MIS = 0x10000, 0x10002       # fake device addresses, never followed: aligned, misaligned
S, N, AL, F, R, HIP = (nq.NQ_ERR_SHAPE, nq.NQ_ERR_NULL, nq.NQ_ERR_ALIGN, nq.NQ_ERR_FORMAT, nq.NQ_ERR_RANGE, nq.NQ_ERR_HIP)
no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the addresses are not real: a launch has to fail")


@pytest.fixture(scope="module")
def L():
    return nq.lib()


def changed(f, good, changes):
    for name, value, status in changes:
        assert name in good
        assert f(*dict(good, **{name: value}).values()) == status, (name, value)


NORM = dict(fmt=2, x=A, xs=5120, res=A, res_out=A, w=A, bias=1.0, eps=1e-6, T=3, K=5120, y=A, scale=A, stream=None)


def test_norm_refusals(L):
    f = L.nq_rmsnorm
    changed(f, NORM, [("fmt", 3, F), ("fmt", -1, F), ("T", -1, S), ("T", 1 << 24, S), ("K", -16, S), ("K", 5112, S), ("K", 32784, S),
                      ("xs", 5112, S), ("xs", 5124, S), ("xs", 1 << 24, S), ("eps", 0.0, R), ("eps", -1.0, R), ("eps", math.nan, R),
                      ("eps", math.inf, R), ("x", None, N), ("y", None, N), ("scale", None, N), ("res_out", None, N), ("x", MIS, AL),
                      ("res", MIS, AL), ("res_out", MIS, AL), ("w", MIS, AL), ("y", MIS, AL), ("scale", MIS, AL), ("y", A + 8, AL)])
    assert f(*dict(NORM, fmt=1, K=5104, xs=5104).values()) == S       # groups of 64
    for fmt in (0, 1, 2):                                             # more threads than a launch has
        assert f(*dict(NORM, fmt=fmt, T=1 << 22, K=6208, xs=6208).values()) == S
    assert f(*dict(NORM, fmt=0, K=5116, xs=5120).values()) == S       # 16-byte pieces
    assert f(*dict(NORM, T=0, x=None, y=None).values()) == nq.NQ_OK
    assert f(*dict(NORM, K=0, x=None, y=None).values()) == nq.NQ_OK


QUANT = dict(x=A, T=3, K=5120, codes=A, scale=A, stream=None)


def test_quantizer_refusals(L):
    changed(L.nq_quantize_act_fp8_b128, QUANT, [("T", -1, S), ("K", -16, S), ("K", 5128, S), ("T", 1 << 31, S), ("T", 1 << 24, S),
                                                ("K", 1 << 31, S), ("x", None, N), ("codes", None, N), ("scale", None, N), ("x", MIS, AL),
                                                ("codes", MIS, AL), ("scale", MIS, AL)])
    assert L.nq_quantize_act_fp8_b128(*dict(QUANT, T=0, x=None).values()) == nq.NQ_OK


PRODUCT = dict(a=A, a_scale=A, w=A, wsi=A, M=33, N=300, K=1040, gr=3, gc=9, out=1, y=A, ws=None, wb=0, stream=None)


def test_product_refusals(L):
    f = L.nq_gemm_fp8_b128
    changed(f, PRODUCT, [("M", -1, S), ("N", -1, S), ("K", -16, S), ("K", 1048, S), ("K", 1 << 20, S), ("M", 1 << 31, S), ("N", 1 << 31, S),
                         ("gr", 2, S), ("gr", 4, S), ("gc", 8, S), ("gc", 10, S), ("wb", -1, S), ("out", 2, F), ("a", None, N),
                         ("a_scale", None, N), ("w", None, N), ("wsi", None, N), ("y", None, N), ("a", MIS, AL), ("w", A + 8, AL),
                         ("a_scale", MIS, AL), ("wsi", MIS, AL), ("y", MIS, AL), ("ws", A + 4, AL)])
    for m, n in ((1, 1 << 28), (64, 1 << 28), (1 << 29, 1 << 29), (1 << 17, 1 << 19), ((1 << 31) - 1024, (1 << 31) - 1024)):
        assert f(*dict(PRODUCT, M=m, N=n, gr=-(-n // 128)).values()) == S          # more tiles than a launch has
        assert L.nq_gemm_fp8_b128_workspace_bytes(m, n, 1040) == 0
    assert f(*dict(PRODUCT, M=0, a=None, y=None).values()) == nq.NQ_OK
    assert f(*dict(PRODUCT, N=0, gr=0, w=None, y=None).values()) == nq.NQ_OK
    for m, n, k in ((0, 10, 16), (10, 0, 16), (-1, 10, 16), (10, 10, 8), (1, 1, 0)):
        assert L.nq_gemm_fp8_b128_workspace_bytes(m, n, k) == 0


@pytest.mark.parametrize("n,k", [(5120, 5120), (5120, 17408), (17408, 5120), (256, 7168), (1024, 5136), (1, 20000), (100, 1040), (300, 900)])
def test_product_workspace_serves_smaller_products(L, n, k):
    """What is asked for at M is enough for every smaller M."""
    f, most = L.nq_gemm_fp8_b128_workspace_bytes, 0
    for m in [*range(1, 1200), *range(1200, 9000, 61), 20000, 70001, 1 << 20]:
        need = f(m, n, k)
        assert need >= most, (m, n, k)
        most = need
    assert most == 0 or k > 7 * 128             # fewer than eight blocks of K are never split


@no_gpu
def test_limits_of_quantizer_and_product(L):
    """The largest sizes that the header allows reach the launch, the next ones are refused."""
    for t, k, status in (((1 << 28) - 1, 16, HIP), (1 << 28, 16, S), (1, (1 << 31) - 16, HIP), (1 << 24, 2048, S), ((1 << 24) - 1, 2048, HIP)):
        assert L.nq_quantize_act_fp8_b128(*dict(QUANT, T=t, K=k).values()) == status, (t, k)
    top = (1 << 31) - 1024
    for m, n, status in ((top, 1, S), (1 << 30, 1, S), ((1 << 30) - 64, 1, HIP), (1, (1 << 28) - 16, HIP), (1, (1 << 28) - 15, S), (65, (1 << 29) - 64, HIP),
                         (65, 1 << 29, S), (64, (1 << 28) - 16, HIP), (2, top + 1, S)):
        assert L.nq_gemm_fp8_b128(*dict(PRODUCT, M=m, N=n, gr=-(-n // 128)).values()) == status, (m, n)


ROPE = dict(fmt=3, q=A, qs=1536, k=A, ks=256, v=A, vs=256, qw=A, kw=A, bias=0.0, eps=1e-6, pos=A, freq=A, rot=64, rope=0, ksc=A, vsc=A,
            table=A, width=8, lens=A, cu=A, B=2, T=5, Hq=6, Hkv=1, D=256, page=64, pages=9, qo=A, qos=1536, ko=None, kos=0, kp=A, vp=A,
            stream=None)


def test_rope_refusals(L):
    f = L.nq_kv_append_rope
    changed(f, ROPE, [("fmt", 2, F), ("fmt", 4, F), ("fmt", -1, F), ("rope", 2, F), ("rope", -1, F), ("rot", -16, S), ("rot", 8, S),
                      ("rot", 72, S), ("rot", 272, S), ("T", -1, S), ("T", 1 << 24, S), ("B", -1, S), ("D", 96, S), ("Hkv", 4, S),
                      ("page", 48, S), ("page", 8, S), ("width", 1 << 25, S), ("pages", -1, S), ("qs", 1528, S), ("ks", 248, S),
                      ("vs", 260, S), ("qos", 1528, S), ("eps", 0.0, R), ("eps", math.nan, R), ("k", None, N), ("v", None, N),
                      ("qo", None, N), ("pos", None, N), ("freq", None, N), ("ksc", None, N), ("vsc", None, N), ("table", None, N),
                      ("lens", None, N), ("cu", None, N), ("kp", None, N), ("vp", None, N), ("q", MIS, AL), ("k", MIS, AL),
                      ("qo", MIS, AL), ("kp", MIS, AL), ("qw", MIS, AL), ("kw", A + 8, AL), ("pos", MIS, AL), ("freq", MIS, AL),
                      ("ksc", MIS, AL), ("lens", MIS, AL)])
    assert f(*dict(ROPE, ko=A, kos=248).values()) == S
    assert f(*dict(ROPE, ko=MIS, kos=256).values()) == AL
    assert f(*dict(ROPE, T=0, k=None).values()) == nq.NQ_OK
    assert f(*dict(ROPE, B=0, cu=None).values()) == nq.NQ_OK


def test_tree_and_compact_with_a_scale_a_row(L):
    tree = dict(fmt=3, q=A, qs=1536, kp=A, vp=A, ks=A, vs=A, table=A, width=8, lens=A, cu=A, mask=A, B=2, max_q=4, T=6, Hq=6, Hkv=1,
                D=256, page=64, pages=9, max_len=100, scale=0.1, out=1, o=A, lse=A, ws=None, wb=0, stream=None)
    changed(L.nq_attn_tree, tree, [("fmt", 4, F), ("ks", None, N), ("vs", None, N), ("ks", MIS, AL), ("vs", MIS, AL)])
    append = dict(fmt=3, k=A, ks=256, v=A, vs=256, k_scale=A, v_scale=A, table=A, width=8, lens=A, cu=A, B=2, T=5, Hkv=1, D=256,
                  page=64, pages=9, kp=A, vp=A, stream=None)
    assert L.nq_kv_append(*append.values()) == F                      # its scales are read only
    compact = dict(pool=A, planes=2, plane_bytes=9 * 16 * 4, Hkv=1, page=16, row=4, pages=9, table=A, width=8, lens=A, accept=A, cu=A,
                   B=2, accepted=4, stream=None)
    changed(L.nq_kv_compact, compact, [("row", 2, S), ("row", 12, S), ("row", 0, S), ("row", -4, S), ("plane_bytes", 9 * 16 * 4 - 16, S)])


@no_gpu
def test_what_is_allowed_reaches_the_launch(L):
    """The smallest alignments and the optional arguments: the checks pass, the launch fails."""
    x = A + 4
    assert L.nq_rmsnorm(*dict(NORM, scale=x).values()) == HIP
    assert L.nq_rmsnorm(*dict(NORM, fmt=0, res=None, res_out=None, w=None, scale=None, xs=5128).values()) == HIP
    assert L.nq_rmsnorm(*dict(NORM, fmt=1, K=32768, xs=32768).values()) == HIP
    assert L.nq_quantize_act_fp8_b128(*dict(QUANT, scale=x, K=5136).values()) == HIP
    assert L.nq_gemm_fp8_b128(*dict(PRODUCT, a_scale=x, wsi=x, ws=A, wb=100).values()) == HIP
    assert L.nq_gemm_fp8_b128(*dict(PRODUCT, K=0, gc=0, a=None, w=None, a_scale=None, wsi=None).values()) == HIP
    assert L.nq_kv_append_rope(*dict(ROPE, pos=x, freq=x, ksc=x, vsc=x, table=x, lens=x, cu=x).values()) == HIP
    assert L.nq_kv_append_rope(*dict(ROPE, rot=0, pos=None, freq=None, q=None, qs=0, qo=None, qos=0, qw=None, kw=None, eps=0.0).values()) == HIP
    assert L.nq_kv_append_rope(*dict(ROPE, width=0, table=None, kp=None, vp=None, ksc=None, vsc=None, ko=A, kos=256).values()) == HIP
    assert L.nq_kv_append_rope(*dict(ROPE, fmt=0, ksc=None, vsc=None, rot=256, rope=1).values()) == HIP
    assert L.nq_kv_compact(A, 2, 9 * 16 * 4, 1, 16, 4, 9, x, 8, x, x, x, 2, 4, None) == HIP


def test_binding_refuses_tensors_that_do_not_fit():
    bf = dict(dtype=torch.bfloat16)
    x, w = torch.zeros((3, 128), **bf), torch.zeros(128, **bf)
    codes, scale = torch.zeros((3, 128), dtype=torch.uint8), torch.zeros((3, 1))
    B, E = nq.NQ_ACT_BF16, nq.NQ_ACT_E4M3_B128
    bad = [
        lambda: nq.nq_rmsnorm(B, x.float(), w, 1e-6, x), lambda: nq.nq_rmsnorm(B, x[0], w, 1e-6, x[0]),
        lambda: nq.nq_rmsnorm(B, x, w[:64], 1e-6, x), lambda: nq.nq_rmsnorm(B, x, w.float(), 1e-6, x),
        lambda: nq.nq_rmsnorm(B, x, w, 1e-6, codes), lambda: nq.nq_rmsnorm(E, x, w, 1e-6, x, scale),
        lambda: nq.nq_rmsnorm(E, x, w, 1e-6, codes, None), lambda: nq.nq_rmsnorm(E, x, w, 1e-6, codes, scale[:2]),
        lambda: nq.nq_rmsnorm(E, x, w, 1e-6, codes[:2], scale), lambda: nq.nq_rmsnorm(B, x, w, 1e-6, x, residual=x[:2], residual_out=x),
        lambda: nq.nq_rmsnorm(B, x.t(), w[:3], 1e-6, x.t()),
        lambda: nq.nq_quantize_act_fp8_b128(x, 3, 128, codes[:2], scale), lambda: nq.nq_quantize_act_fp8_b128(x, 3, 128, codes, scale[:2]),
        lambda: nq.nq_gemm_fp8_b128(codes, scale, codes, scale[:1], 3, 4, 128, x), lambda: nq.nq_gemm_fp8_b128(codes, scale[:2], codes, scale[:1], 3, 3, 128, x),
        lambda: nq.nq_gemm_fp8_b128(codes, scale, codes, scale[:1].double(), 3, 3, 128, x),
        lambda: nq.nq_gemm_fp8_b128(codes, scale, codes, scale[:1], 3, 3, 128, x.half()),
    ]
    q, k = torch.zeros((4, 6, 64), **bf), torch.zeros((4, 2, 64), **bf)
    pages, rows = torch.zeros((3, 2, 16, 64), dtype=torch.uint8), torch.zeros((3, 2, 16))
    table, i1 = torch.zeros((1, 2), dtype=torch.int32), torch.tensor([0, 4], dtype=torch.int32)
    pos, freq = torch.zeros(4, dtype=torch.int32), torch.zeros(16)

    def rope(fmt=nq.NQ_KV_E4M3_TOKEN, q=q, k=k, v=k, pos=pos, freq=freq, ks=rows, vs=rows, qo=q, kp=pages, vp=pages, **more):
        nq.nq_kv_append_rope(fmt, q, k, v, pos, freq, nq.NQ_ROPE_HALVES, ks, vs, table, i1[:1], i1, qo, kp, vp, **more)

    bad += [lambda: rope(ks=rows[:2]), lambda: rope(vs=None), lambda: rope(ks=rows.double()), lambda: rope(fmt=nq.NQ_KV_BF16),
            lambda: rope(qo=None), lambda: rope(qo=q[:3]), lambda: rope(q=q[:3]), lambda: rope(v=k[:3]), lambda: rope(pos=pos[:3]),
            lambda: rope(pos=pos.long()), lambda: rope(freq=freq.double()), lambda: rope(q_weight=w), lambda: rope(k_weight=w[:64].float()),
            lambda: rope(k_out=q), lambda: rope(q=q.float()), lambda: rope(kp=pages[:2]),
            lambda: nq.nq_attn_tree(nq.NQ_KV_E4M3_TOKEN, q, pages, pages, rows, rows[:2], table, i1[:1], i1, torch.zeros(4, dtype=torch.int64),
                                    4, 10, 0.1, torch.zeros((4, 6, 64)))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    with pytest.raises(nq.NQError) as e:
        nq.nq_rmsnorm(B, x, w, 0.0, x.clone())
    assert e.value.status == R
    with pytest.raises(nq.NQError) as e:
        nq.nq_gemm_fp8_b128(codes, scale, codes, torch.zeros((2, 1)), 3, 3, 128, x)
    assert e.value.status == S
