"""nq_attn_prompt and nq_attn_tree against the operators' definitions in 64 bits.

Tolerances, from the arithmetic: an FP32 output sums products that are exact in FP32 with FP32 accumulation, and its
softmax weights carry 22 bits, so it keeps the library's bound for FP32 outputs, 1e-5 relative (Frobenius).  A BF16
output adds the rounding of the weights and of the result, at most 2^-9 each: 2^-8.  The log-sum-exp is FP32: 1e-5 of
max(1, |lse|).
"""

import math

import pytest
import torch

from quantized_weight_linear_amd import nq

pytestmark = pytest.mark.gpu

DEV = "cuda"
FP32_TOL, BF16_TOL, LSE_TOL = 1e-5, 2.0 ** -8, 1e-5


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(shape, seed, size=1.0):
    return (torch.randn(shape, generator=gen(seed)) * size).to(torch.bfloat16)


def cu_of(ns):
    return torch.tensor([0] + list(torch.tensor(ns).cumsum(0)), dtype=torch.int32)


def softmax_rows(q, k, v, seen, scale):
    """One sequence and head in float64: q [n][d], k / v [m][d], seen [n][m] -> o, lse.  Unseen keys are left out, not
    multiplied by zero."""
    n, d = q.shape
    o, lse = torch.zeros((n, d), dtype=torch.float64), torch.full((n,), -math.inf, dtype=torch.float64)
    x = (q.double() @ torch.nan_to_num(k.double()).T) * scale
    clean = bool(torch.isfinite(k).all() and torch.isfinite(v).all())
    if clean:
        x = torch.where(seen, x, torch.tensor(-math.inf, dtype=torch.float64))
        some = seen.any(1)
        o[some] = torch.softmax(x[some], 1) @ v.double()
        lse[some] = torch.logsumexp(x[some], 1)
        return o, lse
    for i in range(n):
        j = seen[i].nonzero()[:, 0]
        if j.numel():
            x = (k[j].double() @ q[i].double()) * scale
            o[i], lse[i] = torch.softmax(x, 0) @ v[j].double(), torch.logsumexp(x, 0)
    return o, lse


def prompt_oracle(q, k, v, nq_, nk_, scale):
    hq, hkv = q.shape[1], k.shape[1]
    o, lse = torch.zeros(q.shape, dtype=torch.float64), torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    a = c = 0
    for n, m in zip(nq_, nk_):
        seen = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)
        for h in range(hq):
            g = h // (hq // hkv)
            o[a:a + n, h], lse[a:a + n, h] = softmax_rows(q[a:a + n, h], k[c:c + m, g], v[c:c + m, g], seen, scale)
        a, c = a + n, c + m
    return o, lse


def check(got_o, got_lse, o, lse, out):
    torch.cuda.synchronize()
    got, ref = got_o.double().cpu(), o
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    got, ref = torch.nan_to_num(got), torch.nan_to_num(ref)
    empty = (lse == -math.inf)
    assert (got[empty] == 0).all()
    err = (got - ref).norm() / ref.norm() if ref.norm() > 0 else (got - ref).norm()
    print("relative error", float(err), flush=True)
    assert err <= (FP32_TOL if out == torch.float32 else BF16_TOL)
    # no row is off by more than its size: a wrong row among many would hide in the norm
    rows = (got - ref).norm(dim=-1) / ref.norm(dim=-1).clamp(min=1e-30)
    assert (rows <= (20 * FP32_TOL if out == torch.float32 else 4 * BF16_TOL)).all()
    if got_lse is not None:
        x = got_lse.double().cpu()
        assert torch.equal(x == -math.inf, empty) and torch.equal(torch.isnan(x), torch.isnan(lse))
        fine = torch.isfinite(lse)
        assert ((x - lse)[fine].abs() <= LSE_TOL * lse[fine].abs().clamp(min=1)).all()


def run_prompt(q, k, v, nq_, nk_, scale, out, fused=False):
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    if fused:
        rows = torch.cat([qd, kd, vd], 1)
        h, g = q.shape[1], k.shape[1]
        qd, kd, vd = rows[:, :h], rows[:, h:h + g], rows[:, h + g:]
    o = torch.full(q.shape, 7.0, dtype=out, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    nq.nq_attn_prompt(qd, kd, vd, cu_of(nq_).to(DEV), cu_of(nk_).to(DEV), scale, o, lse)
    return o, lse


PROMPTS = [
    ([1], [1]),
    ([2], [2]),
    ([31], [31]),
    ([33, 1, 64], [33, 1, 64]),
    ([0, 5, 0, 3, 0], [0, 5, 3, 0, 0]),          # empty sequences, queries without keys, keys without queries
    ([129, 64, 1, 63], [129, 64, 200, 190]),     # chunks on top of a context
    ([200, 65], [70, 1]),                        # more queries than keys: the first rows see nothing
    ([257], [257]),
    ([513, 300], [513, 300]),
]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,d", [(6, 1, 256), (4, 2, 128), (3, 3, 64), (8, 1, 64)])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompt(case, hq, hkv, d, out):
    n, m = PROMPTS[case]
    q, k, v = randn((sum(n), hq, d), 1), randn((sum(m), hkv, d), 2), randn((sum(m), hkv, d), 3)
    scale = 1.7 / math.sqrt(d)
    o, lse = run_prompt(q, k, v, n, m, scale, out, fused=case % 2 == 1 and n == m)
    check(o, lse, *prompt_oracle(q, k, v, n, m, scale), out)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_many_tiles(d):
    n = [1031, 1, 700]
    q, k, v = randn((sum(n), 2, d), 4), randn((sum(n), 1, d), 5), randn((sum(n), 1, d), 6)
    for out in (torch.float32, torch.bfloat16):
        o, lse = run_prompt(q, k, v, n, n, 1 / math.sqrt(d), out)
        check(o, lse, *prompt_oracle(q, k, v, n, n, 1 / math.sqrt(d)), out)


@pytest.mark.parametrize("hq,hkv,longest", [(2, 1, 33), (12, 1, 300)])
def test_prompt_many_sequences(hq, hkv, longest):
    """More sequences than a wave has lanes, empty ones among them and at the ends."""
    g = gen(3)
    ns = [0, 0] + torch.randint(1, longest + 1, (150,), generator=g).tolist() + [0]
    ns[63], ns[64], ns[100] = 0, 0, longest
    ms = [n + int(e) for n, e in zip(ns, torch.randint(0, 3, (len(ns),), generator=g))]
    q, k, v = randn((sum(ns), hq, 64), 4), randn((sum(ms), hkv, 64), 5), randn((sum(ms), hkv, 64), 6)
    o, lse = run_prompt(q, k, v, ns, ms, 0.125, torch.float32)
    check(o, lse, *prompt_oracle(q, k, v, ns, ms, 0.125), torch.float32)


@pytest.mark.parametrize("d", [64, 256])
def test_prompt_rising_and_large_logits(d):
    """Keys that grow along the sequence move the running reference again and again; logits reach several hundred."""
    n = 400
    q, v = randn((n, 2, d), 7), randn((n, 2, d), 8)
    k = (torch.randn((n, 2, d), generator=gen(9)) * (0.05 + torch.arange(n)[:, None, None] / 12.0)).to(torch.bfloat16)
    for scale in (1 / math.sqrt(d), 2.0, 1e-3):
        o, lse = run_prompt(q, k, v, [n], [n], scale, torch.float32)
        ro, rl = prompt_oracle(q, k, v, [n], [n], scale)
        x = lse.double().cpu()
        # FP32 logits of this size are off by up to 2^-22 of themselves, and the weights by that much absolutely
        size = float(rl.abs().max()) * 2.0 ** -20
        assert ((x - rl).abs() <= max(size, 1e-5)).all()
        err = (o.double().cpu() - ro).norm() / ro.norm()
        assert err <= max(1e-5, size)


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_unseen_values_do_not_matter(d, poison):
    """From a token on, keys and values of one sequence hold what no earlier row may see; another sequence is whole."""
    n, at = [150, 90], 100
    q, k, v = randn((240, 2, d), 10), randn((240, 1, d), 11), randn((240, 1, d), 12)
    scale = 1 / math.sqrt(d)
    ro, rl = prompt_oracle(q, k, v, n, n, scale)
    k[at:150], v[at + 7:150] = poison, poison
    for out in (torch.float32, torch.bfloat16):
        o, lse = run_prompt(q, k, v, n, n, scale, out)
        keep = torch.arange(240) < at
        keep |= torch.arange(240) >= 150
        check(o[keep.to(DEV)], lse[keep.to(DEV)], ro[keep], rl[keep], out)


def test_prompt_values_that_are_seen_do_matter():
    n, d = 80, 128
    q, k, v = randn((n, 1, d), 13), randn((n, 1, d), 14), randn((n, 1, d), 15)
    v[50, 0, 3], v[60, 0, 9] = float("inf"), float("nan")
    q[5] = float("nan")
    o, lse = run_prompt(q, k, v, [n], [n], 0.1, torch.float32)
    ro, rl = prompt_oracle(q, k, v, [n], [n], 0.1)
    got = o.double().cpu()
    assert torch.isnan(got[5]).all() and torch.isnan(lse[5]).all()
    rows = torch.arange(n) != 5
    assert torch.equal(torch.isnan(got[rows]), torch.isnan(ro[rows]))
    assert torch.equal(torch.isinf(got[rows]), torch.isinf(ro[rows]))
    assert (got[50:, 0, 3] == math.inf).all() and torch.isnan(got[60:, 0, 9]).all()


def test_prompt_offsets_are_cut_to_the_arrays():
    """Offsets past the packed rows are cut back; rows outside every sequence stay as they were."""
    q, k, v = randn((70, 2, 64), 16).to(DEV), randn((50, 1, 64), 17).to(DEV), randn((50, 1, 64), 18).to(DEV)
    o = torch.full((70, 2, 64), 7.0, device=DEV)
    nq.nq_attn_prompt(q, k, v, torch.tensor([10, 60, 200], dtype=torch.int32, device=DEV),
                      torch.tensor([-5, 20, 1000], dtype=torch.int32, device=DEV), 0.125, o)
    ro, _ = prompt_oracle(q[10:].cpu(), k.cpu(), v.cpu(), [50, 10], [20, 30], 0.125)
    torch.cuda.synchronize()
    assert (o[:10] == 7).all()
    assert (o[10:].double().cpu() - ro).norm() / ro.norm() <= FP32_TOL


def test_prompt_past_32_bit_offsets():
    """A short sequence at the end of key and value rows whose element offsets pass 2^31 (and byte offsets 2^32)."""
    stride, n, d = 8192, 40, 256
    t = (1 << 31) // stride + 3000
    rows = torch.empty((t, stride), dtype=torch.bfloat16, device=DEV)
    small = randn((n, 8, d), 19)
    rows[-n:, :8 * d] = small.reshape(n, -1).to(DEV)
    wide = rows.view(t, stride // d, d)
    o = torch.zeros((t, 4, d), dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 0, t - n, t], dtype=torch.int32, device=DEV)
    k0 = torch.tensor([0, 0, t - n, t], dtype=torch.int32, device=DEV)
    cu[2], k0[2] = t - n, t - n
    cu[1] = t - n                                   # sequence 0 has queries but no keys; 1 is empty; 2 is the small one
    nq.nq_attn_prompt(wide[:, :4], wide[:, 4:6], wide[:, 6:8], cu, k0, 0.0625, o)
    ro, rl = prompt_oracle(small[:, :4], small[:, 4:6], small[:, 6:8], [n], [n], 0.0625)
    check(o[-n:], None, ro, rl, torch.bfloat16)
    assert (o[:1000] == 0).all()


# ---------------------------------------------------------------------------
# the tree over a paged cache
# ---------------------------------------------------------------------------

def e4m3(x):
    """code values of x, rounded to nearest even, saturating"""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


class Cache:
    """A shuffled cache on the CPU with the keys and values it holds, and the same on the GPU."""

    def __init__(self, lens, drafts, hkv, d, page, fp8, seed, spare=3, fill=float("nan"), width=None):
        total = [a + b for a, b in zip(lens, drafts)]
        need = [-(-t // page) for t in total]
        g = gen(seed)
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        self.width = width or max(need + [1]) + 1
        self.table = torch.full((len(lens), self.width), -1, dtype=torch.int32)
        self.k, self.v, self.ks, self.vs = [], [], None, None
        store = torch.float8_e4m3fn if fp8 else torch.bfloat16
        kp = torch.full((pages, hkv, page, d), fill).to(store)      # what lies outside every sequence
        vp = torch.full((pages, hkv, page, d), fill).to(store)
        if fp8:
            self.ks, self.vs = (torch.rand((2, hkv), generator=g) + 0.5) / 100.0
        for b, t in enumerate(total):
            k, v = (torch.randn((t, hkv, d), generator=g) for _ in range(2))
            if fp8:
                k, v = e4m3(k / self.ks[:, None]), e4m3(v / self.vs[:, None])
            else:
                k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
            for i in range(need[b]):
                p = order.pop()
                self.table[b, i] = p
                part = slice(i * page, min(t, (i + 1) * page))
                for pool, x in ((kp, k), (vp, v)):
                    pool.view(torch.uint8 if fp8 else torch.int16)[p, :, :part.stop - part.start] = \
                        x[part].view(torch.uint8 if fp8 else torch.int16).transpose(0, 1)
            self.k.append(k.double() * (self.ks.double()[:, None] if fp8 else 1))
            self.v.append(v.double() * (self.vs.double()[:, None] if fp8 else 1))
        self.kp, self.vp, self.pages, self.page, self.fp8 = kp, vp, pages, page, fp8

    def to_gpu(self):
        raw = torch.uint8 if self.fp8 else torch.bfloat16
        return (self.kp.view(raw).to(DEV), self.vp.view(raw).to(DEV), None if self.ks is None else self.ks.to(DEV),
                None if self.vs is None else self.vs.to(DEV), self.table.to(DEV))


def trees(drafts, seed):
    """Random parents -> ancestor masks (python ints), a token's own bit included."""
    g = gen(seed)
    masks = []
    for n in drafts:
        mine = []
        for i in range(n):
            p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            mine.append((1 << i) | (mine[p] if p >= 0 else 0))
        masks.append(mine)
    return masks


def mask_tensor(masks):
    return torch.tensor([m - (1 << 64) if m >> 63 else m for s in masks for m in s], dtype=torch.int64)


def tree_oracle(q, cache, lens, drafts, masks, scale):
    hq, hkv = q.shape[1], cache.kp.shape[1]
    o, lse = torch.zeros(q.shape, dtype=torch.float64), torch.full(q.shape[:2], -math.inf, dtype=torch.float64)
    a = 0
    for b, (len_, n) in enumerate(zip(lens, drafts)):
        seen = torch.zeros((n, len_ + n), dtype=torch.bool)
        seen[:, :len_] = True
        for i in range(n):
            for j in range(n):
                seen[i, len_ + j] = bool(masks[b][i] >> j & 1)
        for h in range(hq):
            g = h // (hq // hkv)
            o[a:a + n, h], lse[a:a + n, h] = softmax_rows(q[a:a + n, h], cache.k[b][:, g], cache.v[b][:, g], seen, scale)
        a += n
    return o, lse


def run_tree(q, cache, lens, drafts, masks, scale, out, split=True, max_len=None, max_q=None):
    kp, vp, ks, vs, table = cache.to_gpu()
    hq, hkv, d = q.shape[1], kp.shape[1], q.shape[2]
    top, most = max_q or max(drafts), max_len if max_len is not None else max(a + b for a, b in zip(lens, drafts))
    o = torch.full(q.shape, 7.0, dtype=out, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device=DEV)
    ws = nq.alloc_attn_tree_workspace(len(lens), top, hq, hkv, d, most, DEV) if split else None
    if ws is not None:
        ws.fill_(255)           # scratch holds nothing that a call relies on
    nq.nq_attn_tree(nq.NQ_KV_E4M3 if cache.fp8 else nq.NQ_KV_BF16, q.to(DEV), kp, vp, ks, vs, table,
                    torch.tensor(lens, dtype=torch.int32, device=DEV), cu_of(drafts).to(DEV), mask_tensor(masks).to(DEV),
                    top, most, scale, o, lse, ws)
    return o, lse


TREES = [
    ([0], [1]),                                  # nothing committed: the token sees itself
    ([1], [1]),
    ([63, 64, 65], [1, 1, 1]),
    ([700, 3, 0, 1500], [1, 1, 1, 1]),
    ([0, 17, 100], [5, 3, 4]),
    ([250, 0, 30], [33, 9, 0]),
    ([64, 1000], [64, 61]),
    ([40], [64]),
]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,page", [(6, 1, 256, 64), (8, 2, 128, 16), (4, 4, 64, 32), (14, 2, 64, 128)])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(case, hq, hkv, d, page, fp8, out):
    lens, drafts = TREES[case]
    cache, masks = Cache(lens, drafts, hkv, d, page, fp8, 30 + case), trees(drafts, case)
    q = randn((sum(drafts), hq, d), 31)
    scale = 1.3 / math.sqrt(d)
    o, lse = run_tree(q, cache, lens, drafts, masks, scale, out)
    check(o, lse, *tree_oracle(q, cache, lens, drafts, masks, scale), out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,drafts", [(24, 4, 256, 1), (24, 4, 256, 33), (4, 1, 128, 4), (8, 1, 64, 16)])
def test_tree_long_context_split(hq, hkv, d, drafts, fp8):
    """Split over workgroups or not, and whatever length the caller said: the same result up to rounding."""
    lens = [5003]
    cache, masks = Cache(lens, [drafts], hkv, d, 32, fp8, 40), trees([drafts], 41)
    q = randn((drafts, hq, d), 42)
    ref = tree_oracle(q, cache, lens, [drafts], masks, 1 / math.sqrt(d))
    assert nq.nq_attn_tree_workspace_bytes(1, drafts, hq, hkv, d, 5100) > 0
    for split, most in ((True, None), (False, None), (True, 1), (True, 600), (True, 1 << 20)):
        check(*run_tree(q, cache, lens, [drafts], masks, 1 / math.sqrt(d), torch.float32, split, most), *ref, torch.float32)
    check(*run_tree(q, cache, lens, [drafts], masks, 1 / math.sqrt(d), torch.bfloat16), *ref, torch.bfloat16)


@pytest.mark.parametrize("n", [3, 40])
def test_tree_rows_that_see_nothing(n):
    """Masks of zero over no committed tokens: zeros and -infinity; bits past the drafted tokens count for nothing."""
    lens, drafts = [0, 10], [n, n]
    cache = Cache(lens, drafts, 2, 128, 16, False, 50)
    masks = [[0] * n, [0] * n]
    masks[0][1] = 0b1
    masks[1][2] = ((1 << 64) - 1) ^ ((1 << n) - 1)
    q = randn((2 * n, 4, 128), 51)
    o, lse = run_tree(q, cache, lens, drafts, masks, 0.1, torch.float32)
    plain = [[x & ((1 << n) - 1) for x in s] for s in masks]
    check(o, lse, *tree_oracle(q, cache, lens, drafts, plain, 0.1), torch.float32)
    assert (lse[0] == -math.inf).all() and (o[0] == 0).all() and (lse[1] > -math.inf).all()


@pytest.mark.parametrize("poison", [float("nan"), float("inf")])
@pytest.mark.parametrize("fp8,d,n", [(False, 256, 4), (False, 128, 40), (True, 256, 4), (True, 64, 40), (False, 64, 5)])
def test_tree_unseen_drafts_do_not_matter(fp8, d, n, poison):
    """One drafted token's key and value are not finite: only the rows whose ancestor it is may notice."""
    if fp8 and poison == float("inf"):
        pytest.skip("E4M3 has no infinity")
    lens, drafts = [21, 70], [n, n]
    cache, masks = Cache(lens, drafts, 1, d, 16, fp8, 52), trees(drafts, 53)
    bad = 2
    for m in masks:
        for i in range(n):
            m[i] &= ~(1 << bad)
    q = randn((2 * n, 6, d), 54)
    ref = tree_oracle(q, cache, lens, drafts, masks, 0.1)
    for b in range(2):
        at = lens[b] + bad
        p = int(cache.table[b, at // 16])
        cache.kp[p, :, at % 16] = poison
        cache.vp[p, :, at % 16] = poison
    for out in (torch.float32, torch.bfloat16):
        check(*run_tree(q, cache, lens, drafts, masks, 0.1, out), *ref, out)


@pytest.mark.parametrize("n", [2, 40])
def test_tree_scales_of_zero_and_below(n):
    """An all-zero head has a scale of zero; nothing forbids a negative one.  Masked keys stay masked."""
    lens, drafts = [75, 3], [n, n]
    cache, masks = Cache(lens, drafts, 3, 64, 16, True, 63), trees(drafts, 64)
    ks, vs = torch.tensor([0.0, -0.013, 0.01]), torch.tensor([-0.02, 0.01, 0.0])
    for b in range(2):
        cache.k[b] *= (ks.double() / cache.ks.double())[:, None]
        cache.v[b] *= (vs.double() / cache.vs.double())[:, None]
    cache.ks, cache.vs = ks, vs
    q = randn((2 * n, 6, 64), 65)
    o, lse = run_tree(q, cache, lens, drafts, masks, 0.125, torch.float32)
    ref, rl = tree_oracle(q, cache, lens, drafts, masks, 0.125)
    err = (o.double().cpu() - ref).norm() / ref.norm()
    assert err <= FP32_TOL
    assert ((lse.double().cpu() - rl).abs() <= LSE_TOL * rl.abs().clamp(min=1)).all()


def test_tree_pages_outside_the_pool_read_as_zeros():
    lens, drafts = [100], [2]
    cache, masks = Cache(lens, drafts, 1, 64, 16, False, 55), trees(drafts, 56)
    for i, e in ((1, -1), (3, cache.pages), (4, 2 ** 31 - 1)):
        cache.table[0, i] = e
        cache.k[0][16 * i:16 * i + 16], cache.v[0][16 * i:16 * i + 16] = 0, 0
    q = randn((2, 3, 64), 57)
    check(*run_tree(q, cache, lens, drafts, masks, 0.125, torch.float32), *tree_oracle(q, cache, lens, drafts, masks, 0.125),
          torch.float32)


def test_tree_lengths_past_the_table_are_cut():
    """A length past the table's end counts as the table's end: 3 pages of 16, all of them committed."""
    cache, masks = Cache([48], [0], 2, 128, 16, False, 58, width=3), [[1, 3]]
    q = randn((2, 4, 128), 59)
    o, lse = run_tree(q, cache, [60], [2], masks, 0.1, torch.float32)
    x = Cache([48], [0], 2, 128, 16, False, 58, width=3)
    o2 = torch.zeros((2, 4, 128), dtype=torch.float64)
    l2 = torch.zeros((2, 4), dtype=torch.float64)
    for h in range(4):
        o2[:, h], l2[:, h] = softmax_rows(q[:, h], x.k[0][:, h // 2], x.v[0][:, h // 2], torch.ones((2, 48), dtype=torch.bool), 0.1)
    check(o, lse, o2, l2, torch.float32)


def test_tree_past_32_bit_offsets():
    """Pages whose element offsets pass 2^31."""
    hkv, page, d = 4, 64, 256
    pages = (1 << 31) // (hkv * page * d) + 40
    cache, masks = Cache([150], [3], hkv, d, page, False, 60, spare=0, fill=0.0), trees([3], 61)
    q = randn((3, 8, d), 62)
    ref = tree_oracle(q, cache, [150], [3], masks, 0.0625)
    kp, vp = (torch.zeros((pages, hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    n = cache.pages
    kp[-n:], vp[-n:] = cache.kp.to(DEV), cache.vp.to(DEV)
    table = torch.where(cache.table >= 0, cache.table + (pages - n), -1).to(torch.int32).to(DEV)
    o = torch.empty((3, 8, d), dtype=torch.bfloat16, device=DEV)
    nq.nq_attn_tree(nq.NQ_KV_BF16, q.to(DEV), kp, vp, None, None, table, torch.tensor([150], dtype=torch.int32, device=DEV),
                    cu_of([3]).to(DEV), mask_tensor(masks).to(DEV), 3, 153, 0.0625, o)
    check(o, None, *ref, torch.bfloat16)
    # appending there too
    k, v = randn((3, hkv, d), 63).to(DEV), randn((3, hkv, d), 64).to(DEV)
    nq.nq_kv_append(nq.NQ_KV_BF16, k, v, None, None, table, torch.tensor([150], dtype=torch.int32, device=DEV),
                    cu_of([3]).to(DEV), kp, vp)
    p = int(table[0, 150 // page])
    assert torch.equal(kp[p, :, 150 % page:150 % page + 3].transpose(0, 1), k)
    assert torch.equal(vp[p, :, 150 % page:150 % page + 3].transpose(0, 1), v)


def test_one_token_equals_the_prompts_last_row():
    """A prompt's last row and a decode step over the same keys in pages."""
    n, hq, hkv, d, page = 333, 6, 2, 128, 16
    q, k, v = randn((n, hq, d), 65).to(DEV), randn((n, hkv, d), 66).to(DEV), randn((n, hkv, d), 67).to(DEV)
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    o = torch.empty((n, hq, d), dtype=torch.float32, device=DEV)
    nq.nq_attn_prompt(q, k, v, cu, cu, 0.09, o)
    pages = -(-n // page)
    table = torch.randperm(pages, generator=gen(68)).to(torch.int32)[None].to(DEV)
    kp, vp = (torch.zeros((pages, hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    nq.nq_kv_append(nq.NQ_KV_BF16, k, v, None, None, table, zero, cu, kp, vp)
    one = torch.empty((1, hq, d), dtype=torch.float32, device=DEV)
    nq.nq_attn_tree(nq.NQ_KV_BF16, q[-1:], kp, vp, None, None, table, zero + (n - 1), torch.tensor([0, 1], dtype=torch.int32, device=DEV),
                    torch.ones(1, dtype=torch.int64, device=DEV), 1, n, 0.09, one, None,
                    nq.alloc_attn_tree_workspace(1, 1, hq, hkv, d, n, DEV))
    assert (one[0] - o[-1]).norm() / o[-1].norm() <= 2 * FP32_TOL


def test_same_result_every_time_and_on_another_stream():
    lens, drafts = [3000, 100], [9, 9]
    cache, masks = Cache(lens, drafts, 4, 128, 32, True, 70), trees(drafts, 71)
    q = randn((18, 16, 128), 72)
    first = run_tree(q, cache, lens, drafts, masks, 0.1, torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run_tree(q, cache, lens, drafts, masks, 0.1, torch.float32)
        p1 = run_prompt(q, q[:, :4].contiguous(), q[:, 4:8].contiguous(), [18], [18], 0.1, torch.float32)
    torch.cuda.current_stream().wait_stream(side)
    p2 = run_prompt(q, q[:, :4].contiguous(), q[:, 4:8].contiguous(), [18], [18], 0.1, torch.float32)
    torch.cuda.synchronize()
    for a, b in zip(first + p1, second + p2):
        assert torch.equal(a, b)


def test_step_in_a_graph():
    """Append and attention captured once, replayed on new inputs and lengths, each replay against the eager calls."""
    hq, hkv, d, page, n = 8, 2, 128, 16, 5
    lens, drafts = [300, 41], [n, n]
    cache, masks = Cache(lens, drafts, hkv, d, page, False, 73, width=40), trees(drafts, 74)
    kp, vp, _, _, table = cache.to_gpu()
    q, k, v = (torch.empty((2 * n, h, d), dtype=torch.bfloat16, device=DEV) for h in (hq, hkv, hkv))
    ln, cu, mk = torch.tensor(lens, dtype=torch.int32, device=DEV), cu_of(drafts).to(DEV), mask_tensor(masks).to(DEV)
    o, lse = torch.empty((2 * n, hq, d), device=DEV), torch.empty((2 * n, hq), device=DEV)
    ws = nq.alloc_attn_tree_workspace(2, n, hq, hkv, d, 4000, DEV)

    def step(o, lse):
        nq.nq_kv_append(nq.NQ_KV_BF16, k, v, None, None, table, ln, cu, kp, vp)
        nq.nq_attn_tree(nq.NQ_KV_BF16, q, kp, vp, None, None, table, ln, cu, mk, n, 4000, 0.1, o, lse, ws)

    for t in (q, k, v):
        t.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(o, lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(o, lse)
    for rep in range(4):
        for t in (q, k, v):
            t.normal_()
        ln.copy_(torch.tensor([300 - 7 * rep, 41 - rep], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        step(o2, lse2)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        assert torch.isfinite(o).all()


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("hkv", [1, 2, 3])
def test_e4m3_step_with_slices_of_longer_arrays(hkv, n):
    """Scales as rows of one tensor, lengths, offsets, tables and masks as parts of longer ones: the step's keys and
    values appended, then its attention."""
    d, page, lens, drafts = 64, 16, [37, 5], [n, 3]
    cache, masks = Cache(lens, drafts, hkv, d, page, True, 80 + hkv, width=13), trees(drafts, 81)
    q, t = randn((n + 3, 2 * hkv, d), 82), n + 3
    ref = tree_oracle(q, cache, lens, drafts, masks, 0.125)
    new = [torch.cat([x[b][lens[b]:] for b in range(2)]).float() for x in (cache.k, cache.v)]
    scales = torch.stack([cache.ks, cache.vs]).to(DEV)
    kp, vp, _, _, rows = cache.to_gpu()
    for pool in (kp, vp):       # the drafted tokens' places start empty
        for b in range(2):
            for i in range(lens[b], lens[b] + drafts[b]):
                pool[int(rows[b, i // page]), :, i % page] = 0
    table = torch.full((3, 13), -1, dtype=torch.int32, device=DEV)
    table[1:] = rows
    ln = torch.tensor([9] + lens, dtype=torch.int32, device=DEV)
    cu = torch.tensor([9, 0, n, t], dtype=torch.int32, device=DEV)
    mk = torch.cat([torch.zeros(1, dtype=torch.int64), mask_tensor(masks)]).to(DEV)
    lse = torch.full((t * 2 * hkv + 1,), 7.0, device=DEV)
    o = torch.full(q.shape, 7.0, device=DEV)
    # appended as the codes' own values (exact in BF16) under scales of one, so that the codes are those of the cache
    k, v = ((x / s.cpu()[:, None]).to(torch.float8_e4m3fn) for x, s in zip(new, scales))
    one = torch.ones((2, hkv), device=DEV)
    nq.nq_kv_append(nq.NQ_KV_E4M3, k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), one[0], one[1], table[1:], ln[1:],
                    cu[1:], kp, vp)
    nq.nq_attn_tree(nq.NQ_KV_E4M3, q.to(DEV), kp, vp, scales[0], scales[1], table[1:], ln[1:], cu[1:], mk[1:], n if n > 3 else 3,
                    lens[0] + n, 0.125, o, lse[1:])
    check(o, lse[1:].view(t, 2 * hkv), *ref, torch.float32)
    assert lse[0] == 7


def test_prompt_offsets_as_parts_of_longer_arrays():
    q, k, v = randn((40, 2, 64), 83), randn((50, 1, 64), 84), randn((50, 1, 64), 85)
    cu = torch.tensor([3, 0, 10, 40, 5, 0, 20, 50], dtype=torch.int32, device=DEV)
    o, lse = torch.zeros((40, 2, 64), device=DEV), torch.zeros(81, device=DEV)
    nq.nq_attn_prompt(q.to(DEV), k.to(DEV), v.to(DEV), cu[1:4], cu[5:], 0.125, o, lse[1:])
    check(o, lse[1:].view(40, 2), *prompt_oracle(q, k, v, [10, 30], [20, 30], 0.125), torch.float32)


@pytest.mark.parametrize("hq,hkv,d,step,largest", [(24, 4, 256, 21, 33), (8, 1, 64, 16, 17), (4, 1, 128, 3, 3)])
def test_tree_workspace_of_other_sizes(hq, hkv, d, step, largest):
    """A step on the largest step's workspace, and on smaller ones: the keys are split as far as it goes, nothing past
    its end is written, and the result is the same up to rounding."""
    lens = [5003, 900]
    cache, masks = Cache(lens, [step, 2], hkv, d, 32, False, 86), trees([step, 2], 87)
    q = randn((step + 2, hq, d), 88)
    ref = tree_oracle(q, cache, lens, [step, 2], masks, 1 / math.sqrt(d))
    kp, vp, _, _, table = cache.to_gpu()
    ln, cu, mk = torch.tensor(lens, dtype=torch.int32, device=DEV), cu_of([step, 2]).to(DEV), mask_tensor(masks).to(DEV)
    whole = nq.nq_attn_tree_workspace_bytes(2, largest, hq, hkv, d, 5100)
    one = step * hq * (d * 4 + 8)                   # a range's results and sums
    buffer = torch.empty(whole + 4096, dtype=torch.uint8, device=DEV)
    for size, used in ((whole, True), (whole // 3, True), (5 * one + 16, True), (3 * one + 16, True), (3 * one + 15, False), (16, False),
                       (1, False)):
        buffer.fill_(255)
        o, lse = torch.full(q.shape, 7.0, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
        nq.nq_attn_tree(nq.NQ_KV_BF16, q.to(DEV), kp, vp, None, None, table, ln, cu, mk, step, 5100, 1 / math.sqrt(d), o, lse,
                        buffer[:size])
        check(o, lse, *ref, torch.float32)
        assert bool((buffer[:size] != 255).any()) == used, size
        assert (buffer[size:] == 255).all()


# ---------------------------------------------------------------------------
# large values, and rows without a finite logit
# ---------------------------------------------------------------------------

def rising(n, hq, hkv, d, late, top):
    """Rows whose logits (scale 1) are 0 but for some late keys at `top`, natural units, with values near 1e37."""
    q, k = torch.zeros((n, hq, d)), torch.zeros((n, hkv, d))
    q[:, :, 0] = 1.0
    for j in late:
        k[j, :, 0] = top
    v = (1.0 + torch.rand((n, hkv, d), generator=gen(90))) * 1e37
    return q.to(torch.bfloat16), k.to(torch.bfloat16), v.to(torch.bfloat16)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,d", [(4, 64), (4, 256), (132, 64), (68, 256)])        # few tiles, and many
def test_prompt_large_values_under_rising_logits(hq, d, out):
    """A key far above the first ones: the sum of weights times values stays finite where the result is."""
    n = 150
    q, k, v = rising(n, hq, 2, d, [133], 5.0)
    o, lse = run_prompt(q, k, v, [n], [n], 1.0, out)
    check(o, lse, *prompt_oracle(q, k, v, [n], [n], 1.0), out)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("drafts,d", [(2, 256), (40, 128)])
def test_tree_large_values_under_rising_logits(drafts, d, split, out):
    lens = [1500]
    cache, masks = Cache(lens, [drafts], 1, d, 16, False, 91), trees([drafts], 92)
    q, k, v = rising(1500 + drafts, 2, 1, d, [133, 700, 1400], 5.0)
    for i in range(1500 + drafts):
        p = int(cache.table[0, i // 16])
        cache.kp[p, :, i % 16], cache.vp[p, :, i % 16] = k[i], v[i]
    cache.k, cache.v = [k.double()], [v.double()]
    o, lse = run_tree(q[:drafts], cache, lens, [drafts], masks, 1.0, out, split)
    check(o, lse, *tree_oracle(q[:drafts], cache, lens, [drafts], masks, 1.0), out)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,d,n", [(2, 64, 40), (2, 256, 70), (132, 128, 150)])     # few tiles, and many
def test_prompt_rows_of_infinite_negative_logits(hq, d, n, out):
    """Every logit of the first rows is -infinity: zeros and -infinity, whatever the values hold."""
    q, k, v = randn((n, hq, d), 93).abs() + 0.01, randn((n, 1, d), 94), randn((n, 1, d), 95)
    at = n - 5
    k[:at] = -float("inf")
    ro, rl = prompt_oracle(q, k[at:], v[at:], [n], [n - at], 0.1)      # as if these keys were not there
    v[2, 0, 1], v[33, 0, 5], v[at - 3] = float("inf"), float("nan"), -float("inf")
    o, lse = run_prompt(q, k, v, [n], [n], 0.1, out)
    check(o[:at], lse[:at], ro[:at], rl[:at], out)


@pytest.mark.parametrize("drafts,d", [(2, 256), (40, 64)])
@pytest.mark.parametrize("len_", [20, 1500])
def test_tree_rows_of_infinite_negative_logits(len_, drafts, d):
    cache = Cache([len_], [drafts], 1, d, 16, False, 96)
    masks = [[0] * drafts]
    q = randn((drafts, 2, d), 97).abs() + 0.01
    bad = torch.isnan(cache.kp.float())
    cache.kp[:] = -float("inf")
    cache.vp[bad] = float("nan")
    p = int(cache.table[0, 0])
    cache.vp[p, 0, 3, 1], cache.vp[p, 0, 7] = float("inf"), float("nan")
    for out in (torch.float32, torch.bfloat16):
        o, lse = run_tree(q, cache, [len_], [drafts], masks, 0.1, out)
        torch.cuda.synchronize()
        assert (o == 0).all() and (lse == -math.inf).all()


# ---------------------------------------------------------------------------
# many sequences, many parts
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("seqs", [300, 600])
def test_prompt_sequences_past_one_look(seqs):
    """More sequences than a wave takes in at once (256), empty ones around the boundary."""
    g = gen(100)
    ns = torch.randint(1, 20, (seqs,), generator=g).tolist()
    for i in (0, 254, 255, 256, 257, seqs - 1):
        ns[i] = 0
    ns[258] = 200
    ms = [n + int(e) for n, e in zip(ns, torch.randint(0, 3, (seqs,), generator=g))]
    q, k, v = randn((sum(ns), 2, 64), 101), randn((sum(ms), 1, 64), 102), randn((sum(ms), 1, 64), 103)
    o, lse = run_prompt(q, k, v, ns, ms, 0.125, torch.float32)
    check(o, lse, *prompt_oracle(q, k, v, ns, ms, 0.125), torch.float32)


@pytest.mark.parametrize("seqs", [300, 600])
def test_prompt_few_tokens_of_many_sequences(seqs):
    """Few query tiles (their waves take different keys) spread over more than 256 sequences, most of them without queries."""
    ns, ms = [0] * seqs, [70] * seqs
    for i in (0, 3, 254, 256, 257, 299, seqs - 1):
        ns[i] = 1 + i % 40
    q, k, v = randn((sum(ns), 1, 64), 104), randn((sum(ms), 1, 64), 105), randn((sum(ms), 1, 64), 106)
    o, lse = run_prompt(q, k, v, ns, ms, 0.125, torch.float32)
    check(o, lse, *prompt_oracle(q, k, v, ns, ms, 0.125), torch.float32)


@pytest.mark.parametrize("hq,hkv,d,most", [(4, 2, 64, 3), (40, 1, 64, 2), (8, 1, 128, 2)])
@pytest.mark.parametrize("seqs", [70, 130])
def test_tree_many_sequences_split(seqs, hq, hkv, d, most):
    """More sequences than a wave has lanes, some without drafted tokens or without committed ones, a few long."""
    g = gen(107)
    lens = torch.randint(0, 200, (seqs,), generator=g).tolist()
    drafts = torch.randint(0, most + 1, (seqs,), generator=g).tolist()
    for i, n in ((0, 0), (3, 1900), (63, 900), (64, 0), (65, 1300), (seqs - 1, 1000)):
        lens[i] = n
    drafts[1], drafts[63], drafts[64], drafts[65], drafts[seqs - 1] = 0, most, most, 0, most
    cache, masks = Cache(lens, drafts, hkv, d, 32, False, 108), trees(drafts, 109)
    q = randn((sum(drafts), hq, d), 110)
    assert nq.nq_attn_tree_workspace_bytes(seqs, most, hq, hkv, d, 1903) > 0
    o, lse = run_tree(q, cache, lens, drafts, masks, 0.1, torch.float32)
    check(o, lse, *tree_oracle(q, cache, lens, drafts, masks, 0.1), torch.float32)


@pytest.mark.parametrize("hq,d,drafts,len_", [(2, 128, 2, 16300), (2, 128, 2, 17000), (3, 64, 1, 40000), (32, 64, 64, 9000),
                                              (2, 128, 64, 17000)])
@pytest.mark.parametrize("fp8", [False, True])
def test_tree_many_parts(fp8, hq, d, drafts, len_):
    """Up to 128 parts of a sequence, joined by one wave a row (2048 rows) or four."""
    cache, masks = Cache([len_], [drafts], 1, d, 64, fp8, 111), trees([drafts], 112)
    q = randn((drafts, hq, d), 113)
    for out in (torch.float32, torch.bfloat16):
        o, lse = run_tree(q, cache, [len_], [drafts], masks, 1 / math.sqrt(d), out)
        check(o, lse, *tree_oracle(q, cache, [len_], [drafts], masks, 1 / math.sqrt(d)), out)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,d", [(4, 64), (68, 256)])       # few tiles, and many
@pytest.mark.parametrize("scale", [0.125, 1.0, 30.0])
def test_prompt_keys_of_the_lowest_value(scale, hq, d, out):
    """The first keys hold BF16's lowest value: logits of -3.4e38 or, scaled, of -infinity; the later ones are ordinary."""
    n, at = 150, 70
    q, k, v = torch.zeros((n, hq, d), dtype=torch.bfloat16), randn((n, 2, d), 98), randn((n, 2, d), 99)
    q[:, :, 0] = 1.0
    q[:, :, 1:3] = randn((n, hq, 2), 100, 1 / scale)
    k[:at, :, 0], k[:at, :, 1:3] = torch.finfo(torch.bfloat16).min, 0
    o, lse = run_prompt(q, k, v, [n], [n], scale, out)
    ro, rl = prompt_oracle(q, k[at:], v[at:], [n], [n - at], scale)     # from row `at` on, the first keys weigh nothing
    check(o[at:], lse[at:], ro[at:], rl[at:], out)


@pytest.mark.parametrize("drafts,d", [(2, 256), (40, 64)])
@pytest.mark.parametrize("split", [False, True])
def test_tree_keys_of_the_lowest_value(split, drafts, d):
    lens, at = [1500], 200
    cache, masks = Cache(lens, [drafts], 1, d, 16, False, 114), trees([drafts], 115)
    q = torch.zeros((drafts, 2, d), dtype=torch.bfloat16)
    q[:, :, 0], q[:, :, 1:3] = 1.0, randn((drafts, 2, 2), 116)
    for i in range(at):
        cache.kp[int(cache.table[0, i // 16]), :, i % 16] = 0
        cache.kp[int(cache.table[0, i // 16]), :, i % 16, 0] = torch.finfo(torch.bfloat16).min
    o, lse = run_tree(q, cache, lens, [drafts], masks, 1.0, torch.float32, split)
    cache.k, cache.v = [cache.k[0][at:]], [cache.v[0][at:]]
    check(o, lse, *tree_oracle(q, cache, [lens[0] - at], [drafts], masks, 1.0), torch.float32)


@pytest.mark.parametrize("hq,d", [(4, 64), (68, 256)])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e8, 1e9, 1e10, 1e20, 1e30, 1e38])
def test_prompt_far_logits(size, hq, d):
    """Logits of any size: the softmax picks the largest ones."""
    n = 150
    q, k, v = torch.zeros((n, hq, d), dtype=torch.bfloat16), torch.zeros((n, 2, d), dtype=torch.bfloat16), randn((n, 2, d), 117)
    q[:, :, 0], q[:, 1::2, 0] = 1.0, -1.0
    k[:, :, 0] = ((torch.rand((n, 2), generator=gen(118)) * 2 - 1) * size).to(torch.bfloat16)
    k[140:, 0, 0] = k[:140, 0, 0].max()                 # equal ones share
    o, lse = run_prompt(q, k, v, [n], [n], 1.0, torch.float32)
    check(o, lse, *prompt_oracle(q, k, v, [n], [n], 1.0), torch.float32)


@pytest.mark.parametrize("drafts,d", [(2, 256), (40, 64)])
@pytest.mark.parametrize("size", [1e9, 1e20, 1e38])
def test_tree_far_logits(size, drafts, d):
    lens = [1500]
    cache, masks = Cache(lens, [drafts], 1, d, 16, False, 119), trees([drafts], 120)
    q, n = torch.zeros((drafts, 2, d), dtype=torch.bfloat16), 1500 + drafts
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    k = torch.zeros((n, 1, d), dtype=torch.bfloat16)
    k[:, 0, 0] = ((torch.rand(n, generator=gen(121)) * 2 - 1) * size).to(torch.bfloat16)
    for i in range(n):
        cache.kp[int(cache.table[0, i // 16]), :, i % 16] = k[i]
    cache.k = [k.double()]
    for split in (False, True):
        o, lse = run_tree(q, cache, lens, [drafts], masks, 1.0, torch.float32, split)
        check(o, lse, *tree_oracle(q, cache, lens, [drafts], masks, 1.0), torch.float32)
