"""The paged cache's rows and accounting against a plain model on the CPU: whole numbers and moved bits are equal."""

import random

import pytest
import torch

from quantized_weight_linear_amd import nq

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ---- rows in ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("page", [16, 64, 4096])
@pytest.mark.parametrize("hkv,d", [(1, 64), (4, 256), (3, 128)])
def test_append_bf16(hkv, d, page):
    lens, ns = [0, 5, 100, 63], [1, 0, 70, 2]
    t = sum(ns)
    rows = torch.randn((t, 2 * hkv + 1, d), device=DEV).to(torch.bfloat16)       # slices of wider rows
    k, v = rows[:, :hkv], rows[:, hkv:2 * hkv]
    width = 12 if page == 16 else 3
    pages = 4 * width + 1
    table = torch.randperm(pages, device=DEV)[:4 * width].to(torch.int32).view(4, width).contiguous()
    kp, vp = (torch.full((pages, hkv, page, d), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    rk, rv = kp.clone(), vp.clone()
    nq.nq_kv_append(nq.NQ_KV_BF16, k, v, None, None, table, i32(lens), i32([0, 1, 1, 71, 73]), kp, vp)
    at = 0
    for b, n in enumerate(ns):
        for i in range(n):
            p, s = int(table[b, (lens[b] + i) // page]), (lens[b] + i) % page
            rk[p, :, s], rv[p, :, s] = k[at], v[at]
            at += 1
    assert torch.equal(kp, rk) and torch.equal(vp, rv)


def test_append_e4m3_codes():
    """Every code is e4m3_rne_sat(fp32(x / s)), also where x / s saturates, is tiny or is not a number."""
    from oracle import formats as F
    import numpy as np
    hkv, d, page = 2, 64, 16
    x = torch.randn((40, hkv, d)).to(torch.bfloat16)
    x[0], x[1, 0], x[2, 0, :4] = 1e4, -1e4, torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0])
    x[3] = torch.linspace(-500, 500, d)
    x[4] *= 1e-4
    s = torch.tensor([0.37, 1.0])
    table = torch.arange(3, dtype=torch.int32, device=DEV).view(1, 3)
    kp, vp = (torch.zeros((3, hkv, page, d), dtype=torch.uint8, device=DEV) for _ in range(2))
    nq.nq_kv_append(nq.NQ_KV_E4M3, x.to(DEV), x.to(DEV), s.to(DEV), (s * 2).to(DEV), table, i32([0]), i32([0, 40]), kp, vp)
    for pool, by in ((kp, s), (vp, s * 2)):
        got = pool.transpose(1, 2).reshape(48, hkv, d)[:40].cpu().numpy()
        quot = (x.float() / by[:, None]).numpy()
        ref = F.encode_e4m3(quot.astype(np.float64))
        nan = np.isnan(quot)
        assert ((got & 0x7F)[nan] == 0x7F).all()
        assert np.array_equal(got[~nan], ref[~nan])


def test_append_drops_what_has_no_page():
    hkv, d, page = 1, 64, 16
    x = torch.randn((30, hkv, d), device=DEV).to(torch.bfloat16)
    kp, vp = (torch.zeros((4, hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    # row 0: second page missing, third outside the pool; row 1: negative length; rows past the table
    table = i32([[1, -1, 9], [2, 3, 0]])
    nq.nq_kv_append(nq.NQ_KV_BF16, x, x, None, None, table, i32([10, -1]), i32([0, 25, 30]), kp, vp)
    ref = torch.zeros_like(kp)
    ref[1, 0, 10:] = x[:6, 0]
    assert torch.equal(kp, ref) and torch.equal(vp, ref)
    nq.nq_kv_append(nq.NQ_KV_BF16, x, x, None, None, table, i32([1000, 47]), i32([0, 25, 30]), kp, vp)
    ref[0, 0, 15] = x[25, 0]
    assert torch.equal(kp, ref)


# ---- accounting -----------------------------------------------------------------------------------------------------

class Model:
    """Tables and counts as the calls describe them."""

    def __init__(self, pages, rows, width, page):
        self.refs, self.table, self.page = [0] * pages, [[-1] * width for _ in range(rows)], page

    def take(self):
        for i, r in enumerate(self.refs):
            if r == 0:
                self.refs[i] = 1
                return i
        return -1

    def up(self, n):
        return max(0, -(-n // self.page))

    def reserve(self, lens, new):
        short = 0
        for row, a, b in zip(self.table, lens, new):
            for e in range(max(0, a) // self.page, min(self.up(b), len(row))):
                if row[e] < 0:
                    row[e] = self.take()
                    short += row[e] < 0
        return short

    def release(self, table, keep):
        for row, n in zip(table, keep):
            for e in range(self.up(n), len(row)):
                if row[e] >= 0:
                    self.refs[row[e]] -= 1
                    row[e] = -1

    def fork(self, lens, parents):
        child, copies, short = [], [], 0
        for p in parents:
            row = [-1] * len(self.table[0])
            pair = [-1, -1]
            if 0 <= p < len(self.table):
                full = lens[p] // self.page
                if lens[p] % self.page and full < len(row) and self.table[p][full] >= 0:
                    new = self.take()
                    short += new < 0
                    row[full] = new
                    if new >= 0:
                        pair = [self.table[p][full], new]
                row[:full] = self.table[p][:full]
            child.append(row)
            copies.append(pair)
        for row, pair in zip(child, copies):
            for e in row:
                if e >= 0 and e != pair[1]:
                    self.refs[e] += 1
        return child, copies, short


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("pages,rows,width,page", [(40, 5, 7, 16), (300, 40, 20, 32), (20000, 64, 400, 16), (70000, 70, 900, 64)])
def test_reserve_fork_release(pages, rows, width, page, seed):
    r = random.Random(seed)
    m = Model(pages, rows, width, page)
    refs, table = torch.zeros(pages, dtype=torch.int32, device=DEV), torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    free, short = torch.empty(pages, dtype=torch.int32, device=DEV), i32([-7])
    lens = [0] * rows
    for step in range(4):
        new = [min(width * page, n + r.choice([0, 1, r.randrange(1, 3 * page), r.randrange(1, width * page)])) for n in lens]
        if step == 3:
            new[0] = width * page + 999                          # past the table
        nq.nq_kv_reserve(refs, table, i32(lens), i32(new), page, free, short)
        assert m.reserve(lens, new) == int(short)
        assert table.tolist() == m.table and refs.tolist() == m.refs
        parents = [r.randrange(-1, rows + 1) for _ in range(r.choice([1, 3, 1500 if pages < 1000 else 30]))]
        child, copies = torch.full((len(parents), width), -5, dtype=torch.int32, device=DEV), i32([[7, 7]] * len(parents))
        held = [min(n, width * page) for n in new]
        nq.nq_kv_fork(refs, table, i32(held), i32(parents), page, child, copies, free, short)
        mc, mp, ms = m.fork(held, parents)
        assert int(short) == ms
        assert child.tolist() == mc and copies.tolist() == mp and refs.tolist() == m.refs
        some = [r.choice([0, r.randrange(width * page)]) for _ in parents]
        nq.nq_kv_release(refs, child, i32(some), page)
        m.release(mc, some)
        assert child.tolist() == mc and refs.tolist() == m.refs
        nq.nq_kv_release(refs, child, i32([0] * len(parents)), page)
        m.release(mc, [0] * len(parents))
        lens = [r.choice([n, n // 2, 0, max(0, n - 1)]) for n in held]
        nq.nq_kv_release(refs, table, i32(lens), page)
        m.release(m.table, lens)
        assert table.tolist() == m.table and refs.tolist() == m.refs
    nq.nq_kv_release(refs, table, i32([0] * rows), page)
    assert (refs == 0).all() and (table == -1).all()


def test_release_never_counts_below_zero():
    refs, table = i32([1, 0, 2]), i32([[0, 1, 0], [0, 2, 99]])
    nq.nq_kv_release(refs, table, i32([0, -4]), 16)
    assert refs.tolist() == [0, 0, 1] and (table == -1).all()


# ---- pages and rows moved -------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,hkv,page,d", [(torch.bfloat16, 4, 64, 256), (torch.uint8, 1, 16, 64), (torch.bfloat16, 3, 16, 128)])
def test_copy_pages(dtype, hkv, page, d):
    pool = torch.randint(0, 255, (5, 30, hkv, page, d), device=DEV).to(dtype)
    ref = pool.clone()
    pairs = [[3, 0], [3, 1], [-1, -1], [7, 29], [30, 2], [4, 30], [-1, 5], [6, -1], [9, 9], [8, 10]]
    for a, b in pairs:
        if 0 <= a < 30 and 0 <= b < 30:
            ref[:, b] = ref[:, a]
    nq.nq_kv_copy_pages(pool, i32(pairs))
    assert torch.equal(pool, ref)


@pytest.mark.parametrize("dtype,hkv,page,d", [(torch.bfloat16, 4, 64, 256), (torch.uint8, 2, 16, 64), (torch.bfloat16, 1, 16, 128)])
def test_compact(dtype, hkv, page, d):
    r = random.Random(3)
    lens = [0, 5, 15, 16, 100, 77, 40]
    paths = [[0, 1, 2], [0, 2, 5, 63], list(range(1, 64)), [], sorted(r.sample(range(64), 30)), [63], [0, 3, 64, 70]]
    width = 12
    pages = len(lens) * width
    table = torch.randperm(pages, device=DEV).to(torch.int32).view(len(lens), width).contiguous()
    table[6, 3 if page == 16 else 1] = -1
    pool = torch.randint(0, 255, (3, pages, hkv, page, d), device=DEV).to(dtype)
    ref, before = pool.clone(), pool.clone()
    for b, path in enumerate(paths):
        for i, a in enumerate(path):
            if a < 64:
                src, dst = lens[b] + a, lens[b] + i
                ps, pd = int(table[b, src // page]), int(table[b, dst // page])
                if ps >= 0 and pd >= 0:
                    ref[:, pd, :, dst % page] = before[:, ps, :, src % page]
    cu = [0]
    for p in paths:
        cu.append(cu[-1] + len(p))
    nq.nq_kv_compact(pool, table, i32(lens), i32(sum(paths, [])), i32(cu))
    assert torch.equal(pool, ref)


def test_slices_of_longer_arrays():
    """Accounting and moves on parts of a table of width 13, of lengths and of lists: no 16-byte boundary anywhere."""
    page, width, pages = 16, 13, 60
    m = Model(pages, 3, width, page)
    refs = torch.zeros(pages + 1, dtype=torch.int32, device=DEV)[1:]
    whole = torch.full((6, width), -1, dtype=torch.int32, device=DEV)
    lens, new = i32([99, 0, 0, 0]), i32([99, 40, 7, 64])
    free, short = torch.empty(pages + 1, dtype=torch.int32, device=DEV)[1:], i32([5, -7])[1:]
    nq.nq_kv_reserve(refs, whole[1:4], lens[1:], new[1:], page, free, short)
    assert m.reserve([0, 0, 0], [40, 7, 64]) == int(short)
    assert whole[1:4].tolist() == m.table and refs.tolist() == m.refs
    parents, copies = i32([9, 0, 2])[1:], torch.full((5,), 7, dtype=torch.int32, device=DEV)[1:]
    nq.nq_kv_fork(refs, whole[1:4], new[1:], parents, page, whole[4:6], copies, free, short)
    child, pairs, missing = m.fork([40, 7, 64], [0, 2])
    assert whole[4:6].tolist() == child and copies.view(2, 2).tolist() == pairs and int(short) == missing
    assert refs.tolist() == m.refs and (whole[0] == -1).all()
    pool = torch.randint(0, 255, (2, pages, 1, page, 64), device=DEV).to(torch.uint8)
    ref = pool.clone()
    ref[:, pairs[0][1]] = ref[:, pairs[0][0]]
    nq.nq_kv_copy_pages(pool, copies)
    assert torch.equal(pool, ref)
    at = lambda b, i: (int(whole[1 + b, i // page]), i % page)  # noqa: E731
    for b, i, a in ((0, 1, 3), (2, 0, 2), (2, 1, 5)):
        (pd, sd), (ps, ss) = at(b, i + [30, 1, 50][b]), at(b, a + [30, 1, 50][b])
        ref[:, pd, :, sd] = ref[:, ps, :, ss].clone()
    nq.nq_kv_compact(pool, whole[1:4], i32([0, 30, 1, 50])[1:], i32([0, 0, 3, 2, 5])[1:], i32([0, 0, 2, 2, 4])[1:])
    assert torch.equal(pool, ref)
    nq.nq_kv_release(refs, whole[4:6], i32([4, 0, 0])[1:], page)
    m.release(child, [0, 0])
    assert refs.tolist() == m.refs and (whole[4:6] == -1).all()


@pytest.mark.parametrize("planes", [1, 5, 17, 33])
def test_compact_planes(planes):
    """Planes past a wave's, a workgroup's and a row of workgroups'."""
    r = random.Random(planes)
    lens, hkv, page, d, width = [5, 30, 0], 2, 16, 64, 8
    paths = [sorted(r.sample(range(64), 20)), list(range(1, 64)), [2]]
    table = torch.randperm(24, device=DEV).to(torch.int32).view(3, width).contiguous()
    pool = torch.randint(0, 255, (planes, 24, hkv, page, d), device=DEV).to(torch.uint8)
    ref, before = pool.clone(), pool.clone()
    for b, path in enumerate(paths):
        for i, a in enumerate(path):
            src, dst = lens[b] + a, lens[b] + i
            ref[:, int(table[b, dst // page]), :, dst % page] = before[:, int(table[b, src // page]), :, src % page]
    nq.nq_kv_compact(pool, table, i32(lens), i32(sum(paths, [])), i32([0, 20, 83, 84]))
    assert torch.equal(pool, ref)
