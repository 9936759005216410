"""Timed cases of the attention and cache operators (nq_attn_prompt, nq_attn_tree, nq_kv_*).

Each case names one pass a serving engine makes: the attention of a prompt (or a chunk of one), a decode or verify
step over a paged cache (the step's keys and values appended, then the drafted tokens' attention), a beam's
branching (old branches dropped, new ones forked, their last pages copied), and the end of a verify step (the
accepted rows moved together, the pages past them given back).  `run` computes the pass with elementary torch
operations in 32 bits, or, where `own` is true, with the library's kernels.  `exact` gives the attention outputs in
64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
HEADS = [(24, 4, 256), (32, 8, 128), (40, 8, 128), (8, 1, 256), (14, 2, 64), (20, 20, 64)]    # query heads, KV heads, width
PAGES = [16, 32, 64, 128]


def listed():
    return [
        # A chat turn's short prompt alone on the GPU: launch latency and few workgroups.  24 / 4 heads of 256 are the
        # attention shape the projections of this library feed.
        dict(name="prompt-short", op="prompt", seqs=1, q_max=167, context=0, hq=24, hkv=4, d=256, fused=True, out="bf16",
             lens_seed=1),
        # One chunk of 1792 tokens (the prefill chunk) on top of 8192 tokens that came before.
        dict(name="prompt-chunk", op="prompt", seqs=1, q_max=1792, context=8192, hq=24, hkv=4, d=256, fused=False,
             out="bf16", lens_seed=2),
        # A batch of prompts of very different lengths packed together, FP32 out (the bound of the library's FP32 outputs).
        dict(name="prompt-packed", op="prompt", seqs=16, q_max=4097, context=0, hq=32, hkv=8, d=128, fused=True,
             out="f32", lens_seed=3),
        # A long document in one piece.
        dict(name="prompt-long", op="prompt", seqs=1, q_max=16384, context=0, hq=24, hkv=4, d=256, fused=True, out="bf16",
             lens_seed=4),
        # Plain decode of one short conversation: one token, latency.
        dict(name="tree-one-token", op="tree", batch=1, len_max=701, draft_max=1, hq=24, hkv=4, d=256, page=64, fmt="bf16",
             out="bf16", lens_seed=5),
        # A verify step of 33 drafted tokens over a 32K context in an E4M3 cache.
        dict(name="tree-verify", op="tree", batch=1, len_max=32768, draft_max=33, hq=24, hkv=4, d=256, page=64, fmt="e4m3",
             out="bf16", lens_seed=6),
        # A full server: conversations of mixed lengths, a few drafted tokens each, small pages, FP32 out.
        dict(name="tree-batch", op="tree", batch=40, len_max=8191, draft_max=8, hq=32, hkv=8, d=128, page=16, fmt="bf16",
             out="f32", lens_seed=7),
        # Four 128K contexts decoding at the cache's full length.
        dict(name="tree-long", op="tree", batch=4, len_max=131000, draft_max=4, hq=24, hkv=4, d=256, page=128, fmt="bf16",
             out="bf16", lens_seed=8),
        # One conversation forked into four samples: shared pages counted, the last page copied in every plane (K and V
        # of 16 attention layers).
        dict(name="branch-small", op="branch", batch=1, children=4, len_max=1000, planes=32, hkv=4, d=256, page=64,
             fmt="bf16", lens_seed=9),
        # Beams of a batch: 16 conversations, 128 branches.
        dict(name="branch-beams", op="branch", batch=16, children=128, len_max=20000, planes=32, hkv=4, d=256, page=64,
             fmt="bf16", lens_seed=10),
        # The end of one verify step of 33 drafted tokens.
        dict(name="accept-one", op="accept", batch=1, len_max=5000, draft_max=33, planes=32, hkv=4, d=256, page=64,
             fmt="e4m3", lens_seed=11),
        # The end of a batch's verify step.
        dict(name="accept-batch", op="accept", batch=100, len_max=4000, draft_max=64, planes=32, hkv=4, d=256, page=32,
             fmt="bf16", lens_seed=12),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
    n = max(lo, min(hi, n))
    return n - 1 if n == 3072 else n


def draw(rng):
    tops = {}
    for c in listed():
        w = work(c)
        tops[c["op"]] = [max(a, b) for a, b in zip(tops.get(c["op"], (0, 0)), (w["bytes"], w["flops"]))]
    op = rng.choice(["prompt", "prompt", "tree", "tree", "branch", "accept"])
    while True:
        hq, hkv, d = rng.choice(HEADS)
        seed = rng.randrange(1 << 20)
        if op == "prompt":
            context = rng.choice([0, 0, _log(rng, 1, 16384)])
            c = dict(op=op, seqs=_log(rng, 1, 16), q_max=_log(rng, 1, 16384), context=context, hq=hq, hkv=hkv, d=d,
                     fused=context == 0 and rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]), lens_seed=seed)
            fits = c["seqs"] * hq * c["q_max"] * (c["q_max"] + context) * 4 <= 26 << 30
        elif op == "tree":
            c = dict(op=op, batch=_log(rng, 1, 64), len_max=_log(rng, 1, 131000), draft_max=_log(rng, 1, 64), hq=hq, hkv=hkv,
                     d=d, page=rng.choice(PAGES), fmt=rng.choice(["bf16", "e4m3"]), out=rng.choice(["bf16", "f32"]),
                     lens_seed=seed)
            rows = c["batch"] * (c["len_max"] + c["draft_max"])     # the plain form pads every sequence to the longest
            fits = rows * hkv * d * 4 <= 3 << 30 and rows * hq * c["draft_max"] * 4 <= 20 << 30
        elif op == "branch":
            c = dict(op=op, batch=_log(rng, 1, 16), children=_log(rng, 1, 128), len_max=_log(rng, 1, 20000),
                     planes=rng.choice([2, 8, 20, 32]), hkv=hkv, d=d, page=rng.choice(PAGES), fmt=rng.choice(["bf16", "e4m3"]),
                     lens_seed=seed)
            fits = _pool_bytes(c) <= 24 << 30
        else:
            c = dict(op=op, batch=_log(rng, 1, 100), len_max=_log(rng, 1, 4000), draft_max=_log(rng, 1, 64),
                     planes=rng.choice([2, 8, 20, 32]), hkv=hkv, d=d, page=rng.choice(PAGES), fmt=rng.choice(["bf16", "e4m3"]),
                     lens_seed=seed)
            fits = _pool_bytes(c) <= 24 << 30
        w = work(c)
        if fits and w["bytes"] <= tops[op][0] and w["flops"] <= tops[op][1]:
            return c


# ---- what a case says without its data: lengths, drafted tokens, parents, accepted paths ----------------------------

def _spread(rng, n, hi, lo=1):
    """n lengths up to hi, the first of them hi itself, the others spread over the logarithm."""
    return [hi] + [_log(rng, min(lo, hi), hi) for _ in range(n - 1)]


def _prompt_lens(c):
    nq = _spread(random.Random(c["lens_seed"]), c["seqs"], c["q_max"])
    return nq, [n + c["context"] for n in nq]


def _cache_lens(c):
    """(committed lengths, drafted tokens) of each sequence."""
    r = random.Random(c["lens_seed"])
    lo = c["len_max"] // 2 if c["batch"] <= 4 else 1
    lens = _spread(r, c["batch"], c["len_max"], max(1, lo))
    drafts = [c["draft_max"]] + [r.randint(1, c["draft_max"]) for _ in range(c["batch"] - 1)] if "draft_max" in c else None
    return lens, drafts


def _parents(c):
    """The parent (a drafted token of the same sequence, or -1) of each drafted token, sequence by sequence."""
    r = random.Random(c["lens_seed"] + 1)
    return [[r.randint(max(-1, i - 6), i - 1) for i in range(n)] for n in _cache_lens(c)[1]]


def _accepted(c):
    """The drafted tokens each sequence keeps: one path of its tree, root first."""
    r, out = random.Random(c["lens_seed"] + 2), []
    for par in _parents(c):
        path, at = [], r.randrange(len(par))
        while at >= 0:
            path.append(at)
            at = par[at]
        out.append(path[::-1])
    return out


def _forks(c):
    r = random.Random(c["lens_seed"] + 3)
    return [r.randrange(c["batch"]) for _ in range(c["children"])]


def _up(a, b):
    return -(-a // b)


def _pages_held(c):
    lens, drafts = _cache_lens(c)
    return sum(_up(n + (drafts[b] if drafts else 0), c["page"]) for b, n in enumerate(lens))


def _pool_pages(c):
    return _pages_held(c) + c.get("children", 0) + 5        # a few pages stay free


def _pool_bytes(c):
    return c["planes"] * _pool_pages(c) * c["hkv"] * c["page"] * c["d"] * (2 if c["fmt"] == "bf16" else 1)


def work(c):
    size = 2 if c.get("fmt", "bf16") == "bf16" else 1
    if c["op"] == "prompt":
        nq, nk = _prompt_lens(c)
        pairs = sum(n * (k - n) + n * (n + 1) // 2 for n, k in zip(nq, nk))
        out = 2 if c["out"] == "bf16" else 4
        return {"bytes": sum(nq) * c["hq"] * (c["d"] * (2 + out) + 4) + sum(nk) * c["hkv"] * c["d"] * 4,
                "flops": 4 * c["d"] * c["hq"] * pairs}
    lens, drafts = _cache_lens(c)
    if c["op"] == "tree":
        out, t = 2 if c["out"] == "bf16" else 4, sum(drafts)
        seen = sum(n * q + _ancestors(p) for n, q, p in zip(lens, drafts, _parents(c)))
        return {"bytes": (sum(lens) + 2 * t) * c["hkv"] * c["d"] * 2 * size + t * c["hkv"] * c["d"] * 4
                + t * c["hq"] * (c["d"] * (2 + out) + 4) + 4 * sum(_up(n, c["page"]) for n in lens),
                "flops": 4 * c["d"] * c["hq"] * seen}
    row = c["hkv"] * c["d"] * size
    if c["op"] == "branch":
        forks = _forks(c)
        copied = sum(lens[p] % c["page"] != 0 for p in forks)
        entries = sum(_up(lens[p], c["page"]) for p in forks)
        return {"bytes": 2 * copied * c["planes"] * c["page"] * row + 4 * _pool_pages(c) + 24 * entries, "flops": 0}
    moved = sum(sum(i != a for i, a in enumerate(p)) for p in _accepted(c))
    return {"bytes": 2 * moved * c["planes"] * row + 4 * _pool_pages(c) + 16 * c["batch"], "flops": 0}


def _ancestors(par):
    depth = []
    for p in par:
        depth.append(1 + (depth[p] if p >= 0 else 0))
    return sum(depth)


# ---- inputs ---------------------------------------------------------------------------------------------------------

def _cu(ns):
    cu = [0]
    for n in ns:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int32, device=DEV)


def _out_buffers(t, c):
    return (torch.empty((t, c["hq"], c["d"]), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV),
            torch.empty((t, c["hq"]), dtype=torch.float32, device=DEV))


def _table(c, gen, lens, extra):
    """A page table over a shuffled pool: each sequence's pages for lens + extra tokens, -1 past them; and the counts."""
    pages, ps = _pool_pages(c), c["page"]
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    width = max(_up(n + e, ps) for n, e in zip(lens, extra)) + 2
    held = torch.tensor([_up(n + e, ps) for n, e in zip(lens, extra)], device=DEV)
    slot = torch.arange(width, device=DEV)
    start = torch.cumsum(held, 0) - held
    at = (start[:, None] + slot).clamp(max=pages - 1)
    table = torch.where(slot < held[:, None], order[at], -1).to(torch.int32).contiguous()
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    refs[order[: int(sum(_up(n + e, ps) for n, e in zip(lens, extra)))].long()] = 1
    return table, refs


def _pool(c, gen, planes):
    shape = (planes, _pool_pages(c), c["hkv"], c["page"], c["d"])
    if c["fmt"] == "bf16":
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
    codes = torch.randint(0, 254, shape, generator=gen, device=DEV, dtype=torch.uint8)   # every finite code, evenly:
    return codes + (codes >= 127).to(torch.uint8)                                        # 0x7F and 0xFF (NaN) are left out


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"c": c, "scale": 1.0 / math.sqrt(c["d"])}
    if c["op"] == "prompt":
        nq, nk = _prompt_lens(c)
        tq, tk = sum(nq), sum(nk)
        if c["fused"]:      # q, k and v are slices of one projection's output rows
            rows = torch.randn((tq, (c["hq"] + 2 * c["hkv"]), c["d"]), generator=gen, device=DEV, dtype=torch.bfloat16)
            s["q"], s["k"], s["v"] = rows[:, :c["hq"]], rows[:, c["hq"]:-c["hkv"]], rows[:, -c["hkv"]:]
        else:
            s["q"] = torch.randn((tq, c["hq"], c["d"]), generator=gen, device=DEV, dtype=torch.bfloat16)
            s["k"], s["v"] = torch.randn((2, tk, c["hkv"], c["d"]), generator=gen, device=DEV, dtype=torch.bfloat16)
        s["cu_q"], s["cu_k"], s["nq"], s["nk"] = _cu(nq), _cu(nk), max(nq), max(nk)
        s["o"], s["lse"] = _out_buffers(tq, c)
        return s
    lens, drafts = _cache_lens(c)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if c["op"] == "tree":
        t, par = sum(drafts), _parents(c)
        s["table"], _ = _table(c, gen, lens, drafts)
        s["k_pages"], s["v_pages"] = _pool(c, gen, 2)
        if c["fmt"] == "e4m3":      # uniform codes have a deviation near 120: these scales bring keys and values near 1
            s["k_scale"], s["v_scale"] = (0.5 + torch.rand((2, c["hkv"]), generator=gen, device=DEV)) / 120.0
        else:
            s["k_scale"] = s["v_scale"] = None
        s["q"] = torch.randn((t, c["hq"], c["d"]), generator=gen, device=DEV, dtype=torch.bfloat16)
        s["k"], s["v"] = torch.randn((2, t, c["hkv"], c["d"]), generator=gen, device=DEV, dtype=torch.bfloat16)
        masks = []
        for p in par:
            mine = []
            for i, up in enumerate(p):
                mine.append((1 << i) | (mine[up] if up >= 0 else 0))
            masks += mine
        s["mask"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)
        s["cu_q"], s["nq"], s["n"] = _cu(drafts), max(drafts), max(a + b for a, b in zip(lens, drafts))
        s["o"], s["lse"] = _out_buffers(t, c)
        return s
    s["pool"] = _pool(c, gen, c["planes"])
    s["short"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    s["free_list"] = torch.empty(_pool_pages(c), dtype=torch.int32, device=DEV)
    if c["op"] == "branch":
        s["table"], s["refs"] = _table(c, gen, lens, [0] * len(lens))
        s["parents"] = torch.tensor(_forks(c), dtype=torch.int32, device=DEV)
        s["child_table"] = torch.full((c["children"], s["table"].shape[1]), -1, dtype=torch.int32, device=DEV)
        s["none"] = torch.zeros(c["children"], dtype=torch.int32, device=DEV)
        s["copies"] = torch.empty((c["children"], 2), dtype=torch.int32, device=DEV)
    else:
        s["table"], s["refs"] = _table(c, gen, lens, [0] * len(lens))
        width = max(_up(n + q, c["page"]) for n, q in zip(lens, drafts))
        if width > s["table"].shape[1]:
            more = torch.full((len(lens), width - s["table"].shape[1]), -1, dtype=torch.int32, device=DEV)
            s["table"] = torch.cat([s["table"], more], 1).contiguous()
        acc = _accepted(c)
        s["drafted_lens"] = torch.tensor([n + q for n, q in zip(lens, drafts)], dtype=torch.int32, device=DEV)
        s["accept"], s["cu_accept"] = torch.tensor(sum(acc, []), dtype=torch.int32, device=DEV), _cu([len(a) for a in acc])
        s["keep"] = s["lens"]     # all the step's pages are given back, so that another pass can follow
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(s):
    c = s["c"]
    return {"prompt": _prompt, "tree": _tree, "branch": _branch, "accept": _accept}[c["op"]](s, c)


def _owner(cu, t):
    """The sequence of each of t packed rows, and the row's place in it."""
    rows = torch.arange(t, device=DEV)
    b = torch.searchsorted(cu.long(), rows, right=True) - 1
    return b, rows - cu.long()[b]


def _padded(x, cu, n):
    """Packed rows [t][heads][d] as FP32 [sequences][heads][n][d]; what lies past a sequence is some other row."""
    at = (cu[:-1].long()[:, None] + torch.arange(n, device=DEV)).clamp(max=x.shape[0] - 1)
    return x[at].transpose(1, 2).float()


def _attend(q, k, v, seen, scale):
    """Softmax attention in FP32: q [b][hq][nq][d], k / v [b][hkv][nk][d], seen [b][nq][nk] -> o, log-sum-exp."""
    b, hq, nq, d = q.shape
    hkv, nk = k.shape[1], k.shape[2]
    x = torch.matmul(q.reshape(b, hkv, hq // hkv * nq, d), k.transpose(2, 3)).view(b, hkv, hq // hkv, nq, nk)
    x.mul_(scale).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hkv, hq // hkv * nq, nk), v).view(b, hkv, hq // hkv, nq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    return o.reshape(b, hq, nq, d), (top + total.log()).reshape(b, hq, nq)


def _prompt(s, c):
    if own:
        from quantized_weight_linear_amd import nq
        nq.nq_attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["scale"], s["o"], s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    cu_q, cu_k = s["cu_q"], s["cu_k"]
    i, j = torch.arange(s["nq"], device=DEV), torch.arange(s["nk"], device=DEV)
    n_q, n_k = cu_q.diff()[:, None, None], cu_k.diff()[:, None, None]
    seen = (j <= i[:, None] + (n_k - n_q)) & (j < n_k)
    o, lse = _attend(_padded(s["q"], cu_q, s["nq"]), _padded(s["k"], cu_k, s["nk"]), _padded(s["v"], cu_k, s["nk"]), seen,
                     s["scale"])
    b, at = _owner(cu_q, s["q"].shape[0])
    return {"o": o[b, :, at].to(s["o"].dtype), "lse": lse[b, :, at]}


def _as_held(pages, c):
    return pages if c["fmt"] == "bf16" else pages.view(torch.float8_e4m3fn)


def _tree(s, c):
    if own:
        from quantized_weight_linear_amd import nq
        fmt = nq.NQ_KV_BF16 if c["fmt"] == "bf16" else nq.NQ_KV_E4M3
        if "ws" not in s:       # scratch that a program keeps for its stream
            s["ws"] = nq.alloc_attn_tree_workspace(s["lens"].numel(), s["nq"], c["hq"], c["hkv"], c["d"], s["n"], DEV)
        nq.nq_kv_append(fmt, s["k"], s["v"], s["k_scale"], s["v_scale"], s["table"], s["lens"], s["cu_q"], s["k_pages"],
                        s["v_pages"])
        nq.nq_attn_tree(fmt, s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                        s["cu_q"], s["mask"], s["nq"], s["n"], s["scale"], s["o"], s["lse"], s["ws"])
        return {"o": s["o"], "lse": s["lse"], "k_pages": _as_held(s["k_pages"], c), "v_pages": _as_held(s["v_pages"], c)}
    ps, cu, lens = c["page"], s["cu_q"], s["lens"].long()
    b, at = _owner(cu, s["q"].shape[0])
    place = lens[b] + at
    page, slot = s["table"][b, place // ps].long(), place % ps
    j = torch.arange(s["n"], device=DEV)
    held = s["table"][:, j // ps].long().clamp(min=0)
    kv = []
    for new, pages, by in ((s["k"], s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        if by is not None:      # the stored code of x / scale, rounded to nearest even, at most 448 in size
            pages[page, :, slot] = (new.float() / by[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            kv.append(pages[held, :, j % ps].view(torch.float8_e4m3fn).float().mul_(by[:, None]).transpose(1, 2))
        else:
            pages[page, :, slot] = new
            kv.append(pages[held, :, j % ps].float().transpose(1, 2))
    m = s["mask"][(cu[:-1].long()[:, None] + torch.arange(s["nq"], device=DEV)).clamp(max=s["mask"].numel() - 1)]
    far = j - lens[:, None]                                     # a key's place among the drafted tokens
    bit = (m[:, :, None] >> far.clamp(0, 63)[:, None]) & 1
    seen = (far < 0)[:, None] | ((far < cu.diff()[:, None])[:, None] & (bit != 0))
    o, lse = _attend(_padded(s["q"], cu, s["nq"]), kv[0], kv[1], seen, s["scale"])
    return {"o": o[b, :, at].to(s["o"].dtype), "lse": lse[b, :, at], "k_pages": _as_held(s["k_pages"], c),
            "v_pages": _as_held(s["v_pages"], c)}


def _release(refs, table, keep, ps):
    """Entries past the first ceil(keep / ps) of each row are given back and become -1."""
    gone = (torch.arange(table.shape[1], device=DEV) >= ((keep.long() + ps - 1) // ps)[:, None]) & (table >= 0)
    refs.scatter_add_(0, table.long().clamp(min=0).reshape(-1), -gone.to(torch.int32).reshape(-1))
    table.masked_fill_(gone, -1)


def _lowest_free(refs, wanted, free_list, short):
    """For each true entry of `wanted`, in order, the next lowest page that nobody holds (-1 when none is left)."""
    free = refs == 0
    rank = torch.cumsum(free, 0) - 1
    pages = torch.arange(refs.numel(), device=DEV)
    book = torch.full((refs.numel() + wanted.numel() + 1,), -1, dtype=torch.int32, device=DEV)
    book.scatter_(0, torch.where(free, rank, book.numel() - 1), pages.to(torch.int32))
    book[-1] = -1
    flat = wanted.reshape(-1)
    turn = (torch.cumsum(flat, 0) - 1).clamp(min=0)
    got = torch.where(flat, book[turn], -1)
    refs.scatter_add_(0, got.long().clamp(min=0), (got >= 0).to(torch.int32))
    short.copy_((flat & (got < 0)).sum(dtype=torch.int32).reshape(1))
    return got.view(wanted.shape)


def _branch(s, c):
    ps, refs, table, child = c["page"], s["refs"], s["table"], s["child_table"]
    if own:
        from quantized_weight_linear_amd import nq
        nq.nq_kv_release(refs, child, s["none"], ps)
        nq.nq_kv_fork(refs, table, s["lens"], s["parents"], ps, child, s["copies"], s["free_list"], s["short"])
        nq.nq_kv_copy_pages(s["pool"], s["copies"])
    else:
        _release(refs, child, s["none"], ps)
        p = s["parents"].long()
        n, slot = s["lens"].long()[p], torch.arange(table.shape[1], device=DEV)
        full, part = (n // ps)[:, None], n % ps != 0
        mine = torch.where(slot < full, table[p], -1)
        new = _lowest_free(refs, part, s["free_list"], s["short"])
        refs.scatter_add_(0, mine.long().clamp(min=0).reshape(-1), (mine >= 0).to(torch.int32).reshape(-1))
        child.copy_(torch.where((slot == full) & part[:, None], new[:, None], mine))
        last = table[p].gather(1, full.clamp(max=table.shape[1] - 1))[:, 0]
        s["copies"].copy_(torch.stack([torch.where(new >= 0, last, -1), new], 1))
        src, dst = s["copies"][s["copies"][:, 1] >= 0].long().unbind(1)
        s["pool"][:, dst] = s["pool"][:, src]
    return {"refs": refs, "child_table": child, "copies": s["copies"], "short": s["short"], "pool": _as_held(s["pool"], c)}


def _accept(s, c):
    ps, refs, table = c["page"], s["refs"], s["table"]
    if own:
        from quantized_weight_linear_amd import nq
        nq.nq_kv_reserve(refs, table, s["lens"], s["drafted_lens"], ps, s["free_list"], s["short"])
        nq.nq_kv_compact(s["pool"], table, s["lens"], s["accept"], s["cu_accept"])
        held = table.clone()
        nq.nq_kv_release(refs, table, s["keep"], ps)
    else:
        slot = torch.arange(table.shape[1], device=DEV)
        need = (slot < ((s["drafted_lens"].long() + ps - 1) // ps)[:, None]) & (slot >= (s["lens"].long() // ps)[:, None])
        need &= table < 0
        table.copy_(torch.where(need, _lowest_free(refs, need, s["free_list"], s["short"]), table))
        b, i = _owner(s["cu_accept"], s["accept"].numel())
        to, frm = s["lens"].long()[b] + i, s["lens"].long()[b] + s["accept"].long()
        s["pool"][:, table[b, to // ps].long(), :, to % ps] = s["pool"][:, table[b, frm // ps].long(), :, frm % ps]
        held = table.clone()
        _release(refs, table, s["keep"], ps)
    return {"refs": refs, "table": table, "held": held, "short": s["short"], "pool": _as_held(s["pool"], c)}


# ---- 64 bits --------------------------------------------------------------------------------------------------------

def exact(case, seed):
    if case["op"] not in ("prompt", "tree"):
        return None         # nothing is computed there: whole numbers and moved bits
    s = prepare(case, seed)
    c, q = s["c"], s["q"].double()
    out = torch.zeros((q.shape[0], c["hq"], c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.full((q.shape[0], c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    rows = s["cu_q"].tolist()
    keys = s["cu_k"].tolist() if c["op"] == "prompt" else None
    lens = _cache_lens(c)[0] if c["op"] == "tree" else None
    for b in range(len(rows) - 1):
        r0, r1 = rows[b], rows[b + 1]
        n = r1 - r0
        if keys:
            k, v = (s[x][keys[b]:keys[b + 1]].double() for x in ("k", "v"))
            total = k.shape[0]
        else:
            total = lens[b] + n
            ids = s["table"][b, :_up(total, c["page"])].long()
            k, v = (s[x][ids].transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:lens[b]] for x in ("k_pages", "v_pages"))
            k, v = ((x if by is None else x.view(torch.float8_e4m3fn)).double() * (1.0 if by is None else by.double()[:, None])
                    for x, by in ((k, s["k_scale"]), (v, s["v_scale"])))
            fresh = [s[x][r0:r1] for x in ("k", "v")]
            if c["fmt"] == "e4m3":
                fresh = [(x.float() / by[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).double() * by.double()[:, None]
                         for x, by in zip(fresh, (s["k_scale"], s["v_scale"]))]
            k, v = torch.cat([k, fresh[0].double()]), torch.cat([v, fresh[1].double()])
        for h in range(c["hq"]):
            kh, vh = k[:, h // (c["hq"] // c["hkv"])], v[:, h // (c["hq"] // c["hkv"])]
            for a in range(0, n, 4096):
                e = min(n, a + 4096)
                x = (q[r0 + a:r0 + e, h] @ kh.T) / math.sqrt(c["d"])
                at, to = torch.arange(a, e, device=DEV)[:, None], torch.arange(total, device=DEV)
                if keys:
                    hidden = to - (total - n) > at
                else:
                    bits = s["mask"][r0 + a:r0 + e, None] >> (to - lens[b]).clamp(0, 63)
                    hidden = (to >= lens[b]) & (bits % 2 == 0)
                x[hidden] = -math.inf
                lse[r0 + a:r0 + e, h] = torch.logsumexp(x, 1)
                out[r0 + a:r0 + e, h] = torch.softmax(x, 1) @ vh
    return {"o": out, "lse": lse}
