"""Timed cases of a decoder layer's 8-bit step around the projections.

`norm`: RMS norm with the residual's addition and a BF16 or E4M3 output (nq_rmsnorm).  `product`: E4M3 activations times
E4M3 weights with block scales (nq_gemm_fp8_b128).  `append`: heads normalised and rotated by their positions, keys and
values into a paged cache (nq_kv_append_rope).  `attend`: attention of drafted tokens over a cache of E4M3 rows with a
scale each (nq_attn_tree).  `run` computes a pass with elementary torch operations in 32 bits (the rotation's angles in
64), or, where `own` is true, with the library's kernels.  `exact` gives the outputs in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
HEADS = [(24, 4, 256), (32, 8, 128), (40, 8, 128), (8, 1, 256), (14, 2, 64), (20, 20, 64)]    # query heads, KV heads, width
PAGES = [16, 32, 64, 128]
F8 = torch.float8_e4m3fn
EPS = 1e-6


def listed():
    return [
        # A decoding token's hidden state: launch latency.
        dict(name="norm-token", op="norm", tokens=1, width=5120, residual=True, centred=True, out="e4m3"),
        # A prefill chunk of 1792 tokens, ready for the FP8 product.
        dict(name="norm-chunk", op="norm", tokens=1792, width=5120, residual=True, centred=True, out="e4m3"),
        # A long prompt's last norm, without a residual to carry on; an odd number of tokens.
        dict(name="norm-long", op="norm", tokens=16383, width=5120, residual=False, centred=False, out="bf16"),
        # One token through the MLP's first projection: the weights' bytes.
        dict(name="product-token", op="product", m=1, n=17408, k=5120, out="bf16"),
        # A verify step of 33 tokens through the MLP's last projection, FP32 out.
        dict(name="product-verify", op="product", m=33, n=5120, k=17408, out="f32"),
        # A prefill chunk through the MLP's first projection.
        dict(name="product-chunk", op="product", m=1792, n=17408, k=5120, out="bf16"),
        # Sizes that end inside a tile and inside a scale block, FP32 out.
        dict(name="product-odd", op="product", m=457, n=7001, k=5136, out="f32"),
        # One token's heads into an E4M3 cache: 24 / 4 heads of 256 with the first 64 columns rotated.
        dict(name="append-token", op="append", batch=1, len_max=5000, new_max=1, hq=24, hkv=4, d=256, rot=64, pairs=False,
             normed=True, page=64, fmt="token", lens_seed=1),
        # Packed prompts of very different lengths, every column rotated.
        dict(name="append-prompts", op="append", batch=16, len_max=1, new_max=4097, hq=32, hkv=8, d=128, rot=128, pairs=False,
             normed=False, page=16, fmt="bf16", lens_seed=2),
        # Plain decode of one short conversation: latency.
        dict(name="attend-token", op="attend", batch=1, len_max=701, new_max=1, hq=24, hkv=4, d=256, page=64, out="bf16",
             lens_seed=3),
        # A verify step of 33 drafted tokens over a 32K context.
        dict(name="attend-verify", op="attend", batch=1, len_max=32768, new_max=33, hq=24, hkv=4, d=256, page=64, out="bf16",
             lens_seed=4),
        # A batch of conversations of mixed lengths up to 64K, a few drafts each, small pages, FP32 out.
        dict(name="attend-batch", op="attend", batch=16, len_max=65536, new_max=8, hq=32, hkv=8, d=128, page=16, out="f32",
             lens_seed=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    tops = {}
    for c in listed():
        w = work(c)
        tops[c["op"]] = [max(a, b) for a, b in zip(tops.get(c["op"], (0, 0)), (w["bytes"], w["flops"]))]
    op = rng.choice(["norm", "product", "product", "append", "attend", "attend"])
    while True:
        hq, hkv, d = rng.choice(HEADS)
        seed, fits = rng.randrange(1 << 20), True
        if op == "norm":
            c = dict(op=op, tokens=_log(rng, 1, 16384), width=16 * _log(rng, 16, 1088), residual=rng.random() < 0.7,
                     centred=rng.random() < 0.5, out=rng.choice(["bf16", "e4m3", "e4m3"]))
        elif op == "product":
            k = rng.choice([128 * _log(rng, 2, 136), 16 * _log(rng, 16, 1088)])
            c = dict(op=op, m=_log(rng, 1, 8192), n=_log(rng, 64, 20000), k=k, out=rng.choice(["bf16", "bf16", "f32"]))
        elif op == "append":
            c = dict(op=op, batch=_log(rng, 1, 64), len_max=_log(rng, 1, 20000), new_max=_log(rng, 1, 4097), hq=hq, hkv=hkv,
                     d=d, rot=rng.choice([d // 4, d // 2, d]), pairs=rng.random() < 0.3, normed=rng.random() < 0.5,
                     page=rng.choice(PAGES), fmt=rng.choice(["token", "token", "head", "bf16"]), lens_seed=seed)
            fits = _pool_pages(c) * hkv * c["page"] * d * 4 <= 12 << 30
        else:
            c = dict(op=op, batch=_log(rng, 1, 64), len_max=_log(rng, 1, 131000), new_max=_log(rng, 1, 64), hq=hq, hkv=hkv,
                     d=d, page=rng.choice(PAGES), out=rng.choice(["bf16", "f32"]), lens_seed=seed)
            rows = c["batch"] * (c["len_max"] + c["new_max"])       # the plain form pads every sequence to the longest
            fits = rows * hkv * d * 4 <= 5 << 30 and rows * hq * c["new_max"] * 4 <= 20 << 30
        w = work(c)
        if fits and w["bytes"] <= tops[op][0] and w["flops"] <= tops[op][1]:
            return c


# ---- what a case says without its data: lengths, new tokens, parents ------------------------------------------------

def _cache_lens(c):
    """(committed lengths, new tokens) of each sequence."""
    r, n = random.Random(c["lens_seed"]), c["batch"]
    lo = max(1, c["len_max"] // 2 if n <= 4 else 1)
    lens = [c["len_max"]] + [_log(r, lo, c["len_max"]) for _ in range(n - 1)]
    return lens, [c["new_max"]] + [_log(r, 1, c["new_max"]) for _ in range(n - 1)]


def _parents(c):
    """The parent (a drafted token of the same sequence, or -1) of each drafted token, sequence by sequence."""
    r = random.Random(c["lens_seed"] + 1)
    return [[r.randint(max(-1, i - 6), i - 1) for i in range(n)] for n in _cache_lens(c)[1]]


def _up(a, b):
    return -(-a // b)


def _pool_pages(c):
    return sum(_up(n + m, c["page"]) for n, m in zip(*_cache_lens(c))) + 5      # a few pages stay free


def work(c):
    if c["op"] == "norm":
        e, out = c["tokens"] * c["width"], 2 if c["out"] == "bf16" else 1
        scales = 0 if c["out"] == "bf16" else 4 * c["tokens"] * _up(c["width"], 128)
        return {"bytes": e * (2 + out + (4 if c["residual"] else 0)) + scales + 2 * c["width"], "flops": 5 * e}
    if c["op"] == "product":
        m, n, k, g = c["m"], c["n"], c["k"], _up(c["k"], 128)
        return {"bytes": (m + n) * k + 4 * g * (m + _up(n, 128)) + m * n * (2 if c["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    lens, new = _cache_lens(c)
    t, held = sum(new), c["hkv"] * c["d"]
    if c["op"] == "append":
        size = 2 * held if c["fmt"] == "bf16" else held + (4 * c["hkv"] if c["fmt"] == "token" else 0)
        return {"bytes": t * (4 * c["hq"] * c["d"] + 4 * held + 2 * size + 4), "flops": t * (c["hq"] + c["hkv"]) * (3 * c["rot"] + 4 * c["d"])}
    out = 2 if c["out"] == "bf16" else 4
    seen = sum(n * q + _ancestors(p) for n, q, p in zip(lens, new, _parents(c)))
    return {"bytes": (sum(lens) + t) * 2 * (held + 4 * c["hkv"]) + t * c["hq"] * (c["d"] * (2 + out) + 4)
            + 4 * sum(_up(n, c["page"]) for n in lens), "flops": 4 * c["d"] * c["hq"] * seen}


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


def _table(c, gen, held):
    """A page table over a shuffled pool, -1 past each sequence's pages."""
    pages = _pool_pages(c)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    held = torch.tensor(held, device=DEV)
    slot = torch.arange(int(held.max()) + 2, device=DEV)
    at = ((torch.cumsum(held, 0) - held)[:, None] + slot).clamp(max=pages - 1)
    return torch.where(slot < held[:, None], order[at], -1).to(torch.int32).contiguous()


def _codes(gen, shape, spread):
    """Normally spread E4M3 codes, as quantized weights and activations have them."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(spread).clamp_(-448, 448)
    return x.to(F8).view(torch.uint8)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"c": c}

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    def even(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    if c["op"] == "norm":
        t, k = c["tokens"], c["width"]
        s["x"] = normal(t, k) * (0.5 + even(t, 1)).to(torch.bfloat16)
        s["residual"] = normal(t, k) * 4 if c["residual"] else None
        s["weight"] = (0.2 * torch.randn(k, generator=gen, device=DEV) + (0.0 if c["centred"] else 1.0)).to(torch.bfloat16)
        s["y"] = torch.empty((t, k), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.uint8, device=DEV)
        s["scale"] = torch.empty((t, _up(k, 128)), device=DEV) if c["out"] == "e4m3" else None
        s["sum"] = torch.empty((t, k), dtype=torch.bfloat16, device=DEV) if c["residual"] else None
        return s
    if c["op"] == "product":
        m, n, k, g = c["m"], c["n"], c["k"], _up(c["k"], 128)
        s["a"], s["w"] = _codes(gen, (m, k), 110.0), _codes(gen, (n, k), 110.0)
        s["a_scale"] = torch.exp(torch.randn((m, g), generator=gen, device=DEV) * 0.4) * 0.01
        s["w_scale"] = torch.exp(torch.randn((_up(n, 128), g), generator=gen, device=DEV) * 0.4) * 2e-4
        s["y"] = torch.empty((m, n), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
        return s
    lens, new = _cache_lens(c)
    t, hq, hkv, d, pages = sum(new), c["hq"], c["hkv"], c["d"], _pool_pages(c)
    s["lens"], s["cu"] = torch.tensor(lens, dtype=torch.int32, device=DEV), _cu(new)
    s["table"] = _table(c, gen, [_up(n + m, c["page"]) for n, m in zip(lens, new)])
    shape = (2, pages, hkv, c["page"], d)
    if c.get("fmt") == "bf16":
        s["k_pages"], s["v_pages"] = normal(*shape)
        s["k_scale"] = s["v_scale"] = None
    else:       # every finite code, evenly (0x7F and 0xFF, NaN, are left out); their deviation is near 120
        codes = torch.randint(0, 254, shape, generator=gen, device=DEV, dtype=torch.uint8)
        s["k_pages"], s["v_pages"] = codes + (codes >= 127).to(torch.uint8)
        s["k_scale"], s["v_scale"] = (0.5 + even(2, hkv) if c.get("fmt") == "head" else 0.5 + even(2, pages, hkv, c["page"])) / 120.0
    if c["op"] == "append":     # q, k and v are slices of one projection's output rows
        rows = normal(t, hq + 2 * hkv, d)
        s["q"], s["k"], s["v"] = rows[:, :hq], rows[:, hq:-hkv], rows[:, -hkv:]
        s["pos"] = torch.cat([torch.arange(n, n + m, device=DEV) for n, m in zip(lens, new)]).to(torch.int32)
        s["freq"] = (1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])).float()
        s["q_weight"], s["k_weight"] = (1 + 0.2 * normal(2, d)).to(torch.bfloat16) if c["normed"] else (None, None)
        s["q_out"] = torch.empty((t, hq, d), dtype=torch.bfloat16, device=DEV)
        return s
    s["q"] = normal(t, hq, d)
    masks = []
    for p in _parents(c):
        mine = []
        for i, up in enumerate(p):
            mine.append((1 << i) | (mine[up] if up >= 0 else 0))
        masks += mine
    s["mask"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device=DEV)
    s["new"], s["longest"], s["by"] = max(new), max(a + b for a, b in zip(lens, new)), 1.0 / math.sqrt(d)
    s["o"] = torch.empty((t, hq, d), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
    s["lse"] = torch.empty((t, hq), device=DEV)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------

def run(s):
    return {"norm": _norm, "product": _product, "append": _append, "attend": _attend}[s["c"]["op"]](s, s["c"])


def _blocks(x, scale):
    """The scales of blocks of 128 columns, a column each, for x's columns."""
    return scale.repeat_interleave(128, -1)[..., :x.shape[-1]]


def _to_blocks(y):
    """E4M3 codes of y and their scales, one for 128 columns."""
    k = y.shape[-1]
    g = _up(k, 128)
    padded = torch.nn.functional.pad(y, (0, 128 * g - k)).view(-1, g, 128)
    scale = padded.abs().amax(-1) / 448.0
    codes = (padded / scale[..., None]).nan_to_num_(0.0).clamp_(-448, 448).to(F8)
    return codes.view(-1, g * 128)[:, :k].contiguous(), scale


def _norm(s, c):
    if own:
        from quantized_weight_linear_amd import nq
        nq.nq_rmsnorm(nq.NQ_ACT_BF16 if c["out"] == "bf16" else nq.NQ_ACT_E4M3_B128, s["x"], s["weight"], EPS, s["y"], s["scale"],
                      residual=s["residual"], residual_out=s["sum"], weight_bias=1.0 if c["centred"] else 0.0)
        y = s["y"] if c["out"] == "bf16" else s["y"].view(F8)
        return {"y": y, "scale": s["scale"], "sum": s["sum"]}
    h, total = s["x"].float(), None
    if c["residual"]:       # the sum as it is kept is what is normalised
        total = (h + s["residual"].float()).to(torch.bfloat16)
        h = total.float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * (s["weight"].float() + (1.0 if c["centred"] else 0.0))
    if c["out"] == "bf16":
        return {"y": y.to(torch.bfloat16), "scale": None, "sum": total}
    codes, scale = _to_blocks(y)
    return {"y": codes, "scale": scale, "sum": total}


def _product(s, c):
    if own:
        from quantized_weight_linear_amd import nq
        if "ws" not in s:       # scratch that a program keeps for its stream
            s["ws"] = nq.alloc_gemm_fp8_b128_workspace(c["m"], c["n"], c["k"], DEV)
        nq.nq_gemm_fp8_b128(s["a"], s["a_scale"], s["w"], s["w_scale"], c["m"], c["n"], c["k"], s["y"], s["ws"])
        return s["y"]
    a = s["a"].view(F8).float()
    a.mul_(_blocks(a, s["a_scale"]))
    w = s["w"].view(F8).float()
    w.mul_(_blocks(w, s["w_scale"].repeat_interleave(128, 0)[:c["n"]]))
    return torch.matmul(a, w.t()).to(s["y"].dtype)


def _owner(cu, t):
    """The sequence of each of t packed rows, and the row's place in it."""
    rows = torch.arange(t, device=DEV)
    b = torch.searchsorted(cu.long(), rows, right=True) - 1
    return b, rows - cu.long()[b]


def _rotated(x, weight, pos, freq, rot, pairs):
    """Heads x [t][heads][d] normalised (where there is a weight) and turned by their positions."""
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.to(x.dtype)
    angle = pos[:, None].double() * freq.double()
    cos, sin = angle.cos().to(x.dtype)[:, None], angle.sin().to(x.dtype)[:, None]
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _as_held(pages, c):
    return pages if c.get("fmt") == "bf16" else pages.view(F8)


def _append(s, c):
    if own:
        from quantized_weight_linear_amd import nq
        fmt = {"bf16": nq.NQ_KV_BF16, "head": nq.NQ_KV_E4M3, "token": nq.NQ_KV_E4M3_TOKEN}[c["fmt"]]
        nq.nq_kv_append_rope(fmt, s["q"], s["k"], s["v"], s["pos"], s["freq"], nq.NQ_ROPE_PAIRS if c["pairs"] else nq.NQ_ROPE_HALVES,
                             s["k_scale"], s["v_scale"], s["table"], s["lens"], s["cu"], s["q_out"], s["k_pages"], s["v_pages"],
                             q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS)
    else:
        s["q_out"].copy_(_rotated(s["q"].float(), s["q_weight"], s["pos"], s["freq"], c["rot"], c["pairs"]))
        b, i = _owner(s["cu"], s["q"].shape[0])
        place = s["lens"].long()[b] + i
        page, slot = s["table"][b, place // c["page"]].long(), place % c["page"]
        k = _rotated(s["k"].float(), s["k_weight"], s["pos"], s["freq"], c["rot"], c["pairs"])
        _keep(k, s["k_pages"], s["k_scale"], page, slot, c)
        _keep(s["v"].float(), s["v_pages"], s["v_scale"], page, slot, c)
    out = {"q": s["q_out"], "k_pages": _as_held(s["k_pages"], c), "v_pages": _as_held(s["v_pages"], c)}
    return {**out, "k_scale": s["k_scale"], "v_scale": s["v_scale"]} if c["fmt"] == "token" else out


def _keep(x, pages, scale, page, slot, c):
    """Rows x [t][heads][d] into the cache."""
    if c["fmt"] == "bf16":
        pages[page, :, slot] = x.to(torch.bfloat16)
        return
    by = scale
    if c["fmt"] == "token":
        by = x.abs().amax(-1) / 448.0
        scale[page, :, slot] = by
    pages[page, :, slot] = (x / by[..., None]).nan_to_num(0.0).clamp(-448, 448).to(F8).view(torch.uint8)


def _padded(x, cu, n):
    """Packed rows [t][heads][d] as FP32 [sequences][heads][n][d]; what lies past a sequence is some other row."""
    at = (cu[:-1].long()[:, None] + torch.arange(n, device=DEV)).clamp(max=x.shape[0] - 1)
    return x[at].transpose(1, 2).float()


def _attend(s, c):
    if own:
        from quantized_weight_linear_amd import nq
        if "ws" not in s:       # scratch that a program keeps for its stream
            s["ws"] = nq.alloc_attn_tree_workspace(s["lens"].numel(), s["new"], c["hq"], c["hkv"], c["d"], s["longest"], DEV)
        nq.nq_attn_tree(nq.NQ_KV_E4M3_TOKEN, s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["lens"],
                        s["cu"], s["mask"], s["new"], s["longest"], s["by"], s["o"], s["lse"], s["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    ps, cu, lens, hq, hkv, d = c["page"], s["cu"], s["lens"].long(), c["hq"], c["hkv"], c["d"]
    b, at = _owner(cu, s["q"].shape[0])
    j = torch.arange(s["longest"], device=DEV)
    held = s["table"][:, j // ps].long().clamp(min=0)
    k, v = (pages[held, :, j % ps].view(F8).float().mul_(by[held, :, j % ps][..., None]).transpose(1, 2)
            for pages, by in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
    m = s["mask"][(cu[:-1].long()[:, None] + torch.arange(s["new"], device=DEV)).clamp(max=s["mask"].numel() - 1)]
    far = j - lens[:, None]                                     # a key's place among the drafted tokens
    bit = (m[:, :, None] >> far.clamp(0, 63)[:, None]) & 1
    seen = (far < 0)[:, None] | ((far < cu.diff()[:, None])[:, None] & (bit != 0))
    q = _padded(s["q"], cu, s["new"])
    n, nq, nk = q.shape[0], s["new"], s["longest"]
    x = torch.matmul(q.reshape(n, hkv, hq // hkv * nq, d), k.transpose(2, 3)).view(n, hkv, hq // hkv, nq, nk)
    x.mul_(s["by"]).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(n, hkv, hq // hkv * nq, nk), v).view(n, hkv, hq // hkv, nq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).reshape(n, hq, nq, d)
    lse = (top + total.log()).reshape(n, hq, nq)
    return {"o": o[b, :, at].to(s["o"].dtype), "lse": lse[b, :, at]}


# ---- 64 bits --------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm64, "product": _product64, "append": _append64, "attend": _attend64}[case["op"]](s, s["c"])


def _norm64(s, c):
    h, total = s["x"].double(), None
    if c["residual"]:
        total = h + s["residual"].double()
        h = total.float().to(torch.bfloat16).double()
    w = s["weight"].double() + float(c["centred"])
    y = w * h / torch.sqrt((h * h).sum(1, keepdim=True) / c["width"] + EPS)
    if c["out"] == "bf16":
        return {"y": y, "scale": None, "sum": total}
    scale = torch.stack([p.abs().amax(1) / 448.0 for p in y.split(128, 1)], 1)
    codes = torch.cat([torch.where(e > 0, p / e, torch.zeros_like(p)) for p, e in zip(y.split(128, 1), scale.split(1, 1))], 1)
    return {"y": codes, "scale": scale, "sum": total}       # the codes' values before their rounding


def _product64(s, c):
    y = torch.zeros((c["m"], c["n"]), dtype=torch.float64, device=DEV)
    a, w = s["a"].view(F8), s["w"].view(F8)
    rows = s["w_scale"].double().repeat_interleave(128, 0)[:c["n"]]
    for g in range(_up(c["k"], 128)):
        part = slice(128 * g, min(c["k"], 128 * g + 128))
        y += (a[:, part].double() @ w[:, part].double().t()) * s["a_scale"][:, g:g + 1].double() * rows[:, g]
    return y


def _append64(s, c):
    def turned(x, weight):
        x = x.double()
        if weight is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS) * weight.double()
        out = x.clone()
        half = c["rot"] // 2
        for i in range(half):
            p, q = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + half)
            by = (s["pos"].double() * s["freq"][i].double())[:, None]
            out[..., p] = x[..., p] * torch.cos(by) - x[..., q] * torch.sin(by)
            out[..., q] = x[..., p] * torch.sin(by) + x[..., q] * torch.cos(by)
        return out

    got = {"q": turned(s["q"], s["q_weight"])}
    lens, cu = s["lens"].tolist(), s["cu"].tolist()
    for name, rows in (("k", turned(s["k"], s["k_weight"])), ("v", s["v"].double())):
        pages = _as_held(s[name + "_pages"], c).float()             # (float32 holds a row to 2^-24, where it is read to 2^-4 or 2^-9)
        by = s[name + "_scale"]
        scales = by.double().clone() if c["fmt"] == "token" else None
        for b, n in enumerate(lens):
            at = torch.arange(n, n + cu[b + 1] - cu[b], device=DEV)
            page, slot = s["table"][b].long()[at // c["page"]], at % c["page"]
            mine = rows[cu[b]:cu[b + 1]]
            if c["fmt"] == "token":
                e = mine.abs().amax(-1) / 448.0
                scales[page, :, slot] = e
                mine = mine / e[..., None]
            elif c["fmt"] == "head":
                mine = (mine / by.double()[:, None]).clamp(-448, 448)
            pages[page, :, slot] = mine.float()
        got[name + "_pages"] = pages
        if scales is not None:
            got[name + "_scale"] = scales
    return got


def _attend64(s, c):
    t, hq, hkv = s["q"].shape[0], c["hq"], c["hkv"]
    out = torch.zeros((t, hq, c["d"]), dtype=torch.float64, device=DEV)
    lse = torch.full((t, hq), -math.inf, dtype=torch.float64, device=DEV)
    rows, lens = s["cu"].tolist(), s["lens"].tolist()
    for b, n in enumerate(lens):
        r0, r1 = rows[b], rows[b + 1]
        ids, total = s["table"][b].long(), n + r1 - r0
        ids = ids[:_up(total, c["page"])]
        at = torch.arange(total, device=DEV)
        bits = s["mask"][r0:r1, None] >> (at - n).clamp(0, 63)
        hidden = (at >= n) & (bits % 2 == 0)
        for h in range(hkv):
            k, v = ((s[x + "_pages"][ids, h].view(F8).double() * s[x + "_scale"][ids, h].double()[..., None]).reshape(-1, c["d"])[:total]
                    for x in ("k", "v"))
            for e in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                x = (s["q"][r0:r1, e].double() @ k.t()) / math.sqrt(c["d"])
                x[hidden] = -math.inf
                lse[r0:r1, e] = torch.logsumexp(x, 1)
                out[r0:r1, e] = torch.softmax(x, 1) @ v
    return {"o": out, "lse": lse}
