"""One attention layer of a server on the library's kernels: prompts, a forked conversation, a verify step of drafted
tokens that form a tree, the accepted path, and a plain decode step, over one paged cache.

    python examples/speculative_steps.py            # BF16 cache
    python examples/speculative_steps.py --e4m3     # E4M3 cache

Weights, tokens' hidden states and the accepted paths are random: the example shows which calls a step makes and in
which order, and compares each attention output with the formula in 64 bits.
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_weight_linear_amd import nq  # noqa: E402

HIDDEN, HQ, HKV, D = 5120, 24, 4, 256
PAGE, PAGES, WIDTH, ROWS = 64, 64, 16, 8
MAX_Q = 8                                        # drafted tokens of a step


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(counts):
    """Offsets of sequences packed one after another."""
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return i32(cu)


def tree_masks(parents):
    """Bit j of mask i: drafted token i comes after token j in the tree, or is it (parents[i] < i, or -1)."""
    masks = []
    for i, p in enumerate(parents):
        masks.append((masks[p] if p >= 0 else 0) | 1 << i)
    return masks


class Linear:
    """A projection with row-scaled E4M3 weights: the GEMM for chunks, the GEMV for steps."""

    def __init__(self, n, k):
        w = (torch.randn((n, k), device="cuda") / math.sqrt(k)).to(torch.bfloat16)
        self.n, self.k = n, k
        self.codes = torch.empty((n, k), dtype=torch.uint8, device="cuda")
        self.scale = torch.empty(n, dtype=torch.bfloat16, device="cuda")
        nq.nq_encode_fp8row_bf16(w, n, k, self.codes, self.scale)
        self.workspace = nq.alloc_gemv_workspace(-1, 64, n, k, "cuda")

    def __call__(self, x):
        t = x.shape[0]
        y = torch.empty((t, self.n), dtype=torch.bfloat16, device="cuda")
        if t >= 129:
            codes = torch.empty((t, self.k), dtype=torch.uint8, device="cuda")
            scale = torch.empty(t, dtype=torch.float32, device="cuda")
            nq.nq_gemm_fp8row(x, self.codes, self.scale, t, self.n, self.k, codes, scale, y)
        else:
            nq.nq_gemv_fp8row(self.codes, self.scale, x, t, self.n, self.k, y, self.workspace)
        return y


class Cache:
    """Pages of one layer's keys and values, and the rows that say which conversation has which."""

    def __init__(self, fmt):
        kind = torch.uint8 if fmt == nq.NQ_KV_E4M3 else torch.bfloat16
        self.fmt = fmt
        self.pool = torch.empty((2, PAGES, HKV, PAGE, D), dtype=kind, device="cuda")
        self.refs = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
        self.table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.free_list = torch.empty(PAGES, dtype=torch.int32, device="cuda")
        self.shortfall = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = torch.full((HKV,), 1 / 32, device="cuda") if fmt == nq.NQ_KV_E4M3 else None
        self.lens = i32([])                      # committed tokens of each conversation

    def rows(self):
        return self.table[:self.lens.numel()]

    def add(self, conversations):
        self.lens = torch.cat([self.lens, torch.zeros(conversations, dtype=torch.int32, device="cuda")])

    def append(self, k, v, cu):
        """Pages for the step's tokens, then their keys and values behind the committed ones."""
        nq.nq_kv_reserve(self.refs, self.rows(), self.lens, self.lens + (cu[1:] - cu[:-1]), PAGE, self.free_list,
                         self.shortfall)
        nq.nq_kv_append(self.fmt, k, v, self.scale, self.scale, self.rows(), self.lens, cu, self.pool[0], self.pool[1])

    def keep(self, accept):
        """The end of a step: the accepted tokens moved together and counted, pages past them given back."""
        cu = starts([len(a) for a in accept])
        nq.nq_kv_compact(self.pool, self.rows(), self.lens, i32([t for a in accept for t in a]), cu)
        self.lens = self.lens + (cu[1:] - cu[:-1])
        nq.nq_kv_release(self.refs, self.rows(), self.lens, PAGE)

    def fork(self, parents):
        """New conversations that go on where others stand: whole pages shared, a part-filled last page copied."""
        n, c = self.lens.numel(), len(parents)
        copies = torch.empty((c, 2), dtype=torch.int32, device="cuda")
        nq.nq_kv_fork(self.refs, self.rows(), self.lens, i32(parents), PAGE, self.table[n:n + c], copies, self.free_list,
                      self.shortfall)
        nq.nq_kv_copy_pages(self.pool, copies)
        self.lens = torch.cat([self.lens, self.lens[parents]])

    def drop(self):
        nq.nq_kv_release(self.refs, self.rows(), torch.zeros_like(self.lens), PAGE)


class Layer:
    def __init__(self, fmt):
        self.qkv, self.out, self.cache = Linear((HQ + 2 * HKV) * D, HIDDEN), Linear(HIDDEN, HQ * D), Cache(fmt)

    def split(self, x):
        y = self.qkv(x).view(-1, HQ + 2 * HKV, D)
        return y[:, :HQ], y[:, HQ:HQ + HKV], y[:, HQ + HKV:]

    def prompt(self, x, counts):
        """Whole prompts of new conversations, packed."""
        q, k, v = self.split(x)
        cu, o = starts(counts), torch.empty((len(x), HQ, D), dtype=torch.bfloat16, device="cuda")
        nq.nq_attn_prompt(q, k, v, cu, cu, D ** -0.5, o)
        self.cache.append(k, v, cu)
        self.cache.lens = self.cache.lens + (cu[1:] - cu[:-1])
        return self.out(o.view(len(x), -1)), (q, k, v, o)

    def step(self, x, trees):
        """Drafted tokens of every conversation (trees[b]: their parents), not yet committed."""
        c = self.cache
        q, k, v = self.split(x)
        cu, o = starts([len(t) for t in trees]), torch.empty((len(x), HQ, D), dtype=torch.bfloat16, device="cuda")
        masks = torch.tensor([m for t in trees for m in tree_masks(t)], dtype=torch.int64, device="cuda")
        c.append(k, v, cu)
        most = WIDTH * PAGE
        workspace = nq.alloc_attn_tree_workspace(len(trees), MAX_Q, HQ, HKV, D, most, "cuda")
        nq.nq_attn_tree(c.fmt, q, c.pool[0], c.pool[1], c.scale, c.scale, c.rows(), c.lens, cu, masks, MAX_Q, most,
                        D ** -0.5, o, workspace=workspace)
        return self.out(o.view(len(x), -1)), (q, k, v, o)


def attention(q, k, v):
    """The formula in 64 bits: one token's queries over the keys it sees."""
    k, v = (t.double().repeat_interleave(HQ // HKV, 1) for t in (k, v))
    return torch.einsum("hn,nhd->hd", torch.softmax(torch.einsum("hd,nhd->hn", q.double(), k) * D ** -0.5, 1), v)


def main(fmt):
    """Runs the steps; returns the largest relative error of an attention output and the page counts at the end."""
    torch.manual_seed(1)
    layer, worst = Layer(fmt), 0.0
    cache = layer.cache
    hidden = lambda n: torch.randn((n, HIDDEN), device="cuda").to(torch.bfloat16)  # noqa: E731
    stored = lambda t: ((t.float() * 32).to(torch.float8_e4m3fn).double() / 32  # noqa: E731
                        if fmt == nq.NQ_KV_E4M3 else t.double())

    def check(name, got, wanted):
        nonlocal worst
        error = float((got.double() - wanted).norm() / wanted.norm())
        worst = max(worst, error)
        print(f"{name}: {len(got)} tokens, relative error {error:.1e}", flush=True)

    # Two prompts at once.
    counts = [300, 45]
    cache.add(len(counts))
    _, (q, k, v, o) = layer.prompt(hidden(sum(counts)), counts)
    at, held = 0, []                             # held: what each conversation's cache should hold
    wanted = torch.empty(o.shape, dtype=torch.float64, device="cuda")
    for n in counts:
        for i in range(n):
            wanted[at + i] = attention(q[at + i], k[at:at + i + 1], v[at:at + i + 1])
        held.append((stored(k[at:at + n]), stored(v[at:at + n])))
        at += n
    check("prompts", o, wanted)

    # The first conversation is sampled twice more.
    cache.fork([0, 0])
    held += [held[0], held[0]]

    # Verify: a tree of drafted tokens for each (a chain, branches, one token); then paths of them are accepted; then
    # one token each.
    verify = [[-1, 0, 1, 2], [-1, 0, 0, 1, 2, 4], [-1], [-1, 0, 0, 2, 3, 3, 5, 6]]
    accepted = [[0, 1], [0, 2, 4, 5], [0], [0, 2, 3, 5, 6, 7]]
    for name, trees, accept in [("verify", verify, accepted), ("decode", [[-1]] * 4, [[0]] * 4)]:
        _, (q, k, v, o) = layer.step(hidden(sum(len(t) for t in trees)), trees)
        at, wanted = 0, torch.empty(o.shape, dtype=torch.float64, device="cuda")
        for b, tree in enumerate(trees):
            k_new, v_new = stored(k[at:at + len(tree)]), stored(v[at:at + len(tree)])
            for i, m in enumerate(tree_masks(tree)):
                sees = [j for j in range(len(tree)) if m >> j & 1]
                wanted[at + i] = attention(q[at + i], torch.cat([held[b][0], k_new[sees]]),
                                           torch.cat([held[b][1], v_new[sees]]))
            held[b] = (torch.cat([held[b][0], k_new[accept[b]]]), torch.cat([held[b][1], v_new[accept[b]]]))
            at += len(tree)
        check(name, o, wanted)
        cache.keep(accept)

    used = int((cache.refs > 0).sum())
    assert cache.lens.tolist() == [len(h[0]) for h in held] and int(cache.shortfall) == 0
    cache.drop()
    left = int(cache.refs.sum())
    print(f"{used} pages for {[len(h[0]) for h in held]} tokens, {left} after the conversations' end", flush=True)
    return worst, used, left


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("--e4m3", action="store_true", help="an E4M3 cache (BF16 otherwise)")
    main(nq.NQ_KV_E4M3 if parser.parse_args().e4m3 else nq.NQ_KV_BF16)
