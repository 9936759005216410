"""Runs one case of perf/operators.py on the library's kernels, for a profiler or by itself.

    python3 profiles/attention_run.py CASE PASSES [key=value ...]

CASE is a listed case's name; key=value pairs replace its sizes (`tree-long batch=1 len_max=131072`).  `append` is a
prompt's keys and values into a cache (tokens, hkv, d, page, fmt).  Five passes warm up; then five blocks of PASSES
passes are timed with events, launches included, and the median block's time a pass is printed, with the rates that
the case's bytes and operations make of it.
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from perf import operators  # noqa: E402
from quantized_weight_linear_amd import nq  # noqa: E402


def append(tokens, hkv, d, page, fmt):
    """A pass, and its bytes: the rows read, the cache's written."""
    pages, code = -(-tokens // page), fmt == "e4m3"
    k, v = torch.randn((2, tokens, hkv, d), device="cuda").to(torch.bfloat16)
    kp, vp = torch.zeros((2, pages, hkv, page, d), dtype=torch.uint8 if code else torch.bfloat16, device="cuda")
    scale = torch.full((hkv,), 1 / 32, device="cuda") if code else None
    table = torch.randperm(pages, device="cuda").to(torch.int32)[None]
    lens, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0], [0, tokens]))
    kind = nq.NQ_KV_E4M3 if code else nq.NQ_KV_BF16
    return lambda: nq.nq_kv_append(kind, k, v, scale, scale, table, lens, cu, kp, vp), 2 * tokens * hkv * d * (3 if code else 4)


def main(name, passes, *changes):
    if name == "append":
        case = dict(tokens=16384, hkv=4, d=256, page=64, fmt="bf16")
    else:
        case = dict(next(c for c in operators.listed() if c["name"] == name))
    for change in changes:
        key, value = change.split("=")
        if key not in case:
            raise SystemExit(f"{name} has no {key}")
        case[key] = type(case[key])(value)
    if name == "append":
        once, size = append(**case)
        work = {"bytes": size, "flops": 0}
    else:
        operators.own = True
        state, work = operators.prepare(case, 1), operators.work(case)
        once = lambda: operators.run(state)  # noqa: E731
    for _ in range(5):
        once()
    blocks = []
    for _ in range(5):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(int(passes)):
            once()
        end.record()
        end.synchronize()
        blocks.append(start.elapsed_time(end) / int(passes) * 1e3)
    us = sorted(blocks)[2]
    print(f"{' '.join([name, *changes])}: {us:.1f} us, {work['bytes'] / us / 1e3:.0f} GB/s, {work['flops'] / us / 1e6:.0f} TFLOP/s",
          flush=True)


if __name__ == "__main__":
    main(*sys.argv[1:])
