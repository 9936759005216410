"""Runs cases of perf/more_operators.py on the library's kernels, for a profiler.

    python3 profiles/layer_run.py CASE[,CASE ...] PASSES

CASE is a listed case's name, or `all`; passes go over three sets of inputs in turn.
"""

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from perf import more_operators as cases  # noqa: E402


def main(names, passes):
    cases.own = True
    for case in cases.listed():
        if names != ["all"] and case["name"] not in names:
            continue
        sets = [cases.prepare(case, i) for i in range(3)]
        for i in range(passes):
            cases.run(sets[i % 3])
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        del sets
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main(sys.argv[1].split(","), int(sys.argv[2]))
