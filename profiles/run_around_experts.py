"""The workloads of around_experts_rocprofv3.md: each case of perf/more_operators.py 12 times in a row on two sets of inputs
in turn.  Run from the repository's root, alone or under rocprofv3."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from perf import more_operators  # noqa: E402


def main():
    more_operators.own = True
    for case in more_operators.listed():
        st = [more_operators.prepare(case, seed) for seed in (1, 2)]
        for i in range(12):
            more_operators.run(st[i % 2])
        torch.cuda.synchronize()
        print(case["name"], flush=True)


if __name__ == "__main__":
    main()
