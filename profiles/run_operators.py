"""The workloads of operators_rocprofv3.md: each case of perf/operators.py 12 times in a row on two sets of inputs in turn,
then the two largest products with the FP8 instruction's sums.  Run from the repository's root, alone or under rocprofv3."""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_gate_up_amd as mg  # noqa: E402
from perf import operators  # noqa: E402


def fp8_sums(st):
    if st["E"]:
        return mg.moe_decode_matmul_fp8_experts(st["x"], st["sx"], st["counts"], st["w"], st["sw"], st["y"], x_rows=st["x_rows"], fp8_sums=True)
    return mg.moe_decode_matmul_fp8(st["x"], st["sx"], st["w"], st["sw"], st["y"], fp8_sums=True)


def main():
    operators.own = True
    cases = [(c["name"], c, operators.run) for c in operators.listed()]
    cases += [(n + ", FP8 sums", c, fp8_sums) for n, c, _ in cases if n in ("matmul_prompt", "experts_prompt")]
    for name, case, call in cases:
        st = [operators.prepare(case, seed) for seed in (1, 2)]
        for i in range(12):
            call(st[i % 2])
        torch.cuda.synchronize()
        print(name, flush=True)


if __name__ == "__main__":
    main()
