"""One call of each profiled case of the operators between the linears, a 256 MB fill
before it; layer_operators.md has the commands that profile it.

    python profiles/layer_operators.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from perf import operators  # noqa: E402

CASES = ("norm prefill 8192x8192", "norm8 4096x5120 g128", "write prompt 4096 3-axis", "read 65536 e4m3",
         "attend 16x4096 e4m3", "attend 48x3001 window", "attend 64x16384")


def main():
    operators.own = True
    listed = {c["name"]: c for c in operators.listed()}
    fill = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for name in CASES:
        case = dict(listed[name])
        if name == "attend 64x16384":
            case["B"] = 16                                   # a quarter of its memory
        state = operators.prepare(case, 5)
        fill.fill_(1)
        operators.run(state)
        torch.cuda.synchronize()


if __name__ == "__main__":
    main()
