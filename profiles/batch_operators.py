"""One call of each profiled case of the operators of a batch, a 256 MB fill before it;
batch_operators.md has the commands that profile it.

    python profiles/batch_operators.py [CASE ...]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from perf import more_operators  # noqa: E402

CASES = ("extend prompts 48", "lora 64x4096x28672 r16", "lora 8192x4096x4096 r64", "sample 1x151936", "sample 64x151936 mixed",
         "sample 256x100003 top-p")


def main(names):
    more_operators.own = True
    listed = {c["name"]: c for c in more_operators.listed()}
    fill = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for name in names:
        state = more_operators.prepare(listed[name], 5)
        fill.fill_(1)
        more_operators.run(state)
        torch.cuda.synchronize()


if __name__ == "__main__":
    main(sys.argv[1:] or CASES)
