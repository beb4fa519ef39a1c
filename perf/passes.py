"""Passes of one listed case of perf/operators.py through the library's kernels, as a
profiler's target.
usage: python3 perf/passes.py NAME COUNT
"""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
os.chdir(ROOT)
sys.path.insert(0, ROOT)

import torch  # noqa: E402

from perf import operators  # noqa: E402


def main(name, count):
    operators.own = True
    case = next(c for c in operators.listed() if c["name"] == name)
    state = operators.prepare(case, 1)
    for _ in range(count):
        operators.run(state)
    torch.cuda.synchronize()
    print(f"{name}: {count} passes")


if __name__ == "__main__":
    main(sys.argv[1], int(sys.argv[2]))
