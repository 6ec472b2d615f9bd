"""Runs the listed cases of perf/operators.py through the library for a profiler:

    rocprofv3 --kernel-trace --stats -f csv -d OUT -- python3 perf/trace_operators.py [NAME ...]

Each case is prepared three times and run 30 times, the states in turn.  NAME: only cases whose name
contains it.
"""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path[:0] = [ROOT, os.path.join(ROOT, "perf")]

import torch  # noqa: E402

import operators  # noqa: E402


def main(names):
    operators.own = True
    for case in operators.listed():
        if names and not any(n in case["name"] for n in names):
            continue
        states = [operators.prepare(case, seed) for seed in range(3)]
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        for i in range(30):
            operators.run(states[i % 3])
        torch.cuda.synchronize()


if __name__ == "__main__":
    main(sys.argv[1:])
