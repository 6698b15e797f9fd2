"""Runs one case of perf/operators.py through the package's calls, for a profiler:

    python3 profiles/run_case.py CASE PASSES
"""
import importlib.util
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402


def main():
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    operators = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(operators)
    operators.own = True
    case, = (c for c in operators.listed() if c["name"] == sys.argv[1])
    state = operators.prepare(case, 1)
    for _ in range(int(sys.argv[2])):
        operators.run(state)
    torch.cuda.synchronize()
    print("done", flush=True)


if __name__ == "__main__":
    main()
