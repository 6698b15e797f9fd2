"""Runs one case of perf/operators.py or perf/more_operators.py through the package's calls, for a profiler:

    python3 profiles/run_case.py CASE PASSES
"""
import importlib.util
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import torch  # noqa: E402


def case_of(name):
    """The module that lists the case, and the case."""
    for file in "operators", "more_operators":
        spec = importlib.util.spec_from_file_location(file, os.path.join(ROOT, "perf", file + ".py"))
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        for case in module.listed():
            if case["name"] == name:
                return module, case
    raise SystemExit(f"no case {name}")


def main():
    operators, case = case_of(sys.argv[1])
    operators.own = True
    state = operators.prepare(case, 1)
    for _ in range(int(sys.argv[2])):
        operators.run(state)
    torch.cuda.synchronize()
    print("done", flush=True)


if __name__ == "__main__":
    main()
