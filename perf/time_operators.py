"""Times the cases of perf/operators.py, or with --grouped those of perf/more_operators.py, on the current GPU.

    python -m perf.time_operators [--grouped] [--plain] [CASE ...]

For each case, the kernels' calls (--plain: the plain forms) over three states of different inputs in turn, timed
with CUDA events around a run of passes after warm-up: the median of five runs in microseconds a pass, and the
case's bytes and operations at that time.  Host calls are in the time of what the GPU finishes sooner than the host
issues; inputs smaller than L2 stay in it.
"""
import argparse

import torch

from perf import more_operators, operators


def pass_us(states, run=operators.run, budget_ms=60.0):
    """Microseconds a pass over `states` in turn."""
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

    def once(n):
        start.record()
        for i in range(n):
            run(states[i % len(states)])
        stop.record()
        stop.synchronize()
        return start.elapsed_time(stop) / n

    once(3)
    n = max(3, min(2000, int(budget_ms / once(3))))
    return 1e3 * sorted(once(n) for _ in range(5))[2]


def main():
    parser = argparse.ArgumentParser()
    parser.add_argument("--grouped", action="store_true")
    parser.add_argument("--plain", action="store_true")
    parser.add_argument("case", nargs="*")
    args = parser.parse_args()
    cases = more_operators if args.grouped else operators
    cases.own = not args.plain
    known = {c["name"]: c for c in cases.listed()}
    for name in args.case or known:
        if name not in known:
            parser.error(f"no case {name}; there are {', '.join(known)}")
    for name in args.case or known:
        work = cases.work(known[name])
        us = pass_us([cases.prepare(known[name], seed) for seed in range(3)], cases.run)
        print(f"{name:20s} {us:10.2f} us  {work['bytes'] / us * 1e-3:8.0f} GB/s  {work['flops'] / us * 1e-6:8.1f} TFLOP/s",
              flush=True)
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
