"""Retakes the tables of the 4-bit cache's operators beside this file.

    rocprofv3 --kernel-trace --output-format csv -d OUT -- python3 profiles/cache_operators.py run
    python3 profiles/cache_operators.py times OUT/.../*_kernel_trace.csv > profiles/cache_operators_kernel_trace.txt

    rocprofv3 --pmc COUNTERS --output-format csv -d OUT -- python3 profiles/cache_operators.py run
    python3 profiles/cache_operators.py counters OUT*/.../*_counter_collection.csv > profiles/cache_operators_counters.txt

Counters take a pass each of: the SQ counters of layer_operators.py, FETCH_SIZE, WRITE_SIZE.
``run`` takes every case of perf/more_operators.py through the public entry points, PASSES times over two sets of
buffers in turn after WARM passes that are left out (after a pause the clock takes some thirty launches of the long prompt
to settle: 850 to 970 us at first, then 740); one launch of each of a case's kernels per pass, which is how the launches are
told apart afterwards.
"""
from __future__ import annotations

import csv
import os
import re
import statistics
import sys

from layer_operators import PASSES, SQ

WARM = 40
KERNELS = {"append": 2, "compact": 2}  # launches of a pass; 1 for the others


def operators():
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from perf import more_operators as module
    module.own = True
    return module


def run():
    import torch
    op = operators()
    for case in op.listed():
        states = [op.prepare(case, seed) for seed in range(2)]
        for i in range(WARM + PASSES):
            op.run(states[i % 2])
        torch.cuda.synchronize()
        print(case["name"], flush=True)


def launches(path):
    """(case, kernel, rows of the file) in order, the library's kernels only."""
    by_dispatch = {}
    with open(path) as f:
        for r in csv.DictReader(f):  # counters: a row per counter
            if "qmm::" in r["Kernel_Name"]:
                by_dispatch.setdefault(int(r["Dispatch_Id"]), []).append(r)
    left = [by_dispatch[i] for i in sorted(by_dispatch)]
    for case in operators().listed():
        n = KERNELS.get(case["op"], 1)
        taken, left = left[WARM * n:(WARM + PASSES) * n], left[(WARM + PASSES) * n:]
        for j in range(n):
            group = taken[j::n]
            kernel = group[0][0]["Kernel_Name"]
            assert all(g[0]["Kernel_Name"] == kernel for g in group), case["name"]
            short = kernel.replace("void ", "").replace("(anonymous namespace)::", "").replace("qmm::", "")
            yield case["name"], re.sub(r"\(\w+Args\)$", "", short), group
    if left:
        sys.exit(f"{path}: {len(left)} launches more than the cases make")


def times(path):
    print("# Kernel times of the operators of qmm_cache.h, one MI355X, microseconds (profiles/cache_operators.py).")
    print("# rocprofv3 --kernel-trace.")
    for name, kernel, group in launches(path):
        t = sorted((int(g[0]["End_Timestamp"]) - int(g[0]["Start_Timestamp"])) / 1e3 for g in group)
        r = group[0][0]
        print(f"{name:20s} {kernel:44s} grid {r['Grid_Size_X']}x{r['Grid_Size_Y']} vgpr {r['VGPR_Count']} lds {r['LDS_Block_Size']} "
              f"scratch {r['Scratch_Size']} n={len(t)} min {t[0]:.2f} med {statistics.median(t):.2f} max {t[-1]:.2f}")


def counters(paths):
    print("# Counters of the operators of qmm_cache.h, one MI355X (profiles/cache_operators.py). rocprofv3 --pmc.")
    print("# Medians per launch, SQ counters summed over the device. FETCH_SIZE and WRITE_SIZE in KiB as reported:")
    print("# FETCH_SIZE counts every 128-byte read request as 64 bytes on this chip, WRITE_SIZE is exact.")
    found = {}
    for path in paths:
        for at, (name, kernel, group) in enumerate(launches(path)):
            values = found.setdefault((at, name, kernel), {})
            for counter in {r["Counter_Name"] for r in group[0]}:
                values[counter] = statistics.median(float(r["Counter_Value"]) for g in group for r in g if r["Counter_Name"] == counter)
    for (_, name, kernel), values in found.items():
        print(f"{name}: {kernel}")
        for line in (SQ, ("FETCH_SIZE", "WRITE_SIZE")):
            print("    " + " ".join(f"{c}={values[c]:.4g}" for c in line if c in values))


if __name__ == "__main__":
    if sys.argv[1:2] == ["run"]:
        run()
    elif sys.argv[1:2] == ["times"]:
        times(sys.argv[2])
    elif sys.argv[1:2] == ["counters"]:
        counters(sys.argv[2:])
    else:
        sys.exit(__doc__)
