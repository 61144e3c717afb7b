"""Retakes the tables of the layer operators beside this file.

    rocprofv3 --kernel-trace --output-format csv -d OUT -- python3 profiles/layer_operators.py run
    python3 profiles/layer_operators.py times OUT/.../*_kernel_trace.csv > profiles/layer_operators_kernel_trace.txt

    rocprofv3 --pmc COUNTERS --output-format csv -d OUT -- python3 profiles/layer_operators.py run
    python3 profiles/layer_operators.py counters OUT*/.../*_counter_collection.csv > profiles/layer_operators_counters.txt

Counters take a pass each of: the SQ counters below, FETCH_SIZE, WRITE_SIZE.
``run`` takes every case of perf/operators.py through the public entry points,
PASSES times over three sets of buffers in turn; one launch of each of a case's
kernels per pass, which is how the launches are told apart afterwards.
"""
from __future__ import annotations

import csv
import os
import statistics
import sys

PASSES = 12
SQ = ("SQ_ACTIVE_INST_VALU", "SQ_BUSY_CU_CYCLES", "SQ_INSTS_LDS", "SQ_INSTS_MFMA", "SQ_INSTS_VALU", "SQ_LDS_BANK_CONFLICT",
      "SQ_VALU_MFMA_BUSY_CYCLES", "SQ_WAIT_INST_LDS")


def operators():
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from perf import operators as module
    module.own = True
    return module


def run():
    import torch
    op = operators()
    for case in op.listed():
        states = [op.prepare(case, seed) for seed in range(3)]
        for i in range(PASSES):
            op.run(states[i % 3])
        torch.cuda.synchronize()
        print(case["name"], flush=True)


def launches(path):
    """(case, kernel, rows of the file) in order, the library's kernels only."""
    with open(path) as f:
        rows = [r for r in csv.DictReader(f) if "qmm::" in r["Kernel_Name"]]
    rows.sort(key=lambda r: int(r["Dispatch_Id"]))
    by_dispatch = {}
    for r in rows:  # counters: a row per counter
        by_dispatch.setdefault(r["Dispatch_Id"], []).append(r)
    of = [(c["name"], k) for c in operators().listed() for k in range(3 if c["op"] == "moe" else 1)]
    cases, left = {}, list(by_dispatch.values())
    for name, k in of:
        if k == 0:
            kernels = 3 if (name, 2) in of else 1
            taken, left = left[:PASSES * kernels], left[PASSES * kernels:]
            for j in range(kernels):
                cases[name, j] = taken[j::kernels]
    if left:
        sys.exit(f"{path}: {len(left)} launches more than the cases make")
    for (name, _), group in cases.items():
        kernel = group[0][0]["Kernel_Name"].replace("void ", "").replace("qmm::(anonymous namespace)::", "").replace("qmm::", "")
        assert all(g[0]["Kernel_Name"] == group[0][0]["Kernel_Name"] for g in group), name
        yield name, kernel.split("(Moe")[0].split("(Attn")[0].split("(Route")[0].split("(Append")[0].split("(Logprob")[0], group


def times(path):
    print("# Kernel times of the operators of qmm_layer.h, one MI355X, microseconds (profiles/layer_operators.py).")
    print("# rocprofv3 --kernel-trace; the profiler slows the longest kernels down.")
    for name, kernel, group in launches(path):
        t = sorted((int(g[0]["End_Timestamp"]) - int(g[0]["Start_Timestamp"])) / 1e3 for g in group)
        r = group[0][0]
        print(f"{name:19s} {kernel:58s} grid {r['Grid_Size_X']}x{r['Grid_Size_Y']} vgpr {r['VGPR_Count']} lds {r['LDS_Block_Size']} "
              f"scratch {r['Scratch_Size']} n={len(t)} min {t[0]:.2f} med {statistics.median(t):.2f} max {t[-1]:.2f}")


def counters(paths):
    print("# Counters of the operators of qmm_layer.h, one MI355X (profiles/layer_operators.py). rocprofv3 --pmc.")
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
