"""Runs cases of perf/more_operators.py through the library: what products_gated_and_4bit.md was taken with.

    python3 profiles/run_case.py --time CASE ...       us of a pass from Python, median and least of nine runs of passes
    rocprofv3 --kernel-trace ... -d OUT/CASE -- python3 profiles/run_case.py CASE
    python3 profiles/run_case.py --table OUT/CASE ...  each kernel's median and least time in those traces

A CASE is a listed name, "all", or an operator with what differs from its defaults, as gated:rows=48,slots=16,rank=16,
group=128 (rows drawn as ids=uniform unless stated).
"""
import csv
import glob
import os
import re
import statistics
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def cases(specs):
    import perf.more_operators as ops
    ops.own = True
    listed = {c["name"]: c for c in ops.listed()}
    for spec in specs:
        if spec == "all":
            yield from ((ops, c) for c in listed.values())
        elif spec in listed:
            yield ops, listed[spec]
        else:
            op, _, rest = spec.partition(":")
            kw = dict(p.split("=") for p in re.split(r",(?=\w+=)", rest))
            kw = {k: int(v) if v.isdigit() else v for k, v in kw.items()}
            yield ops, ops._case(spec, op, kw.pop("rows"), kw.pop("slots"), kw.pop("ids", "uniform"), **kw)


def passes(ops, case, timed):
    """Passes over three states in turn; timed: the nine runs' us a pass."""
    import torch
    states = [ops.prepare(case, seed) for seed in range(3)]
    for st in states * 20:
        ops.run(st)
    torch.cuda.synchronize()
    us, n = [], 3
    while timed and len(us) < 9:
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        for i in range(n):
            ops.run(states[i % 3])
        end.record()
        torch.cuda.synchronize()
        ms = start.elapsed_time(end)
        if ms < 20 and n < 600:  # too few for the clock
            n *= 2
        else:
            us.append(ms / n * 1e3)
    return us


def table(folders):
    for folder in folders:
        times = {}
        for path in glob.glob(folder + "/**/*kernel_trace.csv", recursive=True):
            for row in csv.DictReader(open(path)):
                name = re.sub(r"lora::|\(anonymous namespace\)::|^void |\(.*\)$", "", row["Kernel_Name"])
                if "lora" in row["Kernel_Name"]:
                    us = (int(row["End_Timestamp"]) - int(row["Start_Timestamp"])) / 1e3
                    times.setdefault(name.replace("false", "0").replace("true", "1"), []).append(us)
        for name, us in times.items():
            us = us[len(us) // 3:]  # (the first passes: cold, and the clock on its way)
            print(f"| {os.path.basename(folder)} | `{name}` | {statistics.median(us):.1f} | {min(us):.1f} |")


if __name__ == "__main__":
    if sys.argv[1] == "--table":
        table(sys.argv[2:])
    else:
        timed = sys.argv[1] == "--time"
        for ops, case in cases(sys.argv[1 + timed:]):
            us = passes(ops, case, timed)
            print(f"{case['name']} {statistics.median(us):.1f} {min(us):.1f}" if timed else f"{case['name']} done", flush=True)
