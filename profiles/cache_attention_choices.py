"""Both sides of the choices that qmm_kv4_attention makes between its kernels, timed shape by shape: retakes
cache_attention_choices.txt beside this file.

    python3 profiles/cache_attention_choices.py build DIR          # a library for each side (needs the default build)
    python3 profiles/cache_attention_choices.py run DIR/SIDE.so > DIR/SIDE.txt     # once for each, on the GPU
    python3 profiles/cache_attention_choices.py table DIR > profiles/cache_attention_choices.txt

The sides are builds of kv4_attention.hip in which one rule is replaced by its answer:
    blocks   blocks of many rows for every call
    rows     never blocks; the rest by its rules
    parts    never blocks; keys in parts for every call of up to kMostTiles tiles
    whole    never blocks, never parts
    single   never blocks, never parts, never two tiles a block
Each shape is timed on the sides that its table compares, in graphs of ten calls; the median of seven.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))

BLOCKS = "bool use_tiles(int B, int T, int Hq, int Hkv, int D, int max_q, int max_kv, bool biased, DeviceTopo topo) {"
NO_BLOCKS = (BLOCKS, BLOCKS + "\n  return false;")
NO_PARTS = ("const bool worth_it =", "const bool worth_it = max_kv < 0 &&")
SIDES = {
    "blocks": ((BLOCKS, BLOCKS + "\n  return true;"),),
    "rows": (NO_BLOCKS,),
    "parts": (NO_BLOCKS, ("const bool worth_it =", "const bool worth_it = max_kv > 0 ||")),
    "whole": (NO_BLOCKS, NO_PARTS),
    "single": (NO_BLOCKS, NO_PARTS, ("p.wide = ", "p.wide = false && ")),
}
TABLES = {"blocks": ("blocks", "rows"), "parts": ("parts", "whole"), "pairs": ("whole", "single")}


def build(directory):
    from weight_only_group_amd import build as b
    source = open(os.path.join(b.CSRC, "kv4_attention.hip")).read()
    objects = os.path.join(b.HERE, "_build", "default")
    os.makedirs(directory, exist_ok=True)
    runs = []
    for side, changes in SIDES.items():
        text = source
        for old, new in changes:
            assert text.count(old) == 1, old
            text = text.replace(old, new)
        at = os.path.join(directory, side)
        with open(at + ".hip", "w") as f:
            f.write(text)
        cmd = [b.hipcc(), *b.compile_flags(), "-Wno-unused-function", "-I", b.CSRC, "-c", at + ".hip", "-o", at + ".o"]
        runs.append((at, subprocess.Popen(cmd, stderr=subprocess.DEVNULL)))
    for at, run in runs:
        assert run.wait() == 0, at
        rest = [os.path.join(objects, s.replace(".hip", ".o")) for s in b.SOURCES if s != "kv4_attention.hip"]
        subprocess.run([b.hipcc(), "-shared", f"--offload-arch={b.ARCH}", "-o", at + ".so", at + ".o", *rest], check=True)


# ---- the shapes ------------------------------------------------------------------------------------

def shapes():
    """(table, what the line says, arguments of time())."""
    import numpy as np
    r = np.random.RandomState(5)
    # Prompts whose rows fill the CUs: plain, with windows and documents, with distances, with the plain mask given.
    for D in (64, 128, 256):
        for Hq, Hkv in ((32, 32), (24, 24), (16, 16), (32, 8)):
            for n, B in ((2000, 1), (4000, 1), (8000, 1), (1000, 4), (2000, 4), (500, 16)):
                for mask in ("none", "given", "window 64", "window 256", "window 1024", "6 documents", "20 documents"):
                    for slopes in (False, True):
                        if n * B * Hkv < 31 * 1024 or n * B * Hq // Hkv < 128 * B:
                            continue
                        yield "blocks", (D, Hq, Hkv, B, n, n, mask, "distances" if slopes else "-"), dict(
                            D=D, Hq=Hq, Hkv=Hkv, keys=[n] * B, queries=[n] * B, mask=mask, slopes=slopes)
    # Fewer rows than that, and sequences of a part of a block.
    for D in (64, 128, 256):
        for Hq, Hkv in ((32, 8), (24, 24)):
            for B, q, n in ((1, 500, 4000), (1, 1000, 4000), (1, 2000, 8000), (8, 100, 2000), (16, 100, 2000), (64, 50, 1000), (64, 100, 1000)):
                yield "blocks", (D, Hq, Hkv, B, q, n, "none", "-"), dict(D=D, Hq=Hq, Hkv=Hkv, keys=[n] * B, queries=[q] * B)
    # Single tokens, of even lengths, of ragged ones, and one sequence of the bound's length among short ones; few and many tiles.
    for D in (64, 128, 256):
        for Hq, Hkv in ((32, 8), (16, 16), (8, 1)):
            for B in (1, 4, 16, 64, 256, 512):
                for n in (200, 400, 1000, 1500, 3000, 8000, 32000):
                    for how in ("even", "ragged", "one"):
                        keys = [n] * B
                        if how == "ragged":
                            keys = np.maximum(1, np.exp(r.uniform(np.log(max(1, n // 64)), np.log(n), B))).astype(int).tolist()
                        if how == "one":
                            keys = [min(n, 300)] * (B - 1) + [n]
                        if B * Hkv > 4096 or sum(keys) * Hkv * D > 2**30 or (B == 1 and how != "even"):
                            continue
                        yield "parts", (D, Hq, Hkv, B, 1, n, how, "-"), dict(D=D, Hq=Hq, Hkv=Hkv, keys=keys, queries=[1] * B)
    # Prompts of few tiles.
    for D in (64, 128, 256):
        for Hq, Hkv in ((4, 4), (8, 2), (16, 4)):
            for B in (1, 2, 3, 4):
                for n in (150, 300, 500, 1000, 2000, 3000):
                    yield "parts", (D, Hq, Hkv, B, n, n, "even", "-"), dict(D=D, Hq=Hq, Hkv=Hkv, keys=[n] * B, queries=[n] * B)
    # Several tiles a sequence.
    for D in (64, 128):
        for Hq, Hkv in ((32, 8), (24, 24)):
            for B in (16, 64, 256):
                for q in (5, 8, 17, 32, 64, 100):
                    for n in (100, 1000, 4000):
                        if 16 < q * Hq // Hkv and n >= q and B * Hkv * n * D <= 2**30 and B * q * Hq * n <= 2**30:
                            yield "pairs", (D, Hq, Hkv, B, q, n, "none", "-"), dict(D=D, Hq=Hq, Hkv=Hkv, keys=[n] * B, queries=[q] * B)


def time(w, torch, D, Hq, Hkv, keys, queries, mask="none", slopes=False, group=64, page=64):
    import numpy as np
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(1)
    per = [-(-n // page) for n in keys]
    size = w.kv4_page_bytes(page, D, group)
    caches = [torch.randint(0, 0x38, (sum(per), Hkv, size), dtype=torch.uint8, device=dev, generator=gen) for _ in range(2)]
    table = np.zeros((len(keys), max(per)), np.int32)
    order = np.random.RandomState(1).permutation(sum(per))
    for b, at in enumerate(np.cumsum([0] + per[:-1])):
        table[b, :per[b]] = order[at:at + per[b]]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(dev)  # noqa: E731
    pos = np.concatenate([np.arange(n - q, n) for n, q in zip(keys, queries)])
    first = end = None
    if mask == "given":
        end = i32(pos + 1)
    elif mask.startswith("window"):
        first = i32(pos + 1 - int(mask.split()[1]))
    elif mask.endswith("documents"):
        starts = np.sort(np.append(0, np.random.RandomState(2).randint(0, max(keys), int(mask.split()[0]) - 1)))
        first = i32(starts[np.searchsorted(starts, pos, side="right") - 1])
    q = torch.randn(sum(queries), Hq, D, device=dev, dtype=torch.bfloat16, generator=gen)
    args = (q, *caches, i32(table), i32(keys), i32(np.cumsum([0] + queries)), max(queries), max(keys), group)
    kw = dict(first=first, end=end, slopes=torch.full((Hq,), 0.1, device=dev) if slopes else None)
    w.qmm_kv4_attention(*args, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(10):
            w.qmm_kv4_attention(*args, **kw)
    graph.replay()
    torch.cuda.synchronize()
    s, e = torch.cuda.Event(True), torch.cuda.Event(True)
    times = []
    for _ in range(7):
        s.record()
        graph.replay()
        e.record()
        e.synchronize()
        times.append(s.elapsed_time(e) * 100)
    return sorted(times)[3]


def run(path):
    import torch
    import weight_only_group_amd as w
    w.LIB_PATH = os.path.abspath(path)
    side = os.path.splitext(os.path.basename(path))[0]
    for table, line, kw in shapes():
        if side in TABLES[table]:
            print(table, *line, f"{time(w, torch, **kw):.1f}", sep="\t", flush=True)


def chosen(name, shape):
    """The side that the rules take; None where they take neither."""
    import weight_only_group_amd as w
    D, Hq, Hkv, B, q, n = map(int, shape[:6])
    kernel = w.kv4_attention_plan_info(B, B * q, Hq, Hkv, D, q, n, biased=shape[7] == "distances")["kernel"]
    if name == "blocks":
        return "blocks" if kernel == "blocks" else "rows"
    return {"parts": {"parts": "parts", "tile": "whole", "pair": "whole"}, "pairs": {"pair": "whole", "tile": "single"}}[name].get(kernel)


def table(directory):
    found = {}
    for side in SIDES:
        for line in open(os.path.join(directory, side + ".txt")):
            *shape, t = line.rstrip("\n").split("\t")
            if len(shape) == 9:
                found.setdefault(tuple(shape), {})[side] = float(t)
    print("# Both sides of the choices between the kernels of qmm_kv4_attention, one MI355X, microseconds a call")
    print("# (profiles/cache_attention_choices.py). Scales per 64 channels, pages of 64, bf16; dimensions, query heads, key heads,")
    print("# sequences, new tokens and keys of each (of the longest), mask or lengths, distance bias; the two times, their quotient,")
    print("# and the side that the rules choose (-: another kernel).")
    for name, (a, b) in TABLES.items():
        print(f"\n# {name}: {a}, {b}, {a} / {b}, chosen")
        ratios = []
        for (kind, *shape), t in found.items():
            if kind == name:
                side = chosen(name, shape)
                print(*shape, f"{t[a]:.1f} {t[b]:.1f} {t[a] / t[b]:.2f}", side or "-")
                if side:
                    ratios.append(t[side] / min(t[a], t[b]))
        ratios.sort()
        print(f"# the chosen side over the faster one, {len(ratios)} shapes: mean {sum(ratios) / len(ratios):.3f}, "
              f"90 of 100 below {ratios[len(ratios) * 9 // 10]:.2f}, most {ratios[-1]:.2f}")


if __name__ == "__main__":
    if len(sys.argv) == 3 and sys.argv[1] in ("build", "run", "table"):
        globals()[sys.argv[1]](sys.argv[2])
    else:
        sys.exit(__doc__)
