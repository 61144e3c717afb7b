"""Inputs and comparisons shared by the GPU tests of the layer operators."""
import sys

import numpy as np
import torch

DEV = "cuda:0"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(shape, dtype, seed, scale=1.0):
    return (torch.randn(shape, generator=gen(seed)) * scale).to(TYPES[dtype]).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, want, bound, what):
    """Every element within its bound, non-finite ones equal."""
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: infinities differ"
    err, lim = np.abs(got - want)[fine], np.broadcast_to(bound, want.shape)[fine]
    if err.size:
        bad = err > lim
        ratio = float(np.max(err / np.maximum(lim, 1e-300)))
        say(f"{what}: max err/bound {ratio:.3f}")
        assert not bad.any(), f"{what}: {int(bad.sum())} of {err.size} off, worst {ratio:.2f} of the bound"


def expert_planes(E, K, N, bits, gs, dtype, strips, seed, zeros="integer"):
    """E random packed weights: (device tuple for the call, numpy K-major tuple for the oracle)."""
    import oracle
    r = np.random.default_rng(seed)
    rows, rows_lo = (K // 16, K // 32) if bits == 3 else (K * bits // 32, 0)
    words = lambda n: r.integers(-2**31, 2**31, (E, n, N), dtype=np.int64).astype(np.int32)  # noqa: E731
    qw, qlo = words(rows), words(rows_lo) if bits == 3 else None
    groups = 1 if gs == -1 else K // gs
    z = r.integers(0, 2**bits, (E, groups, N)).astype(np.float32)
    if zeros == "fraction":
        z = z + r.uniform(-1, 1, z.shape).astype(np.float32)
    s = r.uniform(0.5, 1.5, z.shape).astype(np.float32) / np.sqrt((4.0**bits - 1) / 6 * K)
    z, s = (torch.from_numpy(a.astype(np.float32)).to(TYPES[dtype]).to(DEV) for a in (z, s))
    place = lambda w: None if w is None else torch.from_numpy(  # noqa: E731
        np.stack([oracle.to_strips(e) for e in w]) if strips else w).to(DEV)
    return (place(qw), place(qlo), z, s), (qw, qlo, f64(z), f64(s))


def paged(B, kv_lens, Hkv, D, page, dtype, seed, spare=3, fill=None):
    """Caches with the sequences' pages in any order; places past a sequence's end (and spare pages) hold `fill`."""
    r = np.random.default_rng(seed)
    per = [-(-n // page) for n in kv_lens]
    pages = sum(per) + spare
    order = r.permutation(pages)
    table = np.full((B, max(1, max(per))), pages - 1 if fill is None else 0, np.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    k, v = (torch.from_numpy(r.standard_normal((pages, Hkv, page, D)).astype(np.float32)) for _ in range(2))
    if fill is not None:
        used = np.zeros((pages, page), bool)
        for b, n in enumerate(kv_lens):
            j = np.arange(n)
            used[table[b, j // page], j % page] = True
        for t in (k, v):
            t.permute(0, 2, 1, 3)[torch.from_numpy(~used)] = fill
    return k.to(TYPES[dtype]).to(DEV), v.to(TYPES[dtype]).to(DEV), table


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)
