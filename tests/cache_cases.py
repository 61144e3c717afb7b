"""Inputs shared by the GPU tests of the 4-bit cache."""
import numpy as np
import torch

from layer_cases import DEV
from oracle import cache_oracle as co


def device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def filled(pages, Hkv, page, D, group, keys, seed, scale=1.0, fill=None, used=None):
    """A cache's bytes: random codes, scales and middles as normal values of size `scale` give them; where `used` (pages,
    page) is False scales and middles are `fill`."""
    r = np.random.default_rng(seed)
    G, size = D // group, co.block_bytes(D, group)
    cache = r.integers(0, 256, (pages, Hkv, page // 8, size)).astype(np.uint8)
    x = r.standard_normal((pages, Hkv, page // 8, 8, G, 16)).astype(np.float32) * scale
    s = r.uniform(0.2, 0.4, x.shape[:-1]) * scale
    s = co.bf16_to_f64(co.f64_to_bf16(s)).astype(np.float16)
    m = (x[..., 0] * 0.3).astype(np.float16)
    if fill is not None:
        places = used.reshape(pages, 1, page // 8, 8, 1)
        s, m = (np.where(places, t, np.float16(fill)) for t in (s, m))
    for t in range(8):
        for g in range(G):
            for at, v in zip(co.scale_places(t, g, D, group, keys), (s, m)):
                cache[..., at:at + 2] = np.ascontiguousarray(v[..., t, g])[..., None].view(np.uint8)
    return cache.reshape(pages, Hkv, -1)


def paged4(kv_lens, Hkv, D, page, group, seed, spare=3, fill=None, scale=1.0):
    """Key and value cache (bytes, numpy) with the sequences' pages in any order, and the page table."""
    r = np.random.default_rng(seed)
    per = [-(-n // page) for n in kv_lens]
    pages = sum(per) + spare
    order = r.permutation(pages)
    table = np.full((len(kv_lens), max(1, max(per))), pages - 1 if fill is None else 0, np.int32)
    used = np.zeros((pages, page), bool)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
        j = np.arange(kv_lens[b])
        used[table[b, j // page], j % page] = True
    return (filled(pages, Hkv, page, D, group, True, seed + 1, scale, fill, used),
            filled(pages, Hkv, page, D, group, False, seed + 2, scale, fill, used), table)
