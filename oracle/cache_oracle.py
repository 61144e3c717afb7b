"""Plain implementations of the 4-bit cache and of the care of pages (include/qmm_cache.h), written from their
definitions, and bounds on the rounding errors that a correct kernel may make. Used only by the tests."""
from __future__ import annotations

import numpy as np

from .layer_oracle import F32, ROUNDOFF, TINY, rotate
from .qmm_oracle import bf16_to_f64, f64_to_bf16

LARGEST, LARGEST_SCALE = 16384.0, 2728.0
BLOCK = 8  # tokens of a head that lie interleaved


def block_bytes(D, group):
    return 4 * D + 32 * D // group


def quantise(x, group):
    """Scales, middles (float16) and codes of x (..., D), in the definition's fp32 steps."""
    f32 = np.float32
    x = np.asarray(x, f32)
    x = x.reshape(*x.shape[:-1], -1, group)
    nan = np.isnan(x).any(axis=-1)
    x = np.clip(np.where(np.isnan(x), f32(0), x), f32(-LARGEST), f32(LARGEST))
    lo, hi = x.min(axis=-1), x.max(axis=-1)
    s = bf16_to_f64(f64_to_bf16(((hi - lo) / f32(15)).astype(np.float64))).astype(np.float16)
    m = (lo + f32(8) * s.astype(f32)).astype(np.float16)
    step = np.where(s > 0, s, np.float16(1)).astype(f32)[..., None]
    c = np.clip(np.rint((x - m.astype(f32)[..., None]) / step), -8, 7)
    c = np.where((s > 0)[..., None] & ~nan[..., None], c, 0).astype(np.int64) + 8
    s, m = (np.where(nan, np.float16(np.nan), t) for t in (s, m))
    return s, m, c.reshape(*c.shape[:-2], -1)


# ---- a block's bytes, place by place -----------------------------------------------------

def key_place(t, d, D):
    """Byte and nibble of it of channel d of token t in a block of keys."""
    i, g, e = d // 32, d % 32 // 8, d % 8
    nibble = e // 2 if e % 2 == 0 else 4 + e // 2
    return t * (D // 2) + 4 * ((D // 32) * g + i) + nibble // 2, nibble % 2


def value_place(t, d, D):
    n, r = divmod(d, 4)
    return 2 * (8 * n + t) + r // 2, r % 2


def scale_places(t, g, D, group, keys):
    """Byte offsets of the scale and the middle of token t's group g."""
    G = D // group
    if keys:
        return 4 * D + 2 * (t * 2 * G + g), 4 * D + 2 * (t * 2 * G + G + g)
    return 4 * D + 2 * (g * 2 * BLOCK + t), 4 * D + 2 * (g * 2 * BLOCK + BLOCK + t)


def put(cache, page, head, at, s, m, c, group, keys):
    """Writes one token's head into a cache (pages, Hkv, bytes) of uint8."""
    D = len(c)
    block = cache[page, head][at // BLOCK * block_bytes(D, group):][:block_bytes(D, group)]
    t = at % BLOCK
    for d in range(D):
        byte, half = (key_place if keys else value_place)(t, d, D)
        block[byte] = block[byte] & (0xF0 if half == 0 else 0x0F) | int(c[d]) << (4 * half)
    for g in range(D // group):
        for place, v in zip(scale_places(t, g, D, group, keys), (s[g], m[g])):
            block[place:place + 2] = np.frombuffer(np.float16(v).tobytes(), np.uint8)


def parts(cache, D, group, keys):
    """(pages, Hkv, page_size, D) float64: s (c - 8) and m of every channel; NaN in both where either
    is not finite or the scale is too large."""
    pages, heads, size = cache.shape
    blocks = cache.reshape(pages, heads, -1, block_bytes(D, group))
    step, middle = (np.zeros((pages, heads, blocks.shape[2], BLOCK, D)) for _ in range(2))
    for t in range(BLOCK):
        for g in range(D // group):
            s, m = (np.ascontiguousarray(blocks[..., p:p + 2]).view(np.float16)[..., 0].astype(np.float64)
                    for p in scale_places(t, g, D, group, keys))
            bad = ~((np.abs(s) <= LARGEST_SCALE) & np.isfinite(m))
            s, m = np.where(bad, np.nan, s), np.where(bad, np.nan, m)
            for d in range(g * group, (g + 1) * group):
                byte, half = (key_place if keys else value_place)(t, d, D)
                step[..., t, d] = s * ((blocks[..., byte] >> (4 * half) & 15).astype(np.float64) - 8)
                middle[..., t, d] = m
    shape = (pages, heads, blocks.shape[2] * BLOCK, D)
    return step.reshape(shape), middle.reshape(shape)


def append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, group, page, adjacent):
    """Rotated q (float64) and the sizes that its error goes with; the caches' bytes are written in place. A key is
    rotated in float64 and rounded once to fp32."""
    q_out, q_size = np.zeros(q.shape), np.zeros(q.shape)
    for t in range(len(q)):
        turn = (lambda h: (h.astype(np.float64), np.zeros(h.shape))) if cos is None else (
            lambda h: rotate(h, cos[positions[t]], sin[positions[t]], adjacent))
        for h in range(q.shape[1]):
            q_out[t, h], q_size[t, h] = turn(q[t, h])
        if not 0 <= slots[t] < len(k_cache) * page:
            continue
        p, at = divmod(int(slots[t]), page)
        for h in range(k.shape[1]):
            put(k_cache, p, h, at, *quantise(turn(k[t, h])[0], group), group, True)
            put(v_cache, p, h, at, *quantise(v[t, h], group), group, False)
    return q_out, q_size


# ---- attention -----------------------------------------------------------------------------

WEIGHTS = 2.0**-11  # half a step of the weights, fp16 whatever the data


def attention(q, k_parts, v_parts, table, kv_lens, q_starts, scale, group, softcap=0.0, slopes=None, first=None, end=None,
              dtype="fp16"):
    """out in float64, and a bound on one element's error; k_parts and v_parts as parts() gives them.

    Scores: fp32 sums of D + 3 groups products of the parts' sizes; the query, scaled to a largest value in [1, 2), has
    fp16's spacing of 2^-24 where it is small, and so do its groups' sums. An error d of every score changes the result by
    at most 2 d of sum p |v|. The weights' rounding by at most 2 half steps of that, and by 2^-32 of the largest
    weight where they are small (the largest is kept as 2^7 at least, half of fp16's smallest step is 2^-25); fp32 sums of
    the parts' sizes; one rounding of the result."""
    T, Hq, D = q.shape
    page, Hkv = k_parts[0].shape[2], k_parts[0].shape[1]
    out, bound = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(len(kv_lens)):
        n, q0, q1 = int(kv_lens[b]), int(q_starts[b]), int(q_starts[b + 1])
        for t in range(q0, q1):
            pos = n - (q1 - q0) + t - q0
            lo = 0 if first is None else max(0, int(first[t]))
            hi = min(n, pos + 1 if end is None else int(end[t]))
            if lo >= hi:
                continue
            keys = np.arange(lo, hi)
            at = (table[b, keys // page], keys % page)
            for h in range(Hq):
                ks, km = (x[at[0], h // (Hq // Hkv), at[1]] for x in k_parts)
                vs, vm = (x[at[0], h // (Hq // Hkv), at[1]] for x in v_parts)
                qh = q[t, h].astype(np.float64)
                s = scale * ((ks + km) @ qh)
                sizes = np.abs(ks) + np.abs(km)
                err = (D + 3 * D // group + 16) * F32 * abs(scale) * (sizes @ np.abs(qh))
                err = err + abs(scale) * np.abs(qh).max() * 2.0**-24 * sizes.sum(axis=1)
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                    err = err + 16 * F32 * np.abs(s) + (4 * F32 * softcap if softcap <= 64 else 0.0)
                if slopes is not None:
                    s = s - float(slopes[h]) * np.abs(pos - keys)
                    err = err + 4 * F32 * float(slopes[h]) * np.abs(pos - keys)
                err = err + 8 * F32 * (np.abs(s) + abs(s.max()))
                p = np.exp(s - s.max())
                p /= p.sum()
                V = vs + vm
                out[t, h] = p @ V
                size = p @ np.abs(V)
                moved = ((p * err) @ np.abs(V) + (p @ err) * size) * 1.1
                whole = p @ (np.abs(vs) + np.abs(vm))
                bound[t, h] = moved + 2 * WEIGHTS * size + len(keys) * F32 * 4 * whole
                bound[t, h] += 2 * len(keys) * 2.0**-32 * np.abs(V).max() * p.max()
    return out, bound + ROUNDOFF[dtype] * (np.abs(out) + bound) + TINY[dtype]


# ---- the care of pages ------------------------------------------------------------------------

def copy_pages(cache, src, dst):
    out = cache.copy()
    for a, b in zip(src, dst):
        if 0 <= a < len(cache) and 0 <= b < len(cache):
            out[b] = cache[a]
    return out


def compact(pages, table, kv_lens, page_size):
    """The renamed table, where each page goes (-1: free), the number in use, and the copies (from, to)."""
    used = set()
    for row, n in zip(table, kv_lens):
        used |= {int(p) for p in row[:max(0, -(-int(n) // page_size))] if 0 <= p < pages}
    live = len(used)
    free = [p for p in range(live) if p not in used]
    high = sorted(p for p in used if p >= live)
    moved_to = np.full(pages, -1, np.int32)
    for p in used:
        moved_to[p] = p
    moved_to[high] = free
    new = table.copy()
    for b, n in enumerate(kv_lens):
        for i in range(min(table.shape[1], max(0, -(-int(n) // page_size)))):
            if 0 <= table[b, i] < pages:
                new[b, i] = moved_to[table[b, i]]
    return new, moved_to, live, high, free
