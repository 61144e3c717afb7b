"""Plain float64 implementations of the layer operators (include/qmm_layer.h),
written from their formulas, token by token and head by head, and bounds on the
rounding errors that a correct kernel may make. Used only by the tests."""
from __future__ import annotations

import numpy as np

from .qmm_oracle import bf16_to_f64, f64_to_bf16, unpack

# Unit roundoff of the output types (half a unit in the last place, relative).
ROUNDOFF = {"fp16": 2.0**-11, "bf16": 2.0**-8}
# Half the spacing of their smallest numbers: the absolute rounding error near zero.
TINY = {"fp16": 2.0**-25, "bf16": 2.0**-134}
F32 = 2.0**-24


def largest(values, k):
    """Indices of the k largest, largest first, equal ones by index."""
    return sorted(range(len(values)), key=lambda i: (-values[i], i))[:k]


# ---- mixture of experts ------------------------------------------------------------

def moe_route(x, router, top_k, renormalize):
    logits = x.astype(np.float64) @ router.astype(np.float64).T
    ids = np.array([largest(row, top_k) for row in logits], dtype=np.int32).reshape(len(x), top_k)
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    chosen = np.take_along_axis(e, ids, axis=1)
    return ids, chosen / (chosen if renormalize else e).sum(axis=1, keepdims=True), logits


def expert_weight(planes, e, K, bits, group_size, offset=128.0):
    """Expert e's dequantised weight (K, N) and |s| (q + |z| + offset), which bounds what a kernel may form of a code."""
    qw, qlo, zeros, scales = planes
    codes = unpack(qw[e], None if qlo is None else qlo[e], bits, K)
    s, z = scales[e].astype(np.float64), zeros[e].astype(np.float64)
    g = np.zeros(K, int) if group_size == -1 else np.arange(K) // group_size
    return s[g] * (codes.astype(np.float64) - z[g]), np.abs(s[g]) * (codes + np.abs(z[g]) + offset)


def silu(g):
    return g / (1 + np.exp(-g))


def moe(x, ids, weights, gate_up, down, bits, group_size, dtype):
    """y in float64, and a bound on the error of one kernel element: fp32 sums of K products err by at most
    K 2^-24 of the sum of their sizes, silu(g) u passes its inputs' errors on with slopes of at most 1.1 |u| and
    |silu(g)|, h is kept to 2^-16, and y is rounded once."""
    x = x.astype(np.float64)
    T, H = x.shape
    I = gate_up[2].shape[2] // 2
    y, err = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < len(gate_up[0]):
                continue
            w, formed = expert_weight(gate_up, e, H, bits, group_size)
            both, slack = x[t] @ w, (H + 8) * F32 * (np.abs(x[t]) @ formed)
            g, u = both[:I], both[I:]
            h = silu(g) * u
            h_err = 1.1 * np.abs(u) * slack[:I] + np.abs(silu(g)) * slack[I:] + 2 * slack[:I] * slack[I:] + 2.0**-15 * np.abs(h)
            w, formed = expert_weight(down, e, I, bits, group_size)
            y[t] += float(weights[t, j]) * (h @ w)
            err[t] += float(weights[t, j]) * (h_err @ np.abs(w) + (I + 8) * F32 * (np.abs(h) @ formed))
    err += 16 * F32 * np.abs(y)
    return y, err + ROUNDOFF[dtype] * (np.abs(y) + err) + TINY[dtype]


def rounded(v, dtype):
    """v rounded to the data type, as float64."""
    return v.astype(np.float16).astype(np.float64) if dtype == "fp16" else bf16_to_f64(f64_to_bf16(v))


def moe_hidden(x, ids, gate_up, bits, group_size, offset=128.0):
    """h of every (token, choice), (T, top_k, I), and per choice the root mean square of a weight and of what a
    kernel may form of one (0 for a choice outside)."""
    x = x.astype(np.float64)
    T, k = ids.shape
    I = gate_up[2].shape[2] // 2
    h, sizes = np.zeros((T, k, I)), np.zeros((T, k, 2))
    for e in np.unique(ids):
        if not 0 <= e < len(gate_up[0]):
            continue
        w, formed = expert_weight(gate_up, e, x.shape[1], bits, group_size, offset)
        t, j = np.nonzero(ids == e)
        both = x[t] @ w
        h[t, j] = silu(both[:, :I]) * both[:, I:]
        sizes[t, j] = np.sqrt([np.mean(w**2), np.mean(formed**2)])
    return h, sizes


def moe_down(h, ids, weights, down, bits, group_size):
    """y of the h of every (token, choice), and the largest ratio of a formed weight to a weight (root mean squares)."""
    T, k, I = h.shape
    y, ratio = np.zeros((T, down[2].shape[2])), 0.0
    for e in np.unique(ids):
        if not 0 <= e < len(down[0]):
            continue
        w, formed = expert_weight(down, e, I, bits, group_size)
        ratio = max(ratio, np.sqrt(np.mean(formed**2) / np.mean(w**2)))
        t, j = np.nonzero(ids == e)
        np.add.at(y, t, weights[t, j][:, None] * (h[t, j] @ w))
    return y, ratio


def moe_norm(x, ids, weights, gate_up, down, bits, group_size, dtype):
    """y in float64, and a limit on |error| / |y| (Euclidean norms over the whole result, of some thousand elements).

    Four independent parts. The result's rounding: that of y itself. h in 16 significant bits: 2^-17 of each. The
    fp32 sums of the two products: a chain of up to 128 sums of formed weights (code, zero point and a kernel's offset
    of up to 128; none in the gate and up products of fp16 data, whose codes are halves as they are) in random directions errs by 2^-24 of each partial sum, together 2^-24 sqrt(128^2 / 2) of one term
    where the products' sum is sqrt(128) of one, so 8 2^-24 of the ratio of formed weights to weights; g and u pass
    that on with a slope of 1.1 and 1, so 1.5 times. A tenth on top for what random directions leave open."""
    h, sizes = moe_hidden(x, ids, gate_up, bits, group_size, 0.0 if dtype == "fp16" else 128.0)
    y, down_ratio = moe_down(h, ids, weights, down, bits, group_size)
    gate_ratio = np.max(sizes[..., 1] / np.maximum(sizes[..., 0], 1e-300))
    own = np.linalg.norm(rounded(y, dtype) - y) / np.linalg.norm(y)
    return y, 1.1 * np.sqrt(own**2 + 2.0**-34 + (12 * F32 * gate_ratio)**2 + (8 * F32 * down_ratio)**2)


# ---- append to the paged cache --------------------------------------------------------

def rotate(x, cos, sin, adjacent):
    """One head's values; and |a c| + |b s| per value, which the fp32 error goes with."""
    x = x.astype(np.float64)
    out, size = x.copy(), np.abs(x)
    half = len(cos)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        c, s = float(cos[i]), float(sin[i])
        out[a], out[b] = x[a] * c - x[b] * s, x[b] * c + x[a] * s
        size[a], size[b] = abs(x[a] * c) + abs(x[b] * s), abs(x[b] * c) + abs(x[a] * s)
    return out, size


def kv_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, adjacent):
    """Rotated q, the caches after the call, and for q and the key cache the sizes that errors go with."""
    page = k_cache.shape[2]
    q_out, q_size = np.zeros(q.shape), np.zeros(q.shape)
    kc, vc, k_size = k_cache.astype(np.float64), v_cache.astype(np.float64), np.zeros(k_cache.shape)
    for t in range(len(q)):
        turn = (lambda h: (h.astype(np.float64), np.zeros(h.shape))) if cos is None else (
            lambda h: rotate(h, cos[positions[t]], sin[positions[t]], adjacent))
        for h in range(q.shape[1]):
            q_out[t, h], q_size[t, h] = turn(q[t, h])
        if not 0 <= slots[t] < k_cache.shape[0] * page:
            continue
        p, i = divmod(int(slots[t]), page)
        for h in range(k.shape[1]):
            kc[p, h, i], k_size[p, h, i] = turn(k[t, h])
            vc[p, h, i] = v[t, h]
    return q_out, kc, vc, q_size, k_size


# ---- attention --------------------------------------------------------------------------

def attention(q, k_cache, v_cache, table, kv_lens, q_starts, scale, softcap=0.0, slopes=None, first=None, end=None,
              dtype="fp16"):
    """out in float64, and a bound on one element's error. An error d of every score changes the result by at most
    2 d of sum p |v| (p the softmax); the weights' rounding by at most 2 roundoffs of it; one rounding at the end."""
    T, Hq, D = q.shape
    page, Hkv = k_cache.shape[2], k_cache.shape[1]
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
                K = k_cache[at[0], h // (Hq // Hkv), at[1]].astype(np.float64)
                V = v_cache[at[0], h // (Hq // Hkv), at[1]].astype(np.float64)
                qh = q[t, h].astype(np.float64)
                s = scale * (K @ qh)
                err = (D + 4) * F32 * abs(scale) * (np.abs(K) @ np.abs(qh))
                if softcap > 0:
                    # A cap's own error goes with the score; up to a cap of 64 a few roundings of the cap may come on top.
                    s = softcap * np.tanh(s / softcap)
                    err = err + 16 * F32 * np.abs(s) + (4 * F32 * softcap if softcap <= 64 else 0.0)
                if slopes is not None:
                    s = s - float(slopes[h]) * np.abs(pos - keys)
                    err = err + 4 * F32 * float(slopes[h]) * np.abs(pos - keys)
                err = err + 8 * F32 * (np.abs(s) + abs(s.max()))
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t, h] = p @ V
                size = p @ np.abs(V)
                moved = ((p * err) @ np.abs(V) + (p @ err) * size) * 1.1
                bound[t, h] = moved + (2 * ROUNDOFF[dtype] + len(keys) * F32 * 4) * size
                bound[t, h] += len(keys) * 2.0**-25 * np.abs(V).max() * p.max() if dtype == "fp16" else 0.0
    return out, bound + ROUNDOFF[dtype] * (np.abs(out) + bound) + TINY[dtype]


# ---- log probabilities ---------------------------------------------------------------------

def logprobs(logits, targets, top):
    """logprob, entropy, top log probabilities, top ids."""
    l = logits.astype(np.float64)
    M, V = l.shape
    logprob, entropy = np.zeros(M), np.zeros(M)
    top_lp, top_ids = np.zeros((M, top)), np.zeros((M, top), np.int32)
    for m in range(M):
        row = l[m]
        order = sorted(range(V), key=lambda i: (0 if np.isnan(row[i]) else 1, 0.0 if np.isnan(row[i]) else -row[i], i))[:top]
        top_ids[m] = order
        mx = row.max()
        if not np.isfinite(mx):  # NaN or +inf somewhere, or -inf everywhere
            lse = entropy[m] = np.nan
        else:
            e = np.exp(row - mx)
            lse = mx + np.log(e.sum())
            p = e / e.sum()
            some = p > 0
            entropy[m] = -np.sum(p[some] * (row[some] - lse))
        top_lp[m] = row[order] - lse
        if targets is not None:
            t = int(targets[m])
            logprob[m] = 0.0 if t < 0 else np.nan if t >= V else row[t] - lse
    return logprob, entropy, top_lp, top_ids
