"""The shares that the blocks of qmm_kv4_attention find in parts of the keys (share_of in csrc/kv4_attention.hip), done over
on the host step by step in fp32 for random lengths: as many blocks as the host launches at most, and every part of every
tile has one. Blocks that were counted but not launched would leave a tile without its join."""
import numpy as np
import pytest

from test_layer_host import _lib

F = np.float32
CHUNK, ROWS, LEAST_CHUNKS, MOST_PARTS = 32, 16, 4, 256


def wave_sum(v):
    """Of 64 lanes, in the order of the device's steps: within rows of sixteen, then from row to row."""
    v = v.astype(F)
    for shift in (1, 2, 4, 8):
        rows = v.reshape(4, 16)
        moved = np.zeros_like(rows)
        moved[:, shift:] = rows[:, :-shift]
        v = (rows + moved).reshape(64)
    v = v.copy()
    last = v[[15, 47]]
    v[16:32] += last[0]
    v[48:64] += last[1]
    v[32:64] += v[31]
    return v[63]


def divided_up(n, d):
    """The device's n / d rounded up, of a quotient that may be off by one."""
    inverse = F(1) / F(d)
    q = (n.astype(F) * inverse).astype(np.int64)
    q -= q * d > n
    q += q * d < n
    return q + (q * d < n)


def shares(p, kv_lens, q_lens, group, Hkv):
    """Tiles, chunks a part and parts of each sequence."""
    rows = np.asarray(q_lens) * group
    tiles = np.maximum(-(-rows // ROWS), 1) * Hkv
    chunks = np.where(rows > 0, -(-np.asarray(kv_lens, np.int64) // CHUNK), 0)
    B = len(rows)
    per = -(-B // 64)
    own = np.zeros((64, per), np.int64)
    at = np.arange(B)
    work = np.zeros((64, per), F)
    work.reshape(-1)[at] = tiles.astype(F) * chunks.astype(F)
    lanes = np.zeros(64, F)
    for i in range(per):
        lanes = lanes + work[:, i]
    work = wave_sum(lanes)
    wanted, tries = work / F(p["resident"]), 0
    for i in range(5):
        if i == 4:
            wanted = work / F(p["parts"])
        c = max(int(wanted * F(1.00001)) + 1, LEAST_CHUNKS)
        parts = np.minimum(np.maximum(divided_up(chunks, c), 1), MOST_PARTS)
        own.reshape(-1)[at] = parts * tiles
        tries, total = i + 1, int(own.sum())
        if total <= p["resident"]:
            break
        wanted = F(c) * max(F(total) / F(p["resident"]), F(1.03))
    return tiles, parts, own, total, tries


def share_of(ids, tiles, parts, own, Hkv):
    """(b, part, key head, row tile, block of part 0, step) of the blocks."""
    per = own.shape[1]
    blocks = own.sum(axis=1)
    ends = np.cumsum(blocks)
    lane = np.searchsorted(ends, ids, side="right")  # the first whose blocks reach past the id
    at, b = ends[lane] - blocks[lane], lane * per
    for _ in range(1, per):
        size = parts[np.minimum(b, len(parts) - 1)] * tiles[np.minimum(b, len(parts) - 1)]
        on = ids >= at + size
        at, b = np.where(on, at + size, at), np.where(on, b + 1, b)
    off, rtiles = ids - at, tiles[b] // Hkv
    step = rtiles * Hkv
    part = off // step
    rest = off - part * step
    return b, part, rest // rtiles, rest % rtiles, ids - part * step, step


def lengths(r, B, most, how):
    if how == "even":
        return np.full(B, most)
    if how == "one":
        return np.where(np.arange(B) == r.integers(B), most, min(most, 40))
    n = np.exp(r.uniform(0, np.log(most), B)).astype(np.int64)
    n[r.random(B) < 0.1] = 0
    return n


@pytest.mark.parametrize("how", ["even", "ragged", "one"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_every_part_has_a_block(D, how):
    import weight_only_group_amd as w
    _lib()
    r = np.random.default_rng(D)
    taken, longest = 0, 0
    for B in (1, 2, 5, 17, 63, 64, 65, 127, 130, 500, 511, 1000, 1023, 1024):
        for Hkv, group, max_q in ((1, 1, 1), (1, 8, 1), (2, 4, 3), (8, 4, 1), (4, 5, 40), (3, 1, 700)):
            for max_kv in (1100, 4200, 20000, 131072, (1 << 31) - 1):
                q_lens = np.where(r.random(B) < 0.1, 0, np.full(B, max_q) if how == "even" else r.integers(1, max_q + 1, B))
                kv_lens = lengths(r, B, max_kv, how)
                p = w.kv4_attention_plan_info(B, max(int(q_lens.sum()), 1), Hkv * group, Hkv, D, max_q, max_kv)
                if p["kernel"] != "parts":
                    continue
                taken += 1
                tiles, parts, own, total, tries = shares(p, kv_lens, q_lens, group, Hkv)
                longest = max(longest, tries)
                assert total <= p["blocks"], (B, Hkv, group, max_q, max_kv)
                ids = np.arange(total)
                b, part, hk, rt, first, step = share_of(ids, tiles, parts, own, Hkv)
                assert (b < B).all() and (part < parts[b]).all() and (hk < Hkv).all()
                every = {*zip(b.tolist(), part.tolist(), hk.tolist(), rt.tolist())}
                assert len(every) == total == int((parts * tiles).sum())  # each once
                # The join's slots: the parts of a tile, a step apart.
                same = share_of(first + part * step, tiles, parts, own, Hkv)
                assert all((x == y).all() for x, y in zip(same, (b, part, hk, rt, first, step)))
                start = share_of(first, tiles, parts, own, Hkv)
                assert (start[1] == 0).all() and all((x == y).all() for x, y in zip((start[0], *start[2:4]), (b, hk, rt)))
    assert taken > 50 and longest == 5


def test_quotients_rounded_up():
    r = np.random.default_rng(1)
    for _ in range(200):
        d = int(np.exp(r.uniform(np.log(4), np.log(2**20))))
        n = np.unique(np.concatenate([r.integers(0, min(2**26, d * 2**18), 500), np.arange(0, 20) * d, np.arange(1, 20) * d - 1, np.arange(20) * d + 1]))
        n = n[n <= 2**26]
        assert (divided_up(n, d) == -(-n // d)).all(), d
    n = np.arange(2**26 - 1000, 2**26 + 1)  # far past the most parts: near is enough
    assert (divided_up(n, 4) > MOST_PARTS).all()
