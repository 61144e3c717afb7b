"""A key/value cache held in 4 bits and the care of its pages, as cases to measure: the append that quantises
keys and values on their way into the pages, reading tokens back to 16 bits, the attention to such a cache, the
copy of pages (forked sequences), and the compaction of the pages in use.

``run`` computes a case in elementary torch operations in 32 bits (``own`` false) or through the framework's entry
points (``own`` true), on the same state.

The cache: (pages, Hkv, page_size (D / 2 + 4 D / group)) bytes. A head's tokens of a page lie in blocks of eight,
one behind another; each has scale s and middle m per group of channels (fp16), and a value is m + s (code - 8).
A block of keys: (8 tokens, D / 8) words, then (8 tokens, [s, m], groups). Word (D / 32) g + i of a key has channels
32 i + 8 g to 32 i + 8 g + 7, the even ones in its low half, the odd ones in its high half. A block of values:
(D / 4, 8 tokens) 16-bit words of four channels, then (groups, [s, m], 8 tokens).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
LARGEST = 16384.0  # keys and values are cut to this size


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # the new tokens of a small decode batch, and the read-back of what they became
        _append("kv4_append_decode_7", T=7, Hq=32, Hkv=8, D=128, R=128, page=16, group=64, dtype="bf16"),
        # a long prompt, some of its tokens not kept, half of each head rotated in adjacent pairs
        _append("kv4_append_prompt", T=16381, Hq=24, Hkv=4, D=64, R=32, page=64, group=32, dtype="fp16", adjacent=True,
                skip=True),
        # a shared prefix read back whole
        _gather("kv4_gather_prefix", T=50021, Hkv=8, D=128, page=64, group=128, dtype="bf16"),
        # one sequence decoding on a short context: latency
        _attn("kv4_attn_decode_1", B=1, q="one", kv=1500, Hq=32, Hkv=8, D=128, page=16, group=32, dtype="bf16"),
        # a decode batch of very different lengths, scores capped, a sliding window
        _attn("kv4_attn_decode_48", B=48, q="one", kv=8192, Hq=32, Hkv=8, D=128, page=64, group=64, dtype="fp16", cap=50.0,
              window=4096),
        # what the small cache is for: few sequences on very long contexts
        _attn("kv4_attn_decode_long", B=3, q="one", kv=131071, Hq=32, Hkv=8, D=128, page=128, group=128, dtype="bf16"),
        # a long prompt at once, scores capped
        _attn("kv4_attn_prompt_8192", B=1, q="all", kv=8192, Hq=32, Hkv=8, D=128, page=128, group=64, dtype="bf16", cap=30.0),
        # prompts of several documents after a shared context, with a distance bias and a two-way prefix; rows without keys
        _attn("kv4_attn_documents", B=6, q="part", kv=2600, Hq=24, Hkv=24, D=64, page=24, group=32, dtype="fp16", slopes=True,
              docs=True, prefix=True),
        # sequences forked for a search: the last page of each is copied, in every layer's caches
        _copy("kv_fork_5", n=5, pages=512, caches=16, Hkv=8, page=16, D=128, group=64),
        # a prefix copied for another owner, 16-bit caches
        _copy("kv_copy_1531", n=1531, pages=4096, caches=4, Hkv=8, page=16, D=128, group=0),
        # a cache of many finished sequences, packed to its low pages
        _compact("kv_compact_6000", B=37, pages=6000, live=0.55, caches=4, Hkv=8, page=16, D=128, group=64, shared=0.2),
        # few sequences left in a small pool, one layer's caches
        _compact("kv_compact_64", B=3, pages=64, live=0.4, caches=2, Hkv=8, page=16, D=128, group=32, shared=0.0),
    ]


def _append(name, T, Hq, Hkv, D, R, page, group, dtype, adjacent=False, skip=False):
    return dict(name=name, op="append", T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, page=page, group=group, dtype=dtype,
                adjacent=adjacent, skip=skip)


def _gather(name, T, Hkv, D, page, group, dtype):
    return dict(name=name, op="gather", T=T, Hkv=Hkv, D=D, page=page, group=group, dtype=dtype)


def _attn(name, B, q, kv, Hq, Hkv, D, page, group, dtype, cap=0.0, window=0, slopes=False, docs=False, prefix=False, mix=1):
    return dict(name=name, op="attn", B=B, q=q, kv=kv, Hq=Hq, Hkv=Hkv, D=D, page=page, group=group, dtype=dtype, cap=cap,
                window=window, slopes=slopes, docs=docs, prefix=prefix, mix=mix)


def _copy(name, n, pages, caches, Hkv, page, D, group):
    return dict(name=name, op="copy", n=n, pages=pages, caches=caches, Hkv=Hkv, page=page, D=D, group=group)


def _compact(name, B, pages, live, caches, Hkv, page, D, group, shared, mix=1):
    return dict(name=name, op="compact", B=B, pages=pages, live=live, caches=caches, Hkv=Hkv, page=page, D=D, group=group,
                shared=shared, mix=mix)


def _log_between(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["append", "append", "gather", "attn", "attn", "attn", "attn", "copy", "compact"])
    dtype = rng.choice(["fp16", "bf16"])
    D = rng.choice([64, 128, 128, 256])
    group = rng.choice([g for g in (32, 64, 128) if g <= D])
    page = 8 * rng.choice([1, 2, 3, 8, 16])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    if op == "append":
        T = _log_between(rng, 1, 16384)
        Hq = Hkv * rng.choice([1, 2, 5, 8])
        while T * (Hq + 2 * Hkv) * D > 16381 * 32 * 64:
            T = max(1, T // 2)
        case = _append("", T, Hq, Hkv, D, rng.choice([D, D // 2]), page, group, dtype, rng.random() < 0.5, rng.random() < 0.5)
    elif op == "gather":
        T = min(_log_between(rng, 1, 50000), 50021 * 8 * 128 // (Hkv * D))
        case = _gather("", T, Hkv, D, page, group, dtype)
    elif op == "attn":
        q = rng.choice(["one", "one", "few", "part", "all"])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        B = _log_between(rng, 1, 48 if q in ("one", "few") else 6)
        kv = _log_between(rng, 1, 100000 if q == "one" and rng.random() < 0.3 else 8192)
        while B * kv * Hkv * D > 48 * 8192 * 8 * 128:
            kv //= 2
        if q in ("part", "all"):
            while B * Hq * D * kv * kv > 16 * 128 * 8192 * 8192:
                kv //= 2
        docs = q in ("part", "all") and rng.random() < 0.5
        case = _attn("", B, q, kv, Hq, Hkv, D, page, group, dtype, rng.choice([0.0, 0.0, 20.0, 50.0]),
                     0 if docs else rng.choice([0, 0, _log_between(rng, 16, 4096)]), rng.random() < 0.3, docs,
                     rng.random() < 0.3, rng.randint(1, 1 << 20))
    else:
        group = rng.choice([0, group])
        caches = rng.randint(1, 16)
        size = Hkv * page * (2 * D if group == 0 else D // 2 + 4 * D // group)
        most = min(20000, 600_000_000 // (size * caches))  # bytes of all caches
        pages = _log_between(rng, 8, max(9, most))
        if op == "copy":
            case = _copy("", _log_between(rng, 1, pages // 2), pages, caches, Hkv, page, D, group)
        else:
            B = min(_log_between(rng, 1, 64), pages // 8)
            case = _compact("", B, pages, round(rng.uniform(0.1, 0.95), 3), caches, Hkv, page, D, group,
                            rng.choice([0.0, 0.3]), rng.randint(1, 1 << 20))
    del case["name"]
    return case


# ---- the cache's bytes ------------------------------------------------------------

def _quantised(x, group):
    """Scales and middles (fp16) of the groups of x's (..., D) float32, and the codes (uint8)."""
    x = x.clamp(-LARGEST, LARGEST).unflatten(-1, (-1, group))
    lowest, highest = x.amin(dim=-1), x.amax(dim=-1)
    # (a tensor of 15s: by a number torch multiplies with the inverse, which breaks ties.) 8 bits: products with codes
    # are exact in fp16.
    s = ((highest - lowest) / torch.full_like(lowest, 15.0)).to(torch.bfloat16).to(torch.float16)
    m = (lowest + 8 * s.float()).to(torch.float16)
    q = (x - m.float().unsqueeze(-1)) / s.float().unsqueeze(-1)
    q = torch.where(s.unsqueeze(-1) > 0, q.round().clamp(-8, 7), 0.0)
    return s, m, (q + 8).to(torch.uint8).flatten(-2)


_NIBBLES = [0, 2, 4, 6, 1, 3, 5, 7]  # of a word of keys: the even channels of eight, then the odd ones


def _key_bytes(codes):
    """(..., D) codes -> the D / 2 bytes of a key."""
    c = codes.unflatten(-1, (-1, 4, 8)).transpose(-3, -2)[..., _NIBBLES].flatten(-3).unflatten(-1, (-1, 2))
    return c[..., 0] | c[..., 1] << 4


def _key_codes(b):
    """(..., D / 2) bytes -> codes."""
    c = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)
    back = [_NIBBLES.index(e) for e in range(8)]
    return c.unflatten(-1, (4, -1, 8))[..., back].transpose(-3, -2).flatten(-3)


def _planes(cache, D, group, keys):
    """Views of a cache's codes and of its scales and middles, per block of eight tokens."""
    blocks = cache.view(*cache.shape[:2], -1, 4 * D + 32 * D // group)
    codes, rest = blocks[..., :4 * D], blocks[..., 4 * D:].view(torch.float16)
    if keys:  # (pages, Hkv, blocks, tokens, D / 2), (pages, Hkv, blocks, tokens, 2, groups)
        return codes.unflatten(-1, (8, D // 2)), rest.unflatten(-1, (8, 2, D // group))
    return codes.unflatten(-1, (D // 4, 8, 2)), rest.unflatten(-1, (D // group, 2, 8))


def _put(k_cache, v_cache, k, v, slots, page, group):
    """Quantises k and v (T, Hkv, D) float32 into the slots."""
    at = (slots // page, slots % page // 8, slots % 8)
    D = k.shape[2]
    codes, rest = _planes(k_cache, D, group, True)
    s, m, c = _quantised(k, group)
    codes[at[0], :, at[1], at[2]] = _key_bytes(c)
    rest[at[0], :, at[1], at[2]] = torch.stack([s, m], dim=2)
    codes, rest = _planes(v_cache, D, group, False)
    s, m, c = _quantised(v, group)
    c = c.unflatten(-1, (-1, 2, 2))
    codes[at[0], :, at[1], :, at[2]] = c[..., 0] | c[..., 1] << 4
    rest[at[0], :, at[1], :, :, at[2]] = torch.stack([s, m], dim=3)


def _taken(k_cache, v_cache, slots, page, D, group):
    """k and v (T, Hkv, D) float32 of the slots."""
    at = (slots // page, slots % page // 8, slots % 8)
    codes, rest = _planes(k_cache, D, group, True)
    rest = rest[at[0], :, at[1], at[2]].float().unsqueeze(-1)
    k = rest[:, :, 1] + rest[:, :, 0] * (_key_codes(codes[at[0], :, at[1], at[2]]).float().unflatten(-1, (-1, group)) - 8)
    codes, rest = _planes(v_cache, D, group, False)
    b = codes[at[0], :, at[1], :, at[2]]
    rest = rest[at[0], :, at[1], :, :, at[2]].float().unsqueeze(-1)
    v = torch.stack([b & 15, b >> 4], dim=-1).flatten(-3).float().unflatten(-1, (-1, group))
    v = rest[:, :, :, 1] + rest[:, :, :, 0] * (v - 8)
    return k.flatten(-2), v.flatten(-2)


def _page_bytes(c):
    return c["page"] * (c["D"] // 2 + 4 * c["D"] // c["group"])


def _new_cache(c, pages):
    return torch.zeros((pages, c["Hkv"], _page_bytes(c)), dtype=torch.uint8, device=DEV)


# ---- what a case is made of -----------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def prepare(case, seed):
    state = {"append": _prepare_append, "gather": _prepare_gather, "attn": _prepare_attn, "copy": _prepare_copy,
             "compact": _prepare_compact}[case["op"]](case, _gen(seed))
    state["case"] = case
    return state


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _heads(c, g, n, scale=1.0):
    """n tokens' (Hkv, D) of the data type; keys have channels of other sizes and middles, as learnt ones have."""
    wide = torch.exp(0.5 * _randn((c["Hkv"], c["D"]), g))
    return ((_randn((n, c["Hkv"], c["D"]), g) + 0.5 * _randn((c["Hkv"], c["D"]), g)) * wide * scale).to(TYPES[c["dtype"]])


def _prepare_append(c, g):
    dtype = TYPES[c["dtype"]]
    T, Hq, Hkv, D, R = c["T"], c["Hq"], c["Hkv"], c["D"], c["R"]
    # One product gives q, k and v; the three are views into its rows.
    qkv = _randn((T, (Hq + 2 * Hkv) * D), g).to(dtype)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    start = int(torch.randint(0, 1000, (1,), generator=g, device=DEV))
    angles = torch.arange(T + 1000, device=DEV).double()[:, None] * (10000.0 ** (-torch.arange(R // 2, device=DEV).double() * 2 / R))
    pages = (T + 100) // c["page"] + 2
    slots = torch.randperm(pages * c["page"], generator=g, device=DEV)[:T] if T < 64 else _paged_slots(c, g, pages)
    if c["skip"]:
        slots = torch.where(torch.rand(T, generator=g, device=DEV) < 0.1, -1, slots)
    return dict(q=q, k=k, v=v, cos=angles.cos().float(), sin=angles.sin().float(),
                positions=torch.arange(start, start + T, device=DEV, dtype=torch.int32), slots=slots.to(torch.int64),
                k_cache=_new_cache(c, pages), v_cache=_new_cache(c, pages))


def _paged_slots(c, g, pages):
    """Consecutive places in pages that lie in any order."""
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(c["T"], device=DEV)
    return order[at // c["page"]] * c["page"] + at % c["page"]


def _prepare_gather(c, g):
    pages = (c["T"] + 100) // c["page"] + 2
    k_cache, v_cache, slots = _new_cache(c, pages), _new_cache(c, pages), _paged_slots(c, g, pages)
    for part in slots.split(1 << 15):
        _put(k_cache, v_cache, _heads(c, g, len(part)).float(), _heads(c, g, len(part)).float(), part, c["page"], c["group"])
    return dict(k_cache=k_cache, v_cache=v_cache, slots=slots)


def _lengths(c):
    """Per sequence: cached keys (new ones included) and new tokens. They go by the case alone."""
    r = np.random.RandomState(c["mix"])
    B, kv = c["B"], c["kv"]
    kv_lens = np.maximum(1, np.exp(r.uniform(math.log(max(1, kv // 64)), math.log(kv), B)).astype(np.int64))
    kv_lens[r.randint(B)] = kv
    if c["q"] == "one":
        q_lens = np.ones(B, np.int64)
    elif c["q"] == "few":
        q_lens = np.minimum(kv_lens, r.randint(1, 9, B))
    elif c["q"] == "all":
        q_lens = kv_lens.copy()
    else:
        q_lens = np.maximum(1, (kv_lens * r.uniform(0.2, 0.8, B)).astype(np.int64))
    return kv_lens, q_lens


def _visible(c):
    """Per new token: its position, and the first and past-the-last key that it sees."""
    r = np.random.RandomState(c["mix"] + 1)
    kv_lens, q_lens = _lengths(c)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])
    first, end = np.zeros_like(pos), pos + 1
    if c["window"]:
        first = np.maximum(0, pos + 1 - c["window"])
    if c["docs"]:
        starts = [np.sort(r.randint(0, n, 4)) for n in kv_lens]
        first = np.concatenate([np.where(at >= s[0], s[np.maximum(np.searchsorted(s, at, "right") - 1, 0)], 0)
                                for s, at in zip(starts, np.split(pos, np.cumsum(q_lens)[:-1]))])
    if c["prefix"]:
        limit = np.repeat((kv_lens * 0.3).astype(np.int64), q_lens)
        end = np.maximum(end, limit)
    if c["docs"]:
        end = np.where(r.rand(len(pos)) < 0.01, first, end)  # padding between documents sees nothing
    return pos, first, end


def _prepare_attn(c, g):
    kv_lens, q_lens = _lengths(c)
    pos, first, end = _visible(c)
    per = -(-kv_lens // c["page"])
    pages = int(per.sum()) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((c["B"], int(per.max())), dtype=torch.int32, device=DEV)
    filled = torch.from_numpy(np.arange(per.max())[None] < per[:, None]).to(DEV)
    table[filled] = order[:int(per.sum())]
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    device = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).to(DEV)  # noqa: E731
    k_cache, v_cache = _new_cache(c, pages), _new_cache(c, pages)
    seq, at = np.repeat(np.arange(c["B"]), kv_lens), np.concatenate([np.arange(n) for n in kv_lens])
    slots = table.long()[device(seq).long(), device(at // c["page"]).long()] * c["page"] + device(at % c["page"])
    for part in slots.split(1 << 15):
        _put(k_cache, v_cache, _heads(c, g, len(part)).float(), _heads(c, g, len(part)).float(), part, c["page"], c["group"])
    bounded = c["window"] or c["docs"]
    return dict(q=_randn((int(starts[-1]), c["Hq"], c["D"]), g).to(TYPES[c["dtype"]]), k_cache=k_cache, v_cache=v_cache,
                table=table, kv_lens=device(kv_lens), q_starts=device(starts), max_q=int(q_lens.max()),
                max_kv=int(kv_lens.max()), first=device(first) if bounded else None,
                end=device(end) if c["prefix"] or c["docs"] else None,
                slopes=torch.exp2(-8.0 * torch.arange(1, c["Hq"] + 1, device=DEV) / c["Hq"]) if c["slopes"] else None,
                scale=1.0 / math.sqrt(c["D"]))


def _pools(c, g):
    """Caches of several layers: 16-bit ones (group 0), or 4-bit ones as bytes."""
    if c["group"] == 0:
        return [_randn((c["pages"], c["Hkv"], c["page"], c["D"]), g).to(torch.bfloat16) for _ in range(c["caches"])]
    shape = (c["pages"], c["Hkv"], _page_bytes(c))
    return [torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8) for _ in range(c["caches"])]


def _prepare_copy(c, g):
    order = torch.randperm(c["pages"], generator=g, device=DEV).to(torch.int32)
    src = order[:c["n"]].clone()
    src[1::3] = src[0:len(src[1::3]) * 3:3]  # some pages are copied twice
    return dict(caches=_pools(c, g), src=src, dst=order[c["n"]:2 * c["n"]].clone())


def _prepare_compact(c, g):
    r = np.random.RandomState(c["mix"])
    share = r.dirichlet(np.full(c["B"], 2.0)) * c["live"] * c["pages"]
    per = np.maximum(1, share.astype(np.int64))
    common = int(c["shared"] * per.min())  # pages of a prefix that all sequences have
    order = torch.randperm(c["pages"], generator=g, device=DEV).to(torch.int32)
    table = torch.zeros((c["B"], int(per.max()) + 2), dtype=torch.int32, device=DEV)
    filled = torch.from_numpy((np.arange(table.shape[1])[None] < per[:, None])).to(DEV)
    table[filled] = order[:int(per.sum())]
    table[:, :common] = table[0, :common].clone()
    lens = per * c["page"] - r.randint(0, c["page"], c["B"])
    return dict(caches=_pools(c, g), table=table, lens=torch.from_numpy(lens.astype(np.int32)).to(DEV))


# ---- one pass ---------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"append": _plain_append, "gather": _plain_gather, "attn": _plain_attn, "copy": _plain_copy,
            "compact": _plain_compact}[state["case"]["op"]](state, state["case"])


def _run_own(s):
    import weight_only_group_amd as qmm

    c = s["case"]
    if c["op"] == "append":
        q = qmm.qmm_kv4_append(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["positions"], s["slots"], s["k_cache"],
                               s["v_cache"], c["group"], adjacent=c["adjacent"])
        k, v = qmm.qmm_kv4_gather(s["k_cache"], s["v_cache"], s["slots"], c["D"], c["group"], dtype=s["q"].dtype)
        return {"q": q, "k": k, "v": v}
    if c["op"] == "gather":
        k, v = qmm.qmm_kv4_gather(s["k_cache"], s["v_cache"], s["slots"], c["D"], c["group"], dtype=TYPES[c["dtype"]])
        return {"k": k, "v": v}
    if c["op"] == "attn":
        return {"out": qmm.qmm_kv4_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["q_starts"],
                                             s["max_q"], s["max_kv"], c["group"], scale=s["scale"], softcap=c["cap"],
                                             slopes=s["slopes"], first=s["first"], end=s["end"])}
    if c["op"] == "copy":
        qmm.qmm_kv_copy_pages(s["caches"], s["src"], s["dst"])
        return {"caches": s["caches"]}
    table, moved_to, live = qmm.qmm_kv_compact(s["caches"], s["table"], s["lens"], c["page"])
    return {"caches": s["caches"], "table": table, "moved_to": moved_to, "live": live}


def _rotated(x, cos, sin, adjacent):
    R = 2 * cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if adjacent else (x[..., :R // 2], x[..., R // 2:R])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, dim=-1).flatten(-2) if adjacent else torch.cat(turned, dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _plain_append(s, c):
    cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
    q = _rotated(s["q"].float(), cos, sin, c["adjacent"]).to(s["q"].dtype)
    # Keys next to the border of two codes: rotated in 64 bits.
    k = _rotated(s["k"].double(), cos.double(), sin.double(), c["adjacent"]).float()
    keep = s["slots"] >= 0
    _put(s["k_cache"], s["v_cache"], k[keep], s["v"][keep].float(), s["slots"][keep], c["page"], c["group"])
    k, v = _taken(s["k_cache"], s["v_cache"], s["slots"].clamp(min=0), c["page"], c["D"], c["group"])
    k, v = (torch.where(keep[:, None, None], t, 0.0).to(s["q"].dtype) for t in (k, v))
    return {"q": q, "k": k, "v": v}


def _plain_gather(s, c):
    k, v = _taken(s["k_cache"], s["v_cache"], s["slots"], c["page"], c["D"], c["group"])
    return {"k": k.to(TYPES[c["dtype"]]), "v": v.to(TYPES[c["dtype"]])}


def _plain_attn(s, c):
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    starts, kv_lens, max_q, max_kv = s["q_starts"].long(), s["kv_lens"].long(), s["max_q"], s["max_kv"]
    q_lens = starts[1:] - starts[:-1]
    T = s["q"].shape[0]
    nth = torch.arange(max_q, device=DEV)
    token = (starts[:-1, None] + nth).clamp(max=T - 1)  # (B, max_q); past a sequence's end: any token, not used
    pos = kv_lens[:, None] - q_lens[:, None] + nth
    first = s["first"][token].long() if s["first"] is not None else torch.zeros_like(pos)
    end = s["end"][token].long() if s["end"] is not None else pos + 1
    key = torch.arange(max_kv, device=DEV)
    seen = (key >= first[..., None]) & (key < torch.minimum(end, kv_lens[:, None])[..., None])  # (B, max_q, max_kv)
    slots = s["table"].long()[:, key // page] * page + key % page
    k, v = _taken(s["k_cache"], s["v_cache"], slots.flatten(), page, c["D"], c["group"])
    k, v = (t.unflatten(0, (B, max_kv)).transpose(1, 2) for t in (k, v))  # (B, Hkv, max_kv, D)
    q = s["q"].float()[token].unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # (B, Hkv, G max_q, D)
    scores = (q @ k.transpose(2, 3).contiguous()).unflatten(2, (-1, max_q)) * s["scale"]
    if c["cap"]:
        scores = c["cap"] * torch.tanh(scores / c["cap"])
    if c["slopes"]:
        scores = scores - s["slopes"].view(1, Hkv, -1, 1, 1) * (pos[..., None] - key).abs()[:, None, None]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(scores - scores.amax(dim=-1, keepdim=True).clamp(min=-1e30))
    out = p.flatten(2, 3) @ v.contiguous()
    out = out.unflatten(2, (-1, max_q)) / p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)  # (B, max_q, Hq, D)
    of = torch.searchsorted(starts[1:], torch.arange(T, device=DEV), right=True)
    return {"out": out[of, torch.arange(T, device=DEV) - starts[of]].to(s["q"].dtype)}


def _plain_copy(s, c):
    src, dst = s["src"].long(), s["dst"].long()
    for cache in s["caches"]:
        cache[dst] = cache[src]
    return {"caches": s["caches"]}


def _plain_compact(s, c):
    need = (s["lens"] + c["page"] - 1) // c["page"]
    used = torch.arange(s["table"].shape[1], device=DEV) < need[:, None]
    mark = torch.zeros(c["pages"], dtype=torch.bool, device=DEV)
    mark[s["table"][used].long()] = True
    live = mark.sum()
    here = torch.arange(c["pages"], device=DEV)
    low = here < live
    src, dst = torch.nonzero(mark & ~low).squeeze(1), torch.nonzero(~mark & low).squeeze(1)
    moved_to = torch.where(mark, here, -1)
    moved_to[src] = dst
    for cache in s["caches"]:
        cache[dst] = cache[src]
    table = torch.where(used, moved_to[s["table"].long()].to(torch.int32), s["table"])
    return {"caches": s["caches"], "table": table, "moved_to": moved_to.to(torch.int32), "live": live.to(torch.int32).view(1)}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    c = case
    if c["op"] in ("append", "gather"):
        T, D, Hkv = c["T"], c["D"], c["Hkv"]
        kept = T * 0.9 if c.get("skip") else T
        cached = 2 * kept * Hkv * (D / 2 + 4 * D / c["group"])
        if c["op"] == "gather":
            return {"bytes": cached + 2 * T * Hkv * D * 2 + 8 * T, "flops": 4 * T * Hkv * D}
        return {"bytes": 2 * cached + (2 * T * c["Hq"] + 4 * T * Hkv) * D * 2 + T * (c["R"] * 4 + 12),
                "flops": 3 * T * (c["Hq"] + Hkv) * c["R"] + 12 * T * Hkv * D}
    if c["op"] == "attn":
        kv_lens, q_lens = _lengths(c)
        _, first, end = _visible(c)
        seq = np.repeat(np.arange(c["B"]), q_lens)
        end = np.minimum(end, kv_lens[seq])
        some = end > first
        lowest, highest = kv_lens.copy(), np.zeros_like(kv_lens)
        np.minimum.at(lowest, seq[some], first[some])
        np.maximum.at(highest, seq[some], end[some])
        keys = int(np.maximum(0, highest - lowest).sum())
        return {"bytes": 2 * int(q_lens.sum()) * c["Hq"] * c["D"] * 2 + 2 * keys * c["Hkv"] * (c["D"] / 2 + 4 * c["D"] / c["group"]),
                "flops": 4 * c["D"] * c["Hq"] * int(np.maximum(0, end - first).sum())}
    size = c["caches"] * c["Hkv"] * (c["page"] * c["D"] * 2 if c["group"] == 0 else _page_bytes(c))
    if c["op"] == "copy":
        return {"bytes": 2 * c["n"] * size + 8 * c["n"], "flops": 0}
    # Of the live pages as many lie past the packed part as there are free places in it.
    moves = c["pages"] * c["live"] * (1 - c["live"])
    return {"bytes": 2 * moves * size + c["pages"] * 4 + 2 * c["pages"] * c["live"] * 4, "flops": 0}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    return {"append": _exact_append, "gather": _exact_gather, "attn": _exact_attn, "copy": _exact_copy,
            "compact": _exact_compact}[case["op"]](state, case)


def _exact_values(cache, slots, c, keys):
    """(T, Hkv, D) of the slots: each channel's code looked up by its byte and half of it."""
    D, group, G = c["D"], c["group"], c["D"] // c["group"]
    flat = cache.flatten(1)  # a page's bytes
    d = torch.arange(D, device=DEV)
    block = 4 * D + 32 * G
    start = torch.arange(c["Hkv"], device=DEV) * cache.shape[2] + (slots % c["page"] // 8 * block)[:, None]  # (T, Hkv)
    t = (slots % 8)[:, None, None]
    if keys:
        nibble = d % 8 // 2 + d % 2 * 4
        place = t * (D // 2) + 4 * (d % 32 // 8 * (D // 32) + d // 32) + nibble // 2
        scale_at = 4 * D + 2 * (t * 2 * G + d // group)
        middle_at = scale_at + 2 * G
    else:
        nibble = d % 4
        place = d // 4 * 16 + t * 2 + nibble // 2
        scale_at = 4 * D + 2 * (d // group * 16 + t)
        middle_at = scale_at + 16
    page = (slots // c["page"])[:, None, None]
    byte = lambda at: flat[page, start[..., None] + at].to(torch.int32)  # noqa: E731
    half = lambda at: (byte(at) | byte(at + 1) << 8).to(torch.int16).view(torch.float16).double()  # noqa: E731
    code = byte(place) >> (nibble % 2 * 4) & 15
    return half(middle_at) + half(scale_at) * (code - 8)


def _exact_append(s, c):
    half = c["R"] // 2
    at = s["positions"].long()
    turn = torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None]

    def rotate(x):
        x = x.double().clone()
        first, second = (slice(0, c["R"], 2), slice(1, c["R"], 2)) if c["adjacent"] else (slice(0, half), slice(half, c["R"]))
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    def held(x):
        """The values that x's groups of channels become."""
        x = x.clamp(-LARGEST, LARGEST).reshape(c["T"], c["Hkv"], -1, c["group"])
        low, high = x.min(dim=3, keepdim=True).values, x.max(dim=3, keepdim=True).values
        scale = ((high - low) / 15).to(torch.bfloat16).half().double()
        middle = (low + 8 * scale).half().double()
        steps = torch.clamp(torch.round((x - middle) / torch.where(scale > 0, scale, 1.0)), -8, 7)
        return ((middle + scale * steps).reshape(c["T"], c["Hkv"], c["D"])) * (s["slots"] >= 0)[:, None, None]

    return {"q": rotate(s["q"]), "k": held(rotate(s["k"])), "v": held(s["v"].double())}


def _exact_gather(s, c):
    parts = [[_exact_values(cache, part, c, keys) for part in s["slots"].split(4096)]
             for cache, keys in ((s["k_cache"], True), (s["v_cache"], False))]
    return {"k": torch.cat(parts[0]), "v": torch.cat(parts[1])}


def _exact_attn(s, c):
    kv_lens, q_lens = _lengths(c)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    pos, first, end = (torch.from_numpy(a).to(DEV) for a in _visible(c))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    group = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        n, rows = int(kv_lens[b]), slice(int(starts[b]), int(starts[b + 1]))
        j = torch.arange(n, device=DEV)
        slots = s["table"][b].long()[j // c["page"]] * c["page"] + j % c["page"]
        keys, values = (torch.cat([_exact_values(t, part, c, k) for part in slots.split(8192)]).transpose(0, 1).contiguous()
                        for t, k in ((s["k_cache"], True), (s["v_cache"], False)))
        hidden = (j < first[rows, None]) | (j >= end[rows, None])
        empty = hidden.all(dim=1, keepdim=True)
        for h in range(c["Hq"]):
            score = s["scale"] * (s["q"][rows, h].double() @ keys[h // group].T)
            if c["cap"]:
                score = c["cap"] * torch.tanh(score / c["cap"])
            if c["slopes"]:
                score -= s["slopes"][h].double() * (pos[rows, None] - j).abs()
            score[hidden] = -math.inf
            out[rows, h] = torch.where(empty, 0.0, torch.softmax(score, dim=1).nan_to_num(0.0) @ values[h // group])
    return {"out": out}


def _moved(cache, src, dst):
    come_from = np.arange(cache.shape[0])
    come_from[dst] = src
    return cache.index_select(0, torch.from_numpy(come_from).to(DEV))


def _exact_copy(s, c):
    src, dst = s["src"].cpu().numpy(), s["dst"].cpu().numpy()
    return {"caches": [_moved(cache, src, dst) for cache in s["caches"]]}


def _exact_compact(s, c):
    table, lens = s["table"].cpu().numpy(), s["lens"].cpu().numpy()
    rows = [table[b, :-(-lens[b] // c["page"])] for b in range(c["B"])]
    in_use = sorted(set(np.concatenate(rows).tolist()))
    n = len(in_use)
    free = sorted(set(range(n)) - set(in_use))
    high = [p for p in in_use if p >= n]
    moved_to = np.full(c["pages"], -1, np.int32)
    moved_to[in_use] = in_use
    moved_to[high] = free
    new = table.copy()
    for b, row in enumerate(rows):
        new[b, :len(row)] = moved_to[row]
    there = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    return {"caches": [_moved(cache, high, free) for cache in s["caches"]], "table": there(new), "moved_to": there(moved_to),
            "live": there(np.array([n], np.int32))}
