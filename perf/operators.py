"""The operators between the quantised products of a decoder layer, as cases to
measure: a mixture-of-experts layer with quantised experts, the append to a paged
key/value cache, the attention that reads it, and log probabilities of tokens.

``run`` computes a case in elementary torch operations in 32 bits (``own`` false)
or through the framework's entry points (``own`` true), on the same state.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # one sequence decoding through a layer of many small experts: latency
        _moe("moe_one_token", T=1, H=2048, I=1024, E=64, k=8, bits=4, gs=128, dtype="fp16"),
        # a decode batch, odd in number, most experts in use by a row or two
        _moe("moe_batch_13", T=13, H=4096, I=1280, E=32, k=4, bits=4, gs=64, dtype="bf16"),
        # the most tokens a call takes, on 3-bit experts of a width that is no power of two, several rows each
        _moe("moe_64_tokens_3bit", T=64, H=4096, I=1408, E=16, k=2, bits=3, gs=64, dtype="fp16", renorm=False),
        # the new tokens of a small decode batch
        _append("append_decode_7", T=7, Hq=32, Hkv=8, D=128, R=128, page=16, dtype="bf16"),
        # a long prompt, some of its tokens not kept, half of each head rotated in adjacent pairs
        _append("append_prompt", T=16381, Hq=24, Hkv=4, D=64, R=32, page=64, dtype="fp16", adjacent=True, skip=True),
        # one sequence decoding on a short context: latency
        _attn("attn_decode_1", B=1, q="one", kv=1500, Hq=32, Hkv=8, D=128, page=16, dtype="bf16"),
        # a decode batch of very different lengths, scores capped, a sliding window
        _attn("attn_decode_48", B=48, q="one", kv=8192, Hq=32, Hkv=8, D=128, page=64, dtype="fp16", cap=50.0,
              window=4096),
        # a long prompt at once, scores capped
        _attn("attn_prompt_8192", B=1, q="all", kv=8192, Hq=32, Hkv=8, D=128, page=128, dtype="bf16", cap=30.0),
        # prompts of several documents after a shared context, with a distance bias and a two-way prefix; rows without keys
        _attn("attn_documents", B=6, q="part", kv=2600, Hq=24, Hkv=24, D=64, page=24, dtype="fp16", slopes=True,
              docs=True, prefix=True),
        # the token just sampled, and its alternatives
        _logp("logprobs_one_row", M=1, V=32000, top=5, dtype="fp16"),
        # a decode batch on a large odd vocabulary, rows padded, the most alternatives a call gives
        _logp("logprobs_batch", M=96, V=128257, top=20, dtype="bf16", pad=127, masked=True),
        # scoring a long prompt
        _logp("logprobs_prompt", M=4096, V=50257, top=1, dtype="fp32"),
    ]


def _moe(name, T, H, I, E, k, bits, gs, dtype, renorm=True):
    return dict(name=name, op="moe", T=T, H=H, I=I, E=E, k=k, bits=bits, gs=gs, dtype=dtype, renorm=renorm)


def _append(name, T, Hq, Hkv, D, R, page, dtype, adjacent=False, skip=False):
    return dict(name=name, op="append", T=T, Hq=Hq, Hkv=Hkv, D=D, R=R, page=page, dtype=dtype, adjacent=adjacent,
                skip=skip)


def _attn(name, B, q, kv, Hq, Hkv, D, page, dtype, cap=0.0, window=0, slopes=False, docs=False, prefix=False, mix=1):
    return dict(name=name, op="attn", B=B, q=q, kv=kv, Hq=Hq, Hkv=Hkv, D=D, page=page, dtype=dtype, cap=cap,
                window=window, slopes=slopes, docs=docs, prefix=prefix, mix=mix)


def _logp(name, M, V, top, dtype, pad=0, masked=False):
    return dict(name=name, op="logp", M=M, V=V, top=top, dtype=dtype, pad=pad, masked=masked)


def _log_between(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def _odd_multiple(step, about):
    """An odd multiple of `step`, not over `about` where that can be."""
    return step * max(1, (about // step - 1) | 1 if about // step % 2 == 0 else about // step)


def draw(rng):
    op = rng.choice(["moe", "moe", "append", "attn", "attn", "attn", "logp"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "moe":
        gs = rng.choice([-1, 32, 64, 128])
        step = max(gs, 32)
        H = _odd_multiple(step, _log_between(rng, 256, 4096))
        E = _log_between(rng, 4, 128)
        while True:  # no more words in all than the second listed case
            I = _odd_multiple(step, _log_between(rng, 128, 4096))
            bits = rng.choice([1, 2, 3, 4, 8])
            if E * H * I * bits <= 32 * 4096 * 1280 * 4 and H * I <= 4096 * 1280:
                break
        T = _log_between(rng, 1, 64)
        k = min(E, rng.randint(1, 8), 128 * 4096 * 1280 // (T * H * I))
        if k < 1:
            T, k = 1, 1
        case = _moe("", T, H, I, E, k, bits, gs, dtype, rng.random() < 0.5)
    elif op == "append":
        Hkv = rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 128, 256])
        T = _log_between(rng, 1, 16384)
        Hq = Hkv * rng.choice([2, 5, 8])
        while T * (Hq + 2 * Hkv) * D > 16381 * 32 * 64:
            T = max(1, T // 2)
        case = _append("", T, Hq, Hkv, D, rng.choice([D, D // 2]), rng.choice([1, 16, 24, 64, 100]), dtype,
                       rng.random() < 0.5, rng.random() < 0.5)
    elif op == "attn":
        D = rng.choice([64, 128, 128, 256])
        q = rng.choice(["one", "one", "few", "part", "all"])
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        B = _log_between(rng, 1, 48 if q in ("one", "few") else 6)
        kv = _log_between(rng, 1, 8192)
        if q in ("part", "all"):
            while B * Hq * D * kv * kv > 16 * 128 * 8192 * 8192:
                kv //= 2
        docs = q in ("part", "all") and rng.random() < 0.5
        case = _attn("", B, q, kv, Hq, Hkv, D, rng.choice([16, 24, 64, 128]), dtype, rng.choice([0.0, 0.0, 20.0, 50.0]),
                     0 if docs else rng.choice([0, 0, _log_between(rng, 16, 4096)]), rng.random() < 0.3, docs,
                     rng.random() < 0.3, rng.randint(1, 1 << 20))
    else:
        dtype = rng.choice(["fp16", "bf16", "fp32"])
        M = _log_between(rng, 1, 4096)
        V = min(_log_between(rng, 500, 200000), 4096 * 50257 // M)
        case = _logp("", M, V, rng.choice([0, 1, 5, 20]), dtype, rng.choice([0, 0, 1, 63]), rng.random() < 0.5)
    del case["name"]
    return case


# ---- what a case is made of -----------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def prepare(case, seed):
    state = {"moe": _prepare_moe, "append": _prepare_append, "attn": _prepare_attn, "logp": _prepare_logp}[case["op"]](
        case, _gen(seed))
    state["case"] = case
    return state


def _word_rows(K, bits):
    """Word rows of the packed plane, and of the 1-bit plane of 3-bit codes."""
    return (K // 16, K // 32) if bits == 3 else (K * bits // 32, 0)


def _expert_weights(g, E, K, N, bits, gs, dtype):
    """E packed weights in 16-column strips with their zero points and scales; scales such that columns keep the
    size of what they multiply."""
    rows, rows_lo = _word_rows(K, bits)
    words = lambda r: torch.randint(-2**31, 2**31, (E, N // 16, r, 16), generator=g, device=DEV, dtype=torch.int32)  # noqa: E731
    groups = 1 if gs == -1 else K // gs
    top = 2**bits - 1
    zeros = torch.randint(0, top + 1, (E, groups, N), generator=g, device=DEV).to(dtype)
    spread = math.sqrt((4.0**bits - 1) / 6 * K)  # of the sum of K differences of two such codes
    scales = ((0.5 + torch.rand((E, groups, N), generator=g, device=DEV)) * (1.0 / spread)).to(dtype)
    return words(rows), words(rows_lo) if bits == 3 else None, zeros, scales


def _prepare_moe(c, g):
    dtype = TYPES[c["dtype"]]
    router = (torch.randn((c["E"], c["H"]), generator=g, device=DEV) / math.sqrt(c["H"])).to(dtype)
    # Rows whose chosen experts hang on the last bits of a sum are passed over, so that the choice has one right answer.
    x = torch.randn((2 * c["T"] + 16, c["H"]), generator=g, device=DEV).to(dtype)
    logits = (x.double() @ router.double().T).sort(dim=1, descending=True).values[:, :c["k"] + 1]
    clear = (logits[:, :-1] - logits[:, 1:]).amin(dim=1) > 1e-4 if logits.shape[1] > 1 else logits[:, 0] > -1e9
    x = x[torch.argsort((~clear).to(torch.int32), stable=True)[:c["T"]]].contiguous()
    return dict(x=x, router=router, gate_up=_expert_weights(g, c["E"], c["H"], 2 * c["I"], c["bits"], c["gs"], dtype),
                down=_expert_weights(g, c["E"], c["I"], c["H"], c["bits"], c["gs"], dtype))


def _prepare_append(c, g):
    dtype = TYPES[c["dtype"]]
    T, Hq, Hkv, D, R = c["T"], c["Hq"], c["Hkv"], c["D"], c["R"]
    # One product gives q, k and v; the three are views into its rows.
    qkv = torch.randn((T, (Hq + 2 * Hkv) * D), generator=g, device=DEV).to(dtype)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], dim=1))
    start = int(torch.randint(0, 1000, (1,), generator=g, device=DEV))
    angles = torch.arange(T + 1000, device=DEV).double()[:, None] * (10000.0 ** (-torch.arange(R // 2, device=DEV).double() * 2 / R))
    pages = (T + 100) // c["page"] + 2
    slots = torch.randperm(pages * c["page"], generator=g, device=DEV)[:T] if T < 64 else _paged_slots(c, g, pages)
    if c["skip"]:
        slots = torch.where(torch.rand(T, generator=g, device=DEV) < 0.1, -1, slots)
    shape = (pages, Hkv, c["page"], D)
    return dict(q=q, k=k, v=v, cos=angles.cos().float(), sin=angles.sin().float(),
                positions=torch.arange(start, start + T, device=DEV, dtype=torch.int32), slots=slots.to(torch.int64),
                k_cache=torch.randn(shape, generator=g, device=DEV).to(dtype),
                v_cache=torch.randn(shape, generator=g, device=DEV).to(dtype))


def _paged_slots(c, g, pages):
    """Consecutive places in pages that lie in any order."""
    order = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(c["T"], device=DEV)
    return order[at // c["page"]] * c["page"] + at % c["page"]


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
    dtype = TYPES[c["dtype"]]
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
    shape = (pages, c["Hkv"], c["page"], c["D"])
    bounded = c["window"] or c["docs"]
    return dict(q=(1.5 * torch.randn((int(starts[-1]), c["Hq"], c["D"]), generator=g, device=DEV)).to(dtype),
                k_cache=torch.randn(shape, generator=g, device=DEV).to(dtype),
                v_cache=torch.randn(shape, generator=g, device=DEV).to(dtype),
                table=table, kv_lens=device(kv_lens), q_starts=device(starts), max_q=int(q_lens.max()),
                max_kv=int(kv_lens.max()), first=device(first) if bounded else None,
                end=device(end) if c["prefix"] or c["docs"] else None,
                slopes=torch.exp2(-8.0 * torch.arange(1, c["Hq"] + 1, device=DEV) / c["Hq"]) if c["slopes"] else None,
                scale=1.0 / math.sqrt(c["D"]))


def _prepare_logp(c, g):
    dtype = TYPES[c["dtype"]]
    rows = torch.empty((c["M"], c["V"] + c["pad"]), dtype=dtype, device=DEV)
    logits = rows[:, :c["V"]]
    for at in range(0, c["M"], 256):
        part = 3.0 * torch.randn((min(256, c["M"] - at), c["V"]), generator=g, device=DEV)
        if c["masked"]:  # tokens that a grammar forbids
            part[torch.rand(part.shape, generator=g, device=DEV) < 0.3] = -math.inf
        logits[at:at + 256] = part.to(dtype)
    targets = torch.randint(0, c["V"], (c["M"],), generator=g, device=DEV)
    likely = logits.argmax(dim=1)
    return dict(logits=logits, targets=torch.where(torch.arange(c["M"], device=DEV) % 2 == 0, likely, targets))


# ---- one pass ---------------------------------------------------------------------

def run(state):
    if own:
        return _run_own(state)
    return {"moe": _plain_moe, "append": _plain_append, "attn": _plain_attn, "logp": _plain_logp}[state["case"]["op"]](
        state, state["case"])


def _run_own(s):
    import weight_only_group_amd as qmm

    c = s["case"]
    if c["op"] == "moe":
        ids, weights, logits = qmm.qmm_moe_route(s["x"], s["router"], c["k"], renormalize=c["renorm"])
        y = qmm.qmm_moe(s["x"], ids, weights, s["gate_up"], s["down"], c["bits"], c["gs"], strips=True)
        return {"logits": logits, "ids": ids, "weights": weights, "y": y}
    if c["op"] == "append":
        q = qmm.qmm_kv_append(s["q"], s["k"], s["v"], s["cos"], s["sin"], s["positions"], s["slots"], s["k_cache"],
                              s["v_cache"], adjacent=c["adjacent"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["op"] == "attn":
        return {"out": qmm.qmm_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["q_starts"],
                                         s["max_q"], s["max_kv"], scale=s["scale"], softcap=c["cap"],
                                         slopes=s["slopes"], first=s["first"], end=s["end"])}
    logprob, entropy, top_logprobs, top_ids = qmm.qmm_logprobs(s["logits"], s["targets"], top=c["top"])
    return {"logprob": logprob, "entropy": entropy, "top_logprobs": top_logprobs, "top_ids": top_ids}


def _codes(words, lo, bits):
    """(..., strips, rows, 16) words -> (..., K, columns) codes."""
    def plane(w, b):
        shifts = torch.arange(0, 32, b, device=w.device, dtype=torch.int32)[:, None]
        return ((w.unsqueeze(-2) >> shifts) & (2**b - 1)).flatten(-3, -2)
    codes = plane(words, 2) * 2 + plane(lo, 1) if bits == 3 else plane(words, bits)
    return codes.movedim(-3, -2).flatten(-2)


def _dequantised(weight, experts, bits, gs):
    words, lo, zeros, scales = weight
    codes = _codes(words[experts], lo[experts] if bits == 3 else None, bits).float()
    groups = zeros.shape[1]
    codes = codes.unflatten(1, (groups, -1))
    return (scales[experts].float().unsqueeze(2) * (codes - zeros[experts].float().unsqueeze(2))).flatten(1, 2)


def _plain_moe(s, c):
    x = s["x"].float()
    logits = x @ s["router"].float().T
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, chosen = order.indices[:, :c["k"]], order.values[:, :c["k"]]
    of = chosen if c["renorm"] else logits
    most = logits.amax(dim=1, keepdim=True)
    weights = torch.exp(chosen - most) / torch.exp(of - most).sum(dim=1, keepdim=True)
    flat = ids.flatten()
    rows = x.repeat_interleave(c["k"], dim=0).unsqueeze(1)
    gate, up = (rows @ _dequantised(s["gate_up"], flat, c["bits"], c["gs"])).chunk(2, dim=2)
    hidden = gate / (1 + torch.exp(-gate)) * up
    out = (hidden @ _dequantised(s["down"], flat, c["bits"], c["gs"])).squeeze(1)
    y = (out.unflatten(0, (-1, c["k"])) * weights.unsqueeze(2)).sum(dim=1)
    return {"logits": logits, "ids": ids.to(torch.int32), "weights": weights, "y": y.to(s["x"].dtype)}


def _rotated(x, cos, sin, adjacent):
    R = 2 * cos.shape[1]
    x, cos, sin = x.float(), cos[:, None], sin[:, None]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if adjacent else (x[..., :R // 2], x[..., R // 2:R])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, dim=-1).flatten(-2) if adjacent else torch.cat(turned, dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _plain_append(s, c):
    cos, sin = s["cos"][s["positions"].long()], s["sin"][s["positions"].long()]
    q = _rotated(s["q"], cos, sin, c["adjacent"]).to(s["q"].dtype)
    k = _rotated(s["k"], cos, sin, c["adjacent"]).to(s["k"].dtype)
    keep = s["slots"] >= 0
    page, at = s["slots"][keep] // c["page"], s["slots"][keep] % c["page"]
    s["k_cache"][page, :, at] = k[keep]
    s["v_cache"][page, :, at] = s["v"][keep]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attn(s, c):
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
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
    cached = lambda cache: cache[s["table"].long()].transpose(1, 2).flatten(2, 3)[:, :, :max_kv].float()  # noqa: E731
    q = s["q"].float()[token].unflatten(2, (Hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # (B, Hkv, G max_q, D)
    scores = (q @ cached(s["k_cache"]).transpose(2, 3).contiguous()).unflatten(2, (-1, max_q)) * s["scale"]
    if c["cap"]:
        scores = c["cap"] * torch.tanh(scores / c["cap"])
    if c["slopes"]:
        scores = scores - s["slopes"].view(1, Hkv, -1, 1, 1) * (pos[..., None] - key).abs()[:, None, None]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(scores - scores.amax(dim=-1, keepdim=True).clamp(min=-1e30))
    out = p.flatten(2, 3) @ cached(s["v_cache"])
    out = out.unflatten(2, (-1, max_q)) / p.sum(dim=-1, keepdim=True).clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)  # (B, max_q, Hq, D)
    of = torch.searchsorted(starts[1:], torch.arange(T, device=DEV), right=True)
    return {"out": out[of, torch.arange(T, device=DEV) - starts[of]].to(s["q"].dtype)}


def _plain_logp(s, c):
    l = s["logits"].float()
    most = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - most)
    total = e.sum(dim=1, keepdim=True)
    lse = most + torch.log(total)
    weighted = torch.where(e > 0, e * (l - most), 0.0).sum(dim=1)
    entropy = torch.log(total).squeeze(1) - weighted / total.squeeze(1)
    logprob = l.gather(1, s["targets"][:, None]).squeeze(1) - lse.squeeze(1)
    order = torch.sort(l, dim=1, descending=True, stable=True)
    return {"logprob": logprob, "entropy": entropy, "top_logprobs": order.values[:, :c["top"]] - lse,
            "top_ids": order.indices[:, :c["top"]].to(torch.int32)}


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    c, size = case, SIZE[case["dtype"]]
    if c["op"] == "moe":
        T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
        used = E * (1 - (1 - k / E) ** T)  # experts that T independent choices of k reach, on average
        groups = [1, 1] if c["gs"] == -1 else [H // c["gs"], I // c["gs"]]
        expert = 3 * H * I * c["bits"] / 8 + (groups[0] * 2 * I + groups[1] * H) * 2 * size
        return {"bytes": used * expert + E * H * size + 2 * T * H * size + T * E * 4 + T * k * 8,
                "flops": 2 * T * H * E + 6 * T * k * H * I}
    if c["op"] == "append":
        T, D = c["T"], c["D"]
        return {"bytes": 2 * T * (c["Hq"] + 2 * c["Hkv"]) * D * size + T * (c["R"] * 4 + 12),
                "flops": 3 * T * (c["Hq"] + c["Hkv"]) * c["R"]}
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
        return {"bytes": (2 * int(q_lens.sum()) * c["Hq"] + 2 * keys * c["Hkv"]) * c["D"] * size,
                "flops": 4 * c["D"] * c["Hq"] * int(np.maximum(0, end - first).sum())}
    return {"bytes": c["M"] * (c["V"] * size + 8 + 8 + 8 * c["top"]), "flops": 5 * c["M"] * c["V"]}


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    return {"moe": _exact_moe, "append": _exact_append, "attn": _exact_attn, "logp": _exact_logp}[case["op"]](state, case)


def _exact_weight(weight, e, K, bits, gs):
    """One expert's weight, (K, columns): s (q - z), code by code from the words' bits."""
    words, lo, zeros, scales = weight
    k = torch.arange(K, device=DEV)

    def field(plane, width):
        per = 32 // width
        by_row = plane[e].permute(1, 0, 2).reshape(plane.shape[2], -1).long() & 0xFFFFFFFF  # (rows, columns)
        return (by_row[k // per] >> ((k % per) * width)[:, None]) % 2**width

    q = 2 * field(words, 2) + field(lo, 1) if bits == 3 else field(words, bits)
    g = k // (K if gs == -1 else gs)
    return scales[e].double()[g] * (q.double() - zeros[e].double()[g])


def _exact_moe(s, c):
    x = s["x"].double()
    logits = x @ s["router"].double().T
    chosen, ids = torch.topk(logits, c["k"], dim=1)
    probs = torch.softmax(logits, dim=1).gather(1, ids)
    weights = probs / probs.sum(dim=1, keepdim=True) if c["renorm"] else probs
    y = torch.zeros_like(x)
    for e in ids.unique().tolist():
        token, nth = torch.nonzero(ids == e, as_tuple=True)
        both = x[token] @ _exact_weight(s["gate_up"], e, c["H"], c["bits"], c["gs"])
        hidden = torch.nn.functional.silu(both[:, :c["I"]]) * both[:, c["I"]:]
        part = hidden @ _exact_weight(s["down"], e, c["I"], c["bits"], c["gs"])
        y.index_add_(0, token, weights[token, nth][:, None] * part)
    return {"logits": logits, "ids": ids.to(torch.int32), "weights": weights, "y": y}


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

    def stored(cache, rows):
        flat = cache.double().permute(0, 2, 1, 3).reshape(-1, c["Hkv"], c["D"]).clone()
        kept = (s["slots"] >= 0).nonzero().squeeze(1)
        flat[s["slots"][kept]] = rows[kept]
        return flat.view(cache.shape[0], c["page"], c["Hkv"], c["D"]).permute(0, 2, 1, 3)

    return {"q": rotate(s["q"]), "k_cache": stored(s["k_cache"], rotate(s["k"])),
            "v_cache": stored(s["v_cache"], s["v"].double())}


def _exact_attn(s, c):
    kv_lens, q_lens = _lengths(c)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    pos, first, end = (torch.from_numpy(a).to(DEV) for a in _visible(c))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    group = c["Hq"] // c["Hkv"]
    for b in range(c["B"]):
        n, rows = int(kv_lens[b]), slice(int(starts[b]), int(starts[b + 1]))
        pages = s["table"][b, :-(-n // c["page"])].long()
        keys, values = (t[pages].double().permute(1, 0, 2, 3).flatten(1, 2)[:, :n] for t in (s["k_cache"], s["v_cache"]))
        j = torch.arange(n, device=DEV)
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


def _exact_logp(s, c):
    parts = []
    for at in range(0, c["M"], 512):
        logp = torch.log_softmax(s["logits"][at:at + 512].double(), dim=1)
        entropy = -(logp.exp() * logp.clamp(min=-1e300)).sum(dim=1)
        rank = torch.sort(logp, dim=1, descending=True, stable=True)
        parts.append((logp.gather(1, s["targets"][at:at + 512, None]).squeeze(1), entropy, rank.values[:, :c["top"]],
                      rank.indices[:, :c["top"]].to(torch.int32)))
    return dict(zip(("logprob", "entropy", "top_logprobs", "top_ids"), (torch.cat(p) for p in zip(*parts))))
