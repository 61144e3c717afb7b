"""The operators of the 4-bit cache as they are used together: prompts in pieces, single tokens, graphs on several streams,
a workspace that calls of several kinds pass round; and sizes that only large calls have. The bytes of the cache are held
to the oracle's, the attention to float64 on those bytes (bounds as in the tests of each call)."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import DEV, check, f64, i32, randn, say
from oracle import cache_oracle as co
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,group,page,dtype", [(64, 32, 8, "fp16"), (128, 64, 24, "bf16"), (256, 128, 16, "bf16")])
def test_serving(w, D, group, page, dtype):  # noqa: F811
    """Three sequences: their prompts in two pieces, then tokens one by one, all attended to as they come."""
    Hq, Hkv, P = 6, 2, 128
    r = np.random.default_rng(D)
    angle = r.uniform(0, 6.28, (P, D // 2))
    cos, sin = (torch.from_numpy(f(angle).astype(np.float32)).to(DEV) for f in (np.cos, np.sin))
    per, pages = -(-100 // page), 3 * -(-100 // page) + 2
    table = r.permutation(pages)[:3 * per].reshape(3, per)
    host = [np.zeros((pages, Hkv, page * (D // 2 + 4 * D // group)), np.uint8) for _ in range(2)]
    caches = [device(c) for c in host]
    lens = np.zeros(3, np.int64)
    for step, new in enumerate(([50, 3, 21], [33, 1, 40], [1, 1, 1], [1, 1, 1])):
        starts = np.concatenate([[0], np.cumsum(new)])
        pos = np.concatenate([np.arange(n, n + m) for n, m in zip(lens, new)])
        slots = np.concatenate([table[b, np.arange(n, n + m) // page] * page + np.arange(n, n + m) % page
                                for b, (n, m) in enumerate(zip(lens, new))]).astype(np.int64)
        q, k, v = (randn((sum(new), h, D), dtype, 10 * step + h + i) for i, h in enumerate((Hq, Hkv, Hkv)))
        got = w.qmm_kv4_append(q, k, v, cos, sin, i32(pos), device(slots), *caches, group)
        co.append(f64(q), f64(k), f64(v), f64(cos), f64(sin), pos, slots, *host, group, page, False)
        for a, b in zip(caches, host):
            assert torch.equal(a, device(b)), step
        lens += new
        out = w.qmm_kv4_attention(got, *caches, i32(table), i32(lens), i32(starts), max(new), int(lens.max()), group)
        want, bound = co.attention(f64(got), co.parts(host[0], D, group, True), co.parts(host[1], D, group, False), table, lens, starts,
                                   D**-0.5, group, dtype=dtype)
        say(f"kv4 serving D={D} step {step}")
        check(out, want, bound, f"step {step}")


def test_a_graph_of_a_decoding_step(w):  # noqa: F811
    """Append, attention and the care of the pages in one graph, replayed for other tokens, against the same calls made eagerly."""
    Hq, Hkv, D, page, group, B = 8, 2, 128, 16, 64, 3
    lens = [700, 301, 64]
    k4, v4, table = paged4(lens, Hkv, D, page, group, 1, spare=8)
    tdev = i32(np.pad(table, ((0, 0), (0, 1))))
    caches, other = ([device(c) for c in (k4, v4)] for _ in range(2))
    q, k, v = (randn((B, h, D), "bf16", h + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    kv, slots, starts = i32(np.array(lens)), torch.zeros(B, dtype=torch.int64, device=DEV), i32(np.arange(B + 1))
    src, dst = i32(np.array([-1])), i32(np.array([0]))

    def step(caches):
        got = w.qmm_kv4_append(q, k, v, None, None, None, slots, *caches, group)
        out = w.qmm_kv4_attention(got, *caches, tdev, kv, starts, 1, 704, group)
        w.qmm_kv_copy_pages(caches, src, dst)
        return out, *w.qmm_kv_compact(caches, tdev, kv, page)

    def inputs(i):
        now = np.array(lens) - i
        slots.copy_(device(np.array([table[b, (n - 1) // page] * page + (n - 1) % page for b, n in enumerate(now)], np.int64)))
        kv.copy_(i32(now))
        for t in (q, k, v):
            t.copy_(randn(t.shape, "bf16", 7 * i + t.shape[1]))

    inputs(0)
    for c in (caches, other):
        step(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches)
    for i in (1, 2, 3):
        inputs(i)
        for c, o, a in zip(caches, other, (k4, v4)):
            c.copy_(device(a))
            o.copy_(device(a))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, *caches)]
        for a, b in zip(got, (*step(other), *other)):
            assert torch.equal(a, b), i


def test_two_graphs_at_once(w):  # noqa: F811
    """Each has a workspace of its own: replayed on two streams at a time, with eager calls on a third."""
    def case(seed, lens):
        k, v, table = paged4(lens, 2, 128, 16, 64, seed)
        return (randn((len(lens), 8, 128), "fp16", seed), device(k), device(v), i32(table), i32(np.array(lens)),
                i32(np.arange(len(lens) + 1)), 1, max(lens), 64)

    calls = [case(1, [3000, 700]), case(2, [2500, 1900, 40]), case(3, [4000])]
    want = [w.qmm_kv4_attention(*c) for c in calls]
    graphs, outs = [], []
    for c in calls[:2]:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w.qmm_kv4_attention(*c))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for i in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            third = w.qmm_kv4_attention(*calls[2])
        torch.cuda.synchronize()
        for a, b in zip((*outs, third), want):
            assert torch.equal(a, b), i


def test_a_workspace_passed_round(w):  # noqa: F811
    """One zeroed buffer for calls of several kinds, one after another."""
    k, v, table = paged4([900, 300], 2, 128, 16, 64, 1)
    q = randn((2, 8, 128), "bf16", 2)
    rest = (i32(table), i32(np.array([900, 300])), i32(np.array([0, 1, 2])), 1, 900)
    dk, dv = device(k), device(v)
    k16, v16 = w.qmm_kv4_gather(dk, dv, torch.arange(len(k) * 16, device=DEV), 128, 64, torch.bfloat16)
    k16, v16 = (t.unflatten(0, (len(k), 16)).transpose(1, 2).contiguous() for t in (k16, v16))
    logits = randn((2, 5000), "bf16", 3)
    kinds = [lambda ws: w.qmm_kv4_attention(q, dk, dv, *rest, 64, workspace=ws), lambda ws: w.qmm_attention(q, k16, v16, *rest, workspace=ws),
             lambda ws: w.qmm_kv_compact([dk.clone(), dv.clone()], rest[0], rest[1], 16, workspace=ws)[0],
             lambda ws: w.qmm_logprobs(logits, torch.tensor([3, 7], device=DEV), top=2, workspace=ws)[0]]
    want = [f(None) for f in kinds]
    ws = torch.zeros(1 << 24, dtype=torch.uint8, device=DEV)
    for i in range(3):
        for f, x in zip(kinds, want):
            assert torch.equal(f(ws), x), i


@pytest.mark.parametrize("Hkv,D,group", [(3, 128, 64), (2, 256, 32), (5, 64, 64)])
def test_gather_of_many(w, Hkv, D, group):  # noqa: F811
    """So many that a thread takes several heads (the last of them one short), as in calls of a part each."""
    T, page = (1 << 22) // (Hkv * D) + 3, 16
    k, v, _ = paged4([400], Hkv, D, page, group, 1, spare=2)
    r = np.random.default_rng(2)
    half = np.frombuffer(np.float16(np.nan).tobytes(), np.uint8)
    at = co.scale_places(3, 0, D, group, False)[0]
    v[2, Hkv - 1].reshape(page // 8, -1)[1, at:at + 2] = half
    slots = device(r.integers(-2, len(k) * page + 2, T))
    dk, dv = device(k), device(v)
    got = w.qmm_kv4_gather(dk, dv, slots, D, group, torch.bfloat16)
    assert torch.isnan(got[1]).any()
    for a in range(0, T, 257):
        part = w.qmm_kv4_gather(dk, dv, slots[a:a + 257], D, group, torch.bfloat16)
        for x, y in zip(got, part):
            assert torch.equal(x[a:a + 257].view(torch.int16), y.view(torch.int16)), a


def test_copies_past_32_bits(w):  # noqa: F811
    """Pages whose offsets in a cache pass 2^32 bytes, copied and packed."""
    size, pages = 1 << 20, 4200
    cache = torch.zeros((pages, size), dtype=torch.uint8, device=DEV)
    x = torch.randint(0, 256, (2, size), dtype=torch.uint8, device=DEV)
    cache[3], cache[pages - 1] = x
    w.qmm_kv_copy_pages([cache], i32(np.array([3, pages - 1])), i32(np.array([pages - 2, 8])))
    assert torch.equal(cache[pages - 2], x[0]) and torch.equal(cache[8], x[1])
    new, moved_to, live = w.qmm_kv_compact([cache], i32(np.array([[pages - 2, 8, 3]])), i32(np.array([48])), 16)
    assert int(live) == 3
    for old, data in ((pages - 2, x[0]), (8, x[1]), (3, x[0])):
        assert torch.equal(cache[int(moved_to[old])], data) and int(moved_to[old]) < 3
    assert torch.equal(new[0], moved_to[torch.tensor([pages - 2, 8, 3], device=DEV)])


@pytest.mark.parametrize("kind", ["halves", "normal", "turned"])
def test_codes_of_many_values(w, kind):  # noqa: F811
    """Scales of every mantissa that 8 bits have, and values half way between codes and next to that: the codes are the
    definition's, bit for bit."""
    D, group, page, T, Hkv = 128, 64, 64, 1016, 4
    r = np.random.default_rng(5)
    if kind == "halves":
        step = 2.0 ** r.integers(-9, 3, (T, Hkv, 1)) * (1 + np.arange(T)[:, None, None] % 127)
        x = np.minimum(step * r.integers(0, 31, (T, Hkv, D)) / 2 * (1 + r.integers(-1, 2, (T, Hkv, D)) * 2.0**-11), 15 * step)
        x[..., ::64], x[..., 1::64] = 0, 15 * step
        x *= r.choice([-1.0, 1.0], (T, Hkv, 1))
    else:
        x = r.standard_normal((T, Hkv, D)) * 10.0 ** r.integers(-5, 4, (T, Hkv, 1)) + r.standard_normal((T, Hkv, 1))
    k = torch.from_numpy(x.astype(np.float16)).to(DEV)
    q = randn((T, Hkv, D), "fp16", 1)
    angle = r.uniform(0, 6.28, (T, D // 2))
    turn = [torch.from_numpy(f(angle).astype(np.float32)).to(DEV) for f in (np.cos, np.sin)] if kind == "turned" else [None, None]
    caches = [torch.zeros((T // page + 1, Hkv, w.kv4_page_bytes(page, D, group)), dtype=torch.uint8, device=DEV) for _ in range(2)]
    w.qmm_kv4_append(q, k, k, *turn, i32(np.arange(T)) if kind == "turned" else None, torch.arange(T, device=DEV), *caches, group)
    for cache, keys in zip(caches, (True, False)):
        want = f64(k)
        if keys and kind == "turned":
            (a, b), (c, s) = np.split(want, 2, -1), (f64(t)[:, None] for t in turn)
            want = np.concatenate([a * c - b * s, b * c + a * s], -1)
        s, m, c = co.quantise(want, group)
        got = [t.transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:T] for t in co.parts(cache.cpu().numpy(), D, group, keys)]
        s, m = (np.repeat(t.astype(np.float64), group, -1) for t in (s, m))
        assert np.array_equal(got[0], s * (c - 8)) and np.array_equal(got[1], m), keys
