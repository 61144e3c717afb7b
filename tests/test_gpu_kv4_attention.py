"""qmm_kv4_attention against float64, at the lengths, masks and layouts where it can go wrong. The bound of each
element is the oracle's: fp32 scores and sums of the codes' parts, weights rounded to fp16, one rounding of the result."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import DEV, check, f64, i32, randn, say
from oracle import cache_oracle as co
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def run(w, kv_lens, q_lens, Hq, Hkv, D, page, group, dtype, seed=1, fill=None, view=False, q_scale=1.5, max_kv=None, scale=1.0, **kw):  # noqa: F811
    """The call and the oracle on the same inputs."""
    B, T = len(kv_lens), sum(q_lens)
    say(f"kv4 attention kv={kv_lens} q={q_lens} Hq={Hq} Hkv={Hkv} D={D} page={page} group={group} {dtype} {sorted(kw)}")
    k, v, table = paged4(kv_lens, Hkv, D, page, group, seed, fill=fill, scale=scale)
    if view:
        q = randn((T, (Hq + 3) * D), dtype, seed + 1, q_scale)[:, D:(Hq + 1) * D].unflatten(1, (Hq, D))
    else:
        q = randn((T, Hq, D), dtype, seed + 1, q_scale)
    if max_kv and max_kv > table.shape[1] * page:
        table = np.pad(table, ((0, 0), (0, -(-max_kv // page) - table.shape[1])))
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    dev = {n: (torch.from_numpy(a).float().to(DEV) if n == "slopes" else i32(a)) if isinstance(a, np.ndarray) else a
           for n, a in kw.items()}
    out = w.qmm_kv4_attention(q, device(k), device(v), i32(table), i32(np.array(kv_lens)), i32(starts), max(q_lens),
                              max_kv or max(kv_lens), group, **dev)
    kw.setdefault("scale", D**-0.5)
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"].astype(np.float32)
    want, bound = co.attention(f64(q), co.parts(k, D, group, True), co.parts(v, D, group, False), table, kv_lens, starts,
                               group=group, dtype=dtype, **kw)
    check(out, want, bound, "out")
    return out


SHAPES = [  # Hq, Hkv, D, page, group
    (1, 1, 64, 16, 32), (8, 2, 128, 16, 32), (5, 1, 64, 24, 64), (4, 4, 128, 128, 64), (16, 1, 256, 8, 32), (40, 2, 64, 8, 32),
    (6, 2, 256, 64, 64), (4, 2, 128, 40, 128), (3, 1, 256, 16, 128),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page,group", SHAPES)
def test_one_token(w, Hq, Hkv, D, page, group, dtype):  # noqa: F811
    run(w, [1, 2, 31, 32, 33, 64, 100, 257], [1] * 8, Hq, Hkv, D, page, group, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv", [1, 17, 700, 4099])
def test_one_sequence_split(w, kv, dtype):  # noqa: F811
    """One sequence alone: its keys are split over many blocks and joined."""
    run(w, [kv], [1], 8, 2, 128, 16, 64, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page,group", SHAPES)
def test_few_tokens(w, Hq, Hkv, D, page, group, dtype):  # noqa: F811
    run(w, [5, 40, 9, 130], [5, 3, 1, 8], Hq, Hkv, D, page, group, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page,group", SHAPES)
def test_prompts(w, Hq, Hkv, D, page, group, dtype):  # noqa: F811
    run(w, [70, 1, 150, 129], [70, 1, 65, 128], Hq, Hkv, D, page, group, dtype)


@pytest.mark.parametrize("D,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
def test_longer_prompt(w, D, group):  # noqa: F811
    run(w, [531], [531], 2, 1, D, 32, group, "bf16")


@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.0, True), (5.0, True), (300.0, False)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_cap_and_distance(w, dtype, softcap, slopes):  # noqa: F811
    kw = {"softcap": softcap}
    if slopes:
        kw["slopes"] = 2.0 ** -np.arange(1, 5)
    run(w, [33, 200, 140], [1, 1, 1], 4, 2, 128, 16, 32, dtype, q_scale=4.0, **kw)
    run(w, [90, 200], [90, 70], 4, 2, 64, 16, 64, dtype, q_scale=4.0, **kw)


def _positions(kv_lens, q_lens):
    return np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [3, 2, 8], [90, 40, 130]])
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "any"])
def test_masks(w, kind, q_lens):  # noqa: F811
    kv_lens = [90, 200, 140]
    pos = _positions(kv_lens, q_lens)
    first, end = np.zeros_like(pos), pos + 1
    r = np.random.default_rng(3)
    if kind == "window":
        first = pos + 1 - 20  # negative for early tokens
    elif kind == "documents":
        first = pos // 37 * 37
    elif kind == "prefix":
        end = np.maximum(end, 50)
    else:  # any range, many of them empty, some past either end
        first, end = r.integers(-50, 220, len(pos)), r.integers(-50, 220, len(pos))
    out = run(w, kv_lens, q_lens, 4, 2, 128, 24, 32, "bf16", first=first, end=end)
    kv = np.repeat(kv_lens, q_lens)
    empty = np.maximum(first, 0) >= np.minimum(end, kv)
    assert not f64(out)[empty].any()


def test_all_rows_empty(w):  # noqa: F811
    out = run(w, [40, 300], [2, 100], 4, 2, 128, 16, 64, "fp16", first=np.full(102, 30), end=np.full(102, 30))
    assert not out.any()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 60000.0])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [30, 64, 5]])
def test_places_past_the_end_have_no_part(w, q_lens, fill):  # noqa: F811
    """Unwritten places of the last page, spare pages and rounded-up tiles."""
    run(w, [30, 77, 5], q_lens, 4, 2, 64, 32, 32, "fp16", fill=fill)
    run(w, [30, 77, 5], q_lens, 4, 2, 128, 32, 64, "bf16", fill=fill)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 32)])
@pytest.mark.parametrize("T", [8, 60, 100])
def test_a_bad_group_reaches_only_queries_that_see_it(w, T, D, group, bad):  # noqa: F811
    """A key and a value whose scale or middle is not finite, seen by the last queries only."""
    kv, page = 100, 16
    k, v, table = paged4([kv], 2, D, page, group, 1)
    q = randn((T, 4, D), "bf16", 2)
    starts = np.array([0, T])
    args = (i32(table), i32(np.array([kv])), i32(starts), T, kv, group)
    clean = w.qmm_kv4_attention(q, device(k), device(v), *args)
    half = np.frombuffer(np.float16(bad).tobytes(), np.uint8)
    for cache, head, key, which, keys in ((k, 0, 97, 0, True), (v, 1, 96, 1, False), (v, 0, 98, 0, False)):
        block = cache[table[0, key // page], head].reshape(page // 8, -1)[key % page // 8]
        at = co.scale_places(key % 8, 1 % (D // group), D, group, keys)[which]
        block[at:at + 2] = half
    got = w.qmm_kv4_attention(q, device(k), device(v), *args)
    assert torch.equal(got[:T - 4], clean[:T - 4])  # queries at positions up to 95
    want, bound = co.attention(f64(q), co.parts(k, D, group, True), co.parts(v, D, group, False), table, [kv], starts, D**-0.5,
                               group, dtype="bf16")
    assert np.isnan(want[T - 1]).any()
    check(got, want, bound, "bad groups")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T", [2, 80])
def test_a_bad_query_gives_nan_and_only_there(w, T, bad):  # noqa: F811
    k, v, table = paged4([100], 2, 128, 16, 64, 1)
    q = randn((T, 4, 128), "bf16", 2)
    args = (device(k), device(v), i32(table), i32(np.array([100])), i32(np.array([0, T])), T, 100, 64)
    clean = w.qmm_kv4_attention(q, *args)
    q[1, 2, 77] = bad
    got = w.qmm_kv4_attention(q, *args)
    assert torch.isnan(got[1, 2]).all()
    got[1, 2] = clean[1, 2]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("q_scale,scale", [(300.0, 1.0), (1e-4, 1.0), (1.0, 500.0), (1.0, 1e-3), (3e30, 1.0)])
def test_sizes(w, q_scale, scale):  # noqa: F811
    """Scores of thousands (the softmax is one key's), tiny queries, large and small caches, queries past fp16's range."""
    dtypes = ["bf16"] if q_scale > 1e4 else ["fp16", "bf16"]
    for dtype in dtypes:
        extra = {"softcap": 20.0} if q_scale > 1e4 else {}
        run(w, [200, 90], [1, 90], 4, 2, 128, 16, 64, dtype, q_scale=q_scale, scale=scale, **extra)


def test_a_long_tail_of_small_weights(w):  # noqa: F811
    """Many keys far below a row's largest one: together they count."""
    kv, D, page, group = 3000, 64, 8, 32
    k, v, table = paged4([kv], 1, D, page, group, 1)
    q = randn((1, 1, D), "bf16", 2, 12.0)
    out = w.qmm_kv4_attention(q, device(k), device(v), i32(table), i32(np.array([kv])), i32(np.array([0, 1])), 1, kv, group, scale=0.3)
    want, bound = co.attention(f64(q), co.parts(k, D, group, True), co.parts(v, D, group, False), table, [kv], [0, 1], 0.3, group,
                               dtype="bf16")
    check(out, want, bound, "out")


def test_query_views_and_lengths_below_the_bounds(w):  # noqa: F811
    run(w, [40, 90], [1, 1], 4, 2, 128, 16, 32, "fp16", view=True)
    run(w, [40, 90], [33, 80], 4, 2, 128, 16, 32, "bf16", view=True, max_kv=96)


def test_sequences_without_keys_or_queries(w):  # noqa: F811
    say("kv4 attention with empty sequences")
    D, page, group = 128, 16, 32
    k, v, table = paged4([20, 1, 40, 16], 2, D, page, group, 1)
    q = randn((4, 4, D), "fp16", 2)
    kv = np.array([20, 0, 40, 16])  # sequence 1 has a query and no key; sequence 2 no query
    starts = np.array([0, 1, 2, 2, 4])
    out = w.qmm_kv4_attention(q, device(k), device(v), i32(table), i32(kv), i32(starts), 2, 40, group)
    want, bound = co.attention(f64(q), co.parts(k, D, group, True), co.parts(v, D, group, False), table, kv, starts, D**-0.5, group)
    check(out, want, bound, "out")
    assert not out[1].any()
    assert w.qmm_kv4_attention(q[:0], device(k), device(v), i32(table), i32(kv * 0), i32(starts * 0), 0, 0, group).shape == (0, 4, D)


@pytest.mark.parametrize("starts,kv_lens,max_q,T", [([0, 1, 2, 3], [700, 5, 33], 1, 16), ([2, 3, 4, 5], [70, 5, 33], 1, 6),
                                                    ([0, 5, 6, 9], [70, 5, 33], 2, 11), ([7, 137, 137, 237, 300], [130, 4, 150, 90], 130, 400),
                                                    ([0, 130, 230, 300], [130, 150, 90], 80, 301)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_tokens_of_no_sequence_get_0(w, D, starts, kv_lens, max_q, T):  # noqa: F811
    """A padded batch reads nothing stale, and its other results are those without the padding."""
    say(f"kv4 attention padding D={D} starts={starts} kv={kv_lens} max_q={max_q} T={T}")
    k, v, table = paged4(kv_lens, 2, D, 16, 32, 1)
    q = randn((T, 8, D), "bf16", 2)
    rest = (device(k), device(v), i32(table), i32(np.array(kv_lens)))
    out = torch.ones_like(q)
    w.qmm_kv4_attention(q, *rest, i32(np.array(starts)), max_q, max(kv_lens), 32, out=out)
    of_none = np.ones(T, bool)
    for a, b in zip(starts, starts[1:]):
        of_none[a:min(b, a + max_q)] = False
    none = torch.from_numpy(of_none).to(DEV)
    assert not out[none].any() and out[~none].any()
    first, last = starts[0], starts[-1]
    alone = w.qmm_kv4_attention(q[first:last].contiguous(), *rest, i32(np.array(starts) - first), max_q, max(kv_lens), 32)
    assert torch.equal(out[~none], alone[~none[first:last]])


def test_no_sequences_at_all(w):  # noqa: F811
    q = randn((5, 4, 64), "fp16", 1)
    k = torch.zeros((2, 2, w.kv4_page_bytes(16, 64, 32)), dtype=torch.uint8, device=DEV)
    for table, kv, starts, max_q in ((np.zeros((0, 4)), np.zeros(0), np.zeros(1), 1), (np.zeros((1, 4)), np.ones(1), np.array([0, 5]), 0)):
        out = torch.ones_like(q)
        w.qmm_kv4_attention(q, k, k, i32(table), i32(kv), i32(starts), max_q, 16, 32, out=out)
        assert not out.any()


def test_equal_bits_and_other_stream(w):  # noqa: F811
    k, v, table = paged4([700, 300], 2, 128, 16, 64, 1)
    q = randn((2, 8, 128), "bf16", 2)
    args = (device(k), device(v), i32(table), i32(np.array([700, 300])), i32(np.array([0, 1, 2])), 1, 700, 64)
    a = w.qmm_kv4_attention(q, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = w.qmm_kv4_attention(q, *args)
    s.synchronize()
    for _ in range(5):
        assert torch.equal(a, w.qmm_kv4_attention(q, *args))
    assert torch.equal(a, b)


def test_page_ids_outside_the_cache_are_cut(w):  # noqa: F811
    k, v, table = paged4([40], 1, 64, 16, 32, 1)
    q = randn((1, 2, 64), "fp16", 2)
    bad = table.copy()
    bad[0, 1] = 1 << 30
    bad[0, 2] = -9
    cut = np.clip(bad, 0, len(k) - 1)
    rest = (i32(np.array([40])), i32(np.array([0, 1])), 1, 40, 32)
    assert torch.equal(w.qmm_kv4_attention(q, device(k), device(v), i32(bad), *rest),
                       w.qmm_kv4_attention(q, device(k), device(v), i32(cut), *rest))


def test_large_cache_offsets(w):  # noqa: F811
    """Pages past 2^32 bytes."""
    Hkv, D, page, group = 8, 256, 128, 32
    size = w.kv4_page_bytes(page, D, group)
    pages = (1 << 32) // (Hkv * size) + 5
    k = torch.zeros((pages, Hkv, size), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    last = [device(c) for c in paged4([2 * page], Hkv, D, page, group, 1, spare=0)[:2]]
    k[-2:], v[-2:] = last
    for n in (1, 60):
        q = randn((n, 8, D), "fp16", 3)
        rest = (i32(np.array([200])), i32(np.array([0, n])), n, 200, group)
        out = w.qmm_kv4_attention(q, k, v, i32(np.array([[pages - 1, pages - 2]])), *rest)
        near = w.qmm_kv4_attention(q, *last, i32(np.array([[1, 0]])), *rest)
        assert torch.equal(out, near)
        assert out.any()


def test_attention_in_a_graph(w):  # noqa: F811
    """Captured without a workspace of its own; replayed for other lengths, with eager calls between."""
    k, v, table = paged4([700, 300], 2, 128, 16, 64, 1)
    q = randn((2, 8, 128), "fp16", 2)
    kv = i32(np.array([700, 300]))
    args = (device(k), device(v), i32(table), kv, i32(np.array([0, 1, 2])), 1, 700, 64)
    w.qmm_kv4_attention(q, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w.qmm_kv4_attention(q, *args)
    for n in (700, 1, 433, 650):
        kv.copy_(torch.tensor([n, min(n, 300)]))
        q.copy_(randn((2, 8, 128), "fp16", n))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, w.qmm_kv4_attention(q, *args)), n


def test_refusals_on_tensors(w):  # noqa: F811
    k, v, table = paged4([40], 1, 64, 16, 32, 1)
    q = randn((1, 2, 64), "fp16", 2)
    rest = (i32(table), i32(np.array([40])), i32(np.array([0, 1])), 1, 40)
    dk, dv = device(k), device(v)
    w.qmm_kv4_attention(q, dk, dv, *rest, 32)
    for change, error in ((dict(group=64), ValueError), (dict(group=24), ValueError), (dict(k=dk.view(torch.int8)), TypeError),
                          (dict(v=dv[:-1]), ValueError), (dict(k=dk[0]), ValueError), (dict(q=q.float()), TypeError)):
        a = dict(q=q, k=dk, v=dv, group=32) | change
        with pytest.raises(error):
            w.qmm_kv4_attention(a["q"], a["k"], a["v"], *rest, a["group"])
    with pytest.raises(w.QmmError):
        w.qmm_kv4_attention(q, dk, dv, *rest[:-1], 10_000, 32)
