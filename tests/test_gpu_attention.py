"""qmm_attention against float64, at the lengths, masks and layouts where it can
go wrong. The bound of each element is the oracle's: fp32 scores, weights
rounded to the data type, one rounding of the result."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, check, f64, i32, paged, randn, say
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required")
    import weight_only_group_amd as mod
    mod.library()
    return mod


def run(w, kv_lens, q_lens, Hq, Hkv, D, page, dtype, seed=1, fill=None, view=False, q_scale=1.5, max_kv=None, **kw):
    """The call and the oracle on the same inputs."""
    B, T = len(kv_lens), sum(q_lens)
    say(f"attention kv={kv_lens} q={q_lens} Hq={Hq} Hkv={Hkv} D={D} page={page} {dtype} {sorted(kw)}")
    k, v, table = paged(B, kv_lens, Hkv, D, page, dtype, seed, fill=fill)
    if view:
        q = randn((T, (Hq + 3) * D), dtype, seed + 1, q_scale)[:, D:(Hq + 1) * D].unflatten(1, (Hq, D))
    else:
        q = randn((T, Hq, D), dtype, seed + 1, q_scale)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    dev = {n: (torch.from_numpy(a).float().to(DEV) if n == "slopes" else i32(a)) if isinstance(a, np.ndarray) else a
           for n, a in kw.items()}
    out = w.qmm_attention(q, k, v, i32(table), i32(np.array(kv_lens)), i32(starts), max(q_lens), max_kv or max(kv_lens),
                          **dev)
    kw.setdefault("scale", D**-0.5)
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"].astype(np.float32)
    want, bound = lo.attention(f64(q), f64(k), f64(v), table, kv_lens, starts, dtype=dtype, **kw)
    check(out, want, bound, "out")
    return out


SHAPES = [  # Hq, Hkv, D, page
    (1, 1, 64, 16), (8, 2, 128, 16), (5, 1, 64, 24), (4, 4, 128, 128), (16, 1, 256, 7), (40, 2, 64, 1), (6, 2, 256, 64),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page", SHAPES)
def test_one_token(w, Hq, Hkv, D, page, dtype):
    run(w, [1, 2, 31, 32, 33, 64, 100, 257], [1] * 8, Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv", [1, 17, 700, 4099])
def test_one_sequence_split(w, kv, dtype):
    """One sequence alone: its keys are split over many blocks and joined."""
    run(w, [kv], [1], 8, 2, 128, 16, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page", SHAPES)
def test_few_tokens(w, Hq, Hkv, D, page, dtype):
    run(w, [5, 40, 9, 130], [5, 3, 1, 8], Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page", SHAPES)
def test_prompts(w, Hq, Hkv, D, page, dtype):
    run(w, [70, 1, 150, 129], [70, 1, 65, 128], Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_longer_prompt(w, D):
    run(w, [531], [531], 2, 1, D, 32, "bf16")


@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_cap_and_distance(w, dtype, softcap, slopes):
    kw = {"softcap": softcap}
    if slopes:
        kw["slopes"] = 2.0 ** -np.arange(1, 5)
    run(w, [33, 200, 140], [1, 1, 1], 4, 2, 128, 16, dtype, q_scale=4.0, **kw)
    run(w, [90, 200], [90, 70], 4, 2, 64, 16, dtype, q_scale=4.0, **kw)


def _positions(kv_lens, q_lens):
    return np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [3, 2, 8], [90, 40, 130]])
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "any"])
def test_masks(w, kind, q_lens):
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
    out = run(w, kv_lens, q_lens, 4, 2, 128, 24, "bf16", first=first, end=end)
    kv = np.repeat(kv_lens, q_lens)
    empty = np.maximum(first, 0) >= np.minimum(end, kv)
    assert not f64(out)[empty].any()


def test_all_rows_empty(w):
    out = run(w, [40, 300], [2, 100], 4, 2, 128, 16, "fp16", first=np.full(102, 30), end=np.full(102, 30))
    assert not out.any()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 60000.0])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [30, 64, 5]])
def test_places_past_the_end_have_no_part(w, q_lens, fill):
    """Unwritten places of the last page, spare pages and rounded-up tiles."""
    run(w, [30, 77, 5], q_lens, 4, 2, 64, 32, "fp16", fill=fill)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("q_lens", [[8], [60], [100]])
def test_a_bad_value_reaches_only_queries_that_see_it(w, q_lens, bad):
    """A key and a value that are not finite, seen by the last queries only."""
    kv, D, page = 100, 64, 16
    T = q_lens[0]
    k, v, table = paged(1, [kv], 2, D, page, "bf16", 1)
    q = randn((T, 4, D), "bf16", 2)
    args = (i32(table), i32(np.array([kv])), i32(np.array([0, T])), T, kv)
    clean = w.qmm_attention(q, k, v, *args)
    k[table[0, 97 // page], 0, 97 % page, 3] = bad
    v[table[0, 96 // page], 1, 96 % page, 5] = bad
    got = w.qmm_attention(q, k, v, *args)
    before = T - 4  # queries at positions up to 95
    assert torch.equal(got[:before], clean[:before])
    assert not torch.isfinite(got[T - 1]).all()


def test_huge_scores(w):
    """Scores of thousands: the softmax is one key's, with no overflow."""
    run(w, [200, 90], [1, 90], 4, 2, 128, 16, "fp16", q_scale=300.0)
    run(w, [200, 90], [1, 90], 4, 2, 128, 16, "bf16", q_scale=3000.0)


def test_query_views_and_lengths_below_the_bounds(w):
    run(w, [40, 90], [1, 1], 4, 2, 128, 16, "fp16", view=True)
    run(w, [40, 90], [33, 80], 4, 2, 128, 16, "bf16", view=True, max_kv=96)


def test_sequences_without_keys_or_queries(w):
    say("attention with empty sequences")
    D, page = 128, 16
    k, v, table = paged(4, [20, 1, 40, 16], 2, D, page, "fp16", 1)
    q = randn((4, 4, D), "fp16", 2)
    kv = np.array([20, 0, 40, 16])  # sequence 1 has a query and no key; sequence 2 no query
    starts = np.array([0, 1, 2, 2, 4])
    out = w.qmm_attention(q, k, v, i32(table), i32(kv), i32(starts), 2, 40)
    want, bound = lo.attention(f64(q), f64(k), f64(v), table, kv, starts, D**-0.5)
    check(out, want, bound, "out")
    assert not out[1].any()
    assert w.qmm_attention(q[:0], k, v, i32(table), i32(kv * 0), i32(starts * 0), 0, 0).shape == (0, 4, D)


def test_equal_bits_and_other_stream(w):
    k, v, table = paged(2, [700, 300], 2, 128, 16, "bf16", 1)
    q = randn((2, 8, 128), "bf16", 2)
    args = (k, v, i32(table), i32(np.array([700, 300])), i32(np.array([0, 1, 2])), 1, 700)
    a = w.qmm_attention(q, *args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = w.qmm_attention(q, *args)
    s.synchronize()
    for _ in range(5):
        assert torch.equal(a, w.qmm_attention(q, *args))
    assert torch.equal(a, b)


def test_page_ids_outside_the_cache_are_cut(w):
    k, v, table = paged(1, [40], 1, 64, 16, "fp16", 1)
    q = randn((1, 2, 64), "fp16", 2)
    bad = table.copy()
    bad[0, 1] = 1 << 30
    bad[0, 2] = -9
    cut = np.clip(bad, 0, k.shape[0] - 1)
    rest = (i32(np.array([40])), i32(np.array([0, 1])), 1, 40)
    assert torch.equal(w.qmm_attention(q, k, v, i32(bad), *rest), w.qmm_attention(q, k, v, i32(cut), *rest))


def test_large_cache_offsets(w):
    """Pages past 2^32 bytes."""
    Hkv, D, page = 8, 256, 128
    pages = (1 << 32) // (Hkv * D * page * 2) + 5
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    for c, s in ((k, 1), (v, 2)):
        c[-2:] = randn((2, Hkv, page, D), "fp16", s)
    for n in (1, 60):
        q = randn((n, 8, D), "fp16", 3)
        table = np.array([[pages - 1, pages - 2]])
        out = w.qmm_attention(q, k, v, i32(table), i32(np.array([200])), i32(np.array([0, n])), n, 200)
        near = w.qmm_attention(q, k[-2:].contiguous(), v[-2:].contiguous(), i32(np.array([[1, 0]])), i32(np.array([200])),
                               i32(np.array([0, n])), n, 200)
        assert torch.equal(out, near)
        assert out.any()


def test_attention_in_a_graph(w):
    k, v, table = paged(2, [700, 300], 2, 128, 16, "fp16", 1)
    q = randn((2, 8, 128), "fp16", 2)
    kv = i32(np.array([700, 300]))
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    args = (k, v, i32(table), kv, i32(np.array([0, 1, 2])), 1, 700)
    w.qmm_attention(q, *args, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w.qmm_attention(q, *args, workspace=ws)
    for n in (700, 1, 433, 650):
        kv.copy_(torch.tensor([n, min(n, 300)]))
        q.copy_(randn((2, 8, 128), "fp16", n))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, w.qmm_attention(q, *args, workspace=ws)), n
