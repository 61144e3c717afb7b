"""qmm_kv4_attention in parts of the keys, which the bound of the lengths asks for: short sequences too then go through
the shares, the hand-over and the join. Against float64 and at the bounds of the other tests."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import check, f64, i32, randn
from oracle import cache_oracle as co
from test_gpu_kv4_attention import run
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

KINDS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]
BOUND = 4200


def parts(w, kv_lens, q_lens, Hq, Hkv, D, *args, **kw):  # noqa: F811
    assert w.library().qmm_kv4_attention_workspace_bytes(len(kv_lens), sum(q_lens), Hq, Hkv, D, max(q_lens), BOUND) > 0
    return run(w, kv_lens, q_lens, Hq, Hkv, D, *args, max_kv=BOUND, **kw)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,group", KINDS)
def test_tokens_and_prompts(w, D, group, dtype):  # noqa: F811
    """Sequences of one part, of several, without a query; one and more tiles a key head."""
    parts(w, [1300, 1, 133, 40], [1, 1, 1, 1], 8, 2, D, 24, group, dtype)
    parts(w, [1100, 7, 150, 300], [3, 7, 20, 1], 6, 2, D, 16, group, dtype)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 32)])
@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.0, True), (5.0, True), (300.0, False), (300.0, True)])
def test_cap_and_distance(w, D, group, softcap, slopes):  # noqa: F811
    kw = {"softcap": softcap}
    if slopes:
        kw["slopes"] = 2.0 ** -np.arange(1, 9) ** 0.5
    for q_lens in ([1, 1], [17, 5]):
        parts(w, [700, 140], q_lens, 8, 2, D, 16, group, "fp16", q_scale=4.0, **kw)


@pytest.mark.parametrize("q_lens", [[1, 1], [40, 30]])
@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (256, 64)])
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "any"])
def test_masks(w, kind, D, group, q_lens):  # noqa: F811
    kv_lens = [690, 260]
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])
    first, end = np.zeros_like(pos), pos + 1
    r = np.random.default_rng(3)
    if kind == "window":
        first = pos + 1 - 300
    elif kind == "documents":
        first = pos // 370 * 370
    elif kind == "prefix":
        end = np.maximum(end, 500)
    else:
        first, end = r.integers(-50, 700, len(pos)), r.integers(-50, 700, len(pos))
    out = parts(w, kv_lens, q_lens, 8, 4, D, 24, group, "bf16", first=first, end=end)
    empty = np.maximum(first, 0) >= np.minimum(end, np.repeat(kv_lens, q_lens))
    assert not f64(out)[empty].any()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 60000.0])
@pytest.mark.parametrize("D,group", KINDS)
def test_places_past_the_end_have_no_part(w, D, group, fill):  # noqa: F811
    parts(w, [701, 30], [1, 1], 8, 2, D, 16, group, "fp16", fill=fill)
    parts(w, [333, 30], [20, 3], 8, 2, D, 16, group, "fp16", fill=fill)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T", [1, 30])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
def test_a_bad_group_reaches_only_queries_that_see_it(w, T, D, group, bad):  # noqa: F811
    kv, page = 900, 16
    k, v, table = paged4([kv], 4, D, page, group, 1)
    q = randn((T, 8, D), "bf16", 2)
    half = np.frombuffer(np.float16(bad).tobytes(), np.uint8)
    for cache, head, key, which, keys in ((k, 0, 897, 0, True), (k, 2, 300, 1, True), (v, 1, 450, 1, False), (v, 0, 898, 0, False)):
        block = cache[table[0, key // page], head].reshape(page // 8, -1)[key % page // 8]
        at = co.scale_places(key % 8, 1 % (D // group), D, group, keys)[which]
        block[at:at + 2] = half
    rest = (np.array([kv]), np.array([0, T]))
    out = w.qmm_kv4_attention(q, device(k), device(v), i32(np.pad(table, ((0, 0), (0, 300)))), i32(rest[0]), i32(rest[1]), T, BOUND, group)
    want, bound = co.attention(f64(q), co.parts(k, D, group, True), co.parts(v, D, group, False), table, *rest, D**-0.5, group, dtype="bf16")
    assert np.isnan(want).any()
    check(out, want, bound, "bad groups")


def test_equal_bits_and_a_graph(w):  # noqa: F811
    """The bound alone chooses: the same lengths give the same bits call after call, and replayed for other lengths."""
    k, v, table = paged4([700, 300], 2, 128, 16, 64, 1)
    q = randn((2, 8, 128), "fp16", 2)
    kv = i32(np.array([700, 300]))
    args = (device(k), device(v), i32(np.pad(table, ((0, 0), (0, 230)))), kv, i32(np.array([0, 1, 2])), 1, BOUND, 64)
    first = w.qmm_kv4_attention(q, *args)
    for _ in range(5):
        assert torch.equal(first, w.qmm_kv4_attention(q, *args))
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
