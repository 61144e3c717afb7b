"""qmm_kv4_attention in blocks of many rows (prompts that fill the CUs), against float64 and at the bounds of the other
tests. Many heads make enough blocks of short sequences."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import DEV, check, f64, i32, randn, say
from oracle import cache_oracle as co
from test_gpu_kv4_attention import run
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

KINDS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


def in_blocks(w, B, T, Hq, Hkv, D, max_q, max_kv):  # noqa: F811
    """Such a call needs no workspace, whatever its masks: its keys are not split."""
    return w.library().qmm_kv4_attention_workspace_bytes(B, T, Hq, Hkv, D, max_q, max_kv) == 0


def tiles(w, kv_lens, q_lens, Hq, Hkv, D, *args, **kw):  # noqa: F811
    assert in_blocks(w, len(kv_lens), sum(q_lens), Hq, Hkv, D, max(q_lens), kw.get("max_kv") or max(kv_lens))
    return run(w, kv_lens, q_lens, Hq, Hkv, D, *args, **kw)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,group", KINDS)
def test_prompts(w, D, group, dtype):  # noqa: F811
    """Ragged sequences, some of a token, rows that end inside a block."""
    tiles(w, [139, 1, 66, 133], [139, 1, 65, 70], 128, 64, D, 24, group, dtype)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 32)])
@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.0, True), (5.0, True), (300.0, False), (300.0, True)])
def test_cap_and_distance(w, D, group, softcap, slopes):  # noqa: F811
    kw = {"softcap": softcap}
    if slopes:
        kw["slopes"] = 2.0 ** -np.arange(1, 257) ** 0.5
    tiles(w, [101, 40], [101, 35], 256, 128, D, 16, group, "fp16", q_scale=4.0, **kw)


@pytest.mark.parametrize("D,group", [(64, 64), (128, 32), (256, 64)])
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "any"])
def test_masks(w, kind, D, group):  # noqa: F811
    kv_lens, q_lens = [90, 200], [90, 130]
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])
    first, end = np.zeros_like(pos), pos + 1
    r = np.random.default_rng(3)
    if kind == "window":
        first = pos + 1 - 20
    elif kind == "documents":
        first = pos // 37 * 37
    elif kind == "prefix":
        end = np.maximum(end, 50)
    else:
        first, end = r.integers(-50, 220, len(pos)), r.integers(-50, 220, len(pos))
    out = tiles(w, kv_lens, q_lens, 160, 80, D, 24, group, "bf16", first=first, end=end)
    kv = np.repeat(kv_lens, q_lens)
    empty = np.maximum(first, 0) >= np.minimum(end, kv)
    assert not f64(out)[empty].any()


@pytest.mark.parametrize("kind", ["window", "prefix"])
def test_a_key_head_for_each(w, kind):  # noqa: F811
    """Blocks of as many tokens as rows."""
    pos = np.concatenate([np.arange(150), np.arange(10, 210)])
    masks = {"first": pos - 30} if kind == "window" else {"end": np.maximum(pos + 1, 100)}
    tiles(w, [150, 210], [150, 200], 96, 96, 128, 24, 64, "fp16", **masks)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 128), (256, 32)])
def test_negative_scale_and_views(w, D, group):  # noqa: F811
    k, v, table = paged4([100, 70], 100, D, 8, group, 1)
    q = randn((170, 203 * D), "bf16", 2)[:, D:201 * D].unflatten(1, (200, D))
    starts = np.array([0, 100, 170])
    assert in_blocks(w, 2, 170, 200, 100, D, 100, 100)
    for scale in (-0.1, 0.05):
        out = w.qmm_kv4_attention(q, device(k), device(v), i32(table), i32(np.array([100, 70])), i32(starts), 100, 100, group, scale=scale)
        want, bound = co.attention(f64(q), co.parts(k, D, group, True), co.parts(v, D, group, False), table, [100, 70], starts, scale,
                                   group, dtype="bf16")
        check(out, want, bound, f"scale {scale}")


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 60000.0])
@pytest.mark.parametrize("D,group", KINDS)
def test_places_past_the_end_have_no_part(w, D, group, fill):  # noqa: F811
    tiles(w, [30, 77], [30, 70], 352, 88, D, 16, group, "fp16", fill=fill)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
def test_a_bad_group_reaches_only_queries_that_see_it(w, D, group, bad):  # noqa: F811
    kv = T = 100
    Hkv, page = 168, 16
    k, v, table = paged4([kv], Hkv, D, page, group, 1)
    q = randn((T, 336, D), "bf16", 2)
    starts = np.array([0, T])
    args = (i32(table), i32(np.array([kv])), i32(starts), T, kv, group)
    assert in_blocks(w, 1, T, 336, Hkv, D, T, kv)
    clean = w.qmm_kv4_attention(q, device(k), device(v), *args)
    half = np.frombuffer(np.float16(bad).tobytes(), np.uint8)
    for cache, head, key, which, keys in ((k, 0, 97, 0, True), (v, 1, 96, 1, False), (v, 30, 98, 0, False), (v, 2, 60, 0, False)):
        block = cache[table[0, key // page], head].reshape(page // 8, -1)[key % page // 8]
        at = co.scale_places(key % 8, 1 % (D // group), D, group, keys)[which]
        block[at:at + 2] = half
    got = w.qmm_kv4_attention(q, device(k), device(v), *args)
    assert torch.equal(got[:60], clean[:60])
    same = [h for h in range(336) if h // 2 not in (0, 1, 2, 30)]
    assert torch.equal(got[:, same], clean[:, same])
    some = [0, 1, 2, 3, 4, 5, 60, 61]  # the query heads of those key heads
    part = lambda c, keys: [x[:, [0, 1, 2, 30]] for x in co.parts(c, D, group, keys)]  # noqa: E731
    want, bound = co.attention(f64(q)[:, some], part(k, True), part(v, False), table, [kv], starts, D**-0.5, group, dtype="bf16")
    assert np.isnan(want).any(axis=(1, 2)).sum() == 40
    check(got[:, some], want, bound, "bad groups")


def test_a_bad_query_gives_nan_and_only_there(w):  # noqa: F811
    k, v, table = paged4([100], 168, 128, 16, 64, 1)
    q = randn((100, 336, 128), "bf16", 2)
    assert in_blocks(w, 1, 100, 336, 168, 128, 100, 100)
    args = (device(k), device(v), i32(table), i32(np.array([100])), i32(np.array([0, 100])), 100, 100, 64)
    clean = w.qmm_kv4_attention(q, *args)
    q[7, 3, 77] = float("nan")
    q[9, 4, 1] = float("inf")
    got = w.qmm_kv4_attention(q, *args)
    assert torch.isnan(got[7, 3]).all() and torch.isnan(got[9, 4]).all()
    got[7, 3], got[9, 4] = clean[7, 3], clean[9, 4]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("q_scale,scale", [(300.0, 1.0), (1e-4, 1.0), (1.0, 500.0), (1.0, 1e-3)])
def test_sizes(w, q_scale, scale):  # noqa: F811
    for dtype in ("fp16", "bf16"):
        tiles(w, [90], [90], 384, 192, 128, 16, 64, dtype, q_scale=q_scale, scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_padded_batches(w, D):  # noqa: F811
    """Tokens of no sequence get 0, and the others what they get without the padding."""
    say(f"kv4 attention in blocks, padded, D={D}")
    starts, kv_lens, max_q, T = [7, 137, 137, 237, 300], [130, 4, 150, 90], 110, 400
    k, v, table = paged4(kv_lens, 60, D, 16, 32, 1)
    q = randn((T, 120, D), "bf16", 2)
    rest = (device(k), device(v), i32(table), i32(np.array(kv_lens)))
    assert in_blocks(w, 4, T, 120, 60, D, max_q, 150)
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


def test_blocks_agree_with_tiles(w):  # noqa: F811
    """A long prompt in blocks, and a part of its queries in a call of their own that splits the keys."""
    kv, D, group = 3000, 128, 64
    k, v, table = paged4([kv], 8, D, 128, group, 1)
    q = randn((kv, 32, D), "bf16", 2)
    dk, dv = device(k), device(v)
    assert in_blocks(w, 1, kv, 32, 8, D, kv, kv) and not in_blocks(w, 1, 4, 32, 8, D, 4, kv)
    whole = w.qmm_kv4_attention(q, dk, dv, i32(table), i32(np.array([kv])), i32(np.array([0, kv])), kv, kv, group)
    for at in (3, 64, 1500, 3000):
        part = w.qmm_kv4_attention(q[at - 3:at].contiguous(), dk, dv, i32(table), i32(np.array([at])), i32(np.array([0, 3])), 3, kv, group)
        d = (whole[at - 3:at].float() - part.float()).norm() / part.float().norm()
        say(f"queries up to {at}: {float(d):.2e} apart")
        assert d < 2 * 2.0**-8  # two roundings


def test_in_a_graph(w):  # noqa: F811
    k, v, table = paged4([139, 66], 80, 64, 16, 32, 1)
    q = randn((205, 160, 64), "fp16", 2)
    assert in_blocks(w, 2, 205, 160, 80, 64, 139, 139)
    kv = i32(np.array([139, 66]))
    args = (device(k), device(v), i32(table), kv, i32(np.array([0, 139, 205])), 139, 139, 32)
    w.qmm_kv4_attention(q, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w.qmm_kv4_attention(q, *args)
    for n in (139, 100, 139):
        kv.copy_(torch.tensor([n, min(n, 66)]))
        q.copy_(randn(q.shape, "fp16", n))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, w.qmm_kv4_attention(q, *args)), n


def test_large_cache_offsets(w):  # noqa: F811
    """Pages past 2^32 bytes."""
    Hq, Hkv, D, page, group, n = 168, 8, 256, 128, 32, 200
    size = w.kv4_page_bytes(page, D, group)
    pages = (1 << 32) // (Hkv * size) + 5
    k = torch.zeros((pages, Hkv, size), dtype=torch.uint8, device=DEV)
    v = torch.zeros_like(k)
    last = [device(c) for c in paged4([2 * page], Hkv, D, page, group, 1, spare=0)[:2]]
    k[-2:], v[-2:] = last
    q = randn((n, Hq, D), "fp16", 3)
    assert in_blocks(w, 1, n, Hq, Hkv, D, n, n)
    rest = (i32(np.array([n])), i32(np.array([0, n])), n, n, group)
    out = w.qmm_kv4_attention(q, k, v, i32(np.array([[pages - 1, pages - 2]])), *rest)
    assert torch.equal(out, w.qmm_kv4_attention(q, *last, i32(np.array([[1, 0]])), *rest)) and out.any()


@pytest.mark.parametrize("D,group", KINDS)
def test_infinite_middles_that_all_see(w, D, group):  # noqa: F811
    """Such a group stands for NaN, in blocks and where each sequence has few rows."""
    Hq, Hkv, n, page = 336, 168, 200, 8
    k, v, table = paged4([n], Hkv, D, page, group, 1)
    for cache, head, keys, sign in ((k, 0, True, 1), (k, 1, True, -1), (v, 2, False, 1), (v, 3, False, -1)):
        at = co.scale_places(5, 0, D, group, keys)[1]
        cache[table[0, 0], head].reshape(1, -1)[0, at:at + 2] = np.frombuffer(np.float16(sign * np.inf).tobytes(), np.uint8)
    some = np.r_[0:8, 20]
    part = lambda c, keys: [x[:, [0, 1, 2, 3, 10]] for x in co.parts(c, D, group, keys)]  # noqa: E731
    for T in (100, 3):
        assert in_blocks(w, 1, T, Hq, Hkv, D, T, n) or T == 3
        q = randn((T, Hq, D), "fp16", 2)
        got = w.qmm_kv4_attention(q, device(k), device(v), i32(table), i32(np.array([n])), i32(np.array([0, T])), T, n, group)
        assert torch.isfinite(got[:, 8:]).all()
        want, bound = co.attention(f64(q)[:, np.r_[0:8, 20, 21]], part(k, True), part(v, False), table, [n], [0, T], D**-0.5, group)
        check(got[:, some], want[:, :9], bound[:, :9], f"T={T}")
