"""qmm_kv4_attention where a block takes two tiles of sixteen rows (many short sequences of several tiles each, whose keys
are not split), against float64 and at the bounds of the other tests. Many heads make enough tiles of few sequences."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import check, f64, i32, randn, say
from oracle import cache_oracle as co
from test_gpu_kv4_attention import run
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

KINDS = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]
HQ, HKV = 256, 128


def wide(w, kv_lens, q_lens, D, *args, **kw):  # noqa: F811
    """Too few rows a sequence for blocks of many rows; no workspace, as the keys are not split."""
    B, T, group = len(kv_lens), sum(q_lens), HQ // HKV
    assert T * group < 128 * B and 16 < max(q_lens) * group <= 128
    assert w.library().qmm_kv4_attention_workspace_bytes(B, T, HQ, HKV, D, max(q_lens), kw.get("max_kv") or max(kv_lens)) == 0
    return run(w, kv_lens, q_lens, HQ, HKV, D, *args, **kw)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,group", KINDS)
def test_ragged(w, D, group, dtype):  # noqa: F811
    """Sequences that end in a block's first tile, in its second, with one row, and behind many keys."""
    wide(w, [40, 17, 30, 200], [40, 17, 1, 8], D, 24, group, dtype)


@pytest.mark.parametrize("D,group", [(64, 32), (128, 64)])
@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.0, True), (5.0, True), (300.0, True)])
def test_cap_and_distance(w, D, group, softcap, slopes):  # noqa: F811
    kw = {"softcap": softcap}
    if slopes:
        kw["slopes"] = 2.0 ** -np.arange(1, HQ + 1) ** 0.5
    wide(w, [70, 40, 33, 9], [40, 35, 33, 9], D, 16, group, "fp16", q_scale=4.0, **kw)


@pytest.mark.parametrize("D,group", [(64, 64), (128, 32)])
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "any"])
def test_masks(w, kind, D, group):  # noqa: F811
    kv_lens, q_lens = [90, 60, 150, 40], [40, 30, 20, 40]
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
        first, end = r.integers(-50, 170, len(pos)), r.integers(-50, 170, len(pos))
    out = wide(w, kv_lens, q_lens, D, 24, group, "bf16", first=first, end=end)
    empty = np.maximum(first, 0) >= np.minimum(end, np.repeat(kv_lens, q_lens))
    assert not f64(out)[empty].any()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 60000.0])
@pytest.mark.parametrize("D,group", KINDS)
def test_places_past_the_end_have_no_part(w, D, group, fill):  # noqa: F811
    wide(w, [30, 77, 41, 3], [30, 40, 17, 3], D, 16, group, "fp16", fill=fill)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64)])
def test_a_bad_group_reaches_only_queries_that_see_it(w, D, group, bad):  # noqa: F811
    B, n, page = 5, 40, 8
    kv_lens, starts = [n] * B, np.arange(B + 1) * n
    k, v, table = paged4(kv_lens, HKV, D, page, group, 1)
    q = randn((B * n, HQ, D), "bf16", 2)
    rest = (i32(table), i32(np.array(kv_lens)), i32(starts), n, n, group)
    clean = w.qmm_kv4_attention(q, device(k), device(v), *rest)
    half = np.frombuffer(np.float16(bad).tobytes(), np.uint8)
    for cache, head, key, which, keys in ((k, 0, 37, 0, True), (v, 1, 36, 1, False), (v, 30, 5, 0, False)):
        block = cache[table[2, key // page], head].reshape(page // 8, -1)[key % page // 8]
        at = co.scale_places(key % 8, 1 % (D // group), D, group, keys)[which]
        block[at:at + 2] = half
    got = w.qmm_kv4_attention(q, device(k), device(v), *rest)
    others = np.r_[0:2 * n, 3 * n:B * n]
    assert torch.equal(got[others], clean[others]) and torch.equal(got[2 * n:2 * n + 5], clean[2 * n:2 * n + 5])
    same = [h for h in range(HQ) if h // 2 not in (0, 1, 30)]
    assert torch.equal(got[:, same], clean[:, same])
    some = [0, 1, 2, 3, 60, 61]  # the query heads of those key heads
    part = lambda c, keys: [x[:, [0, 1, 30]] for x in co.parts(c, D, group, keys)]  # noqa: E731
    want, bound = co.attention(f64(q)[2 * n:3 * n][:, some], part(k, True), part(v, False), table[2:3], [n], [0, n], D**-0.5, group,
                               dtype="bf16")
    assert np.isnan(want).any()
    check(got[2 * n:3 * n][:, some], want, bound, "bad groups")


def test_padding_and_equal_bits(w):  # noqa: F811
    """Tokens of no sequence get 0; the others the same whatever stands around them, call after call."""
    say("kv4 attention, two tiles a block, padded")
    D, group, B, n = 128, 64, 6, 21
    kv_lens = [50, 21, 90, 33, 21, 60]
    k, v, table = paged4(kv_lens, HKV, D, 16, group, 1)
    rest = (device(k), device(v), i32(table), i32(np.array(kv_lens)))
    starts = 5 + np.arange(B + 1) * n
    q = randn((5 + B * n + 9, HQ, D), "fp16", 2)
    out = torch.ones_like(q)
    w.qmm_kv4_attention(q, *rest, i32(starts), n, 90, group, out=out)
    assert not out[:5].any() and not out[5 + B * n:].any()
    alone = w.qmm_kv4_attention(q[5:5 + B * n].contiguous(), *rest, i32(starts - 5), n, 90, group)
    assert torch.equal(out[5:5 + B * n], alone) and alone.any()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        again = w.qmm_kv4_attention(q[5:5 + B * n].contiguous(), *rest, i32(starts - 5), n, 90, group)
    s.synchronize()
    assert torch.equal(alone, again)
    # Sequences in calls of their own, of fewer tiles and so in parts or one tile a block: near.
    for b in (0, 2, 5):
        one = w.qmm_kv4_attention(q[starts[b]:starts[b + 1]].contiguous(), *rest[:2], i32(table[b:b + 1]), i32(np.array(kv_lens[b:b + 1])),
                                  i32(np.array([0, n])), n, 90, group)
        d = (one.float() - out[starts[b]:starts[b + 1]].float()).norm() / one.float().norm()
        assert d < 2 * 2.0**-11, b  # two roundings
