"""qmm_kv_copy_pages and qmm_kv_compact against their definition: everything is whole numbers and equal."""
import numpy as np
import pytest
import torch

from cache_cases import device
from layer_cases import DEV, i32, randn, say
from oracle import cache_oracle as co
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def pools(n, pages, seed):
    """Caches of several kinds and sizes."""
    r = np.random.default_rng(seed)
    made = []
    for i in range(n):
        shape = [(pages, 2, 576), (pages, 16), (pages, 3, 8 * 1024), (pages, 48), (pages, 20480 + 16)][i % 5]
        made.append(device(r.integers(0, 256, shape).astype(np.uint8)))
    return made


@pytest.mark.parametrize("caches,pages,n", [(1, 2, 1), (5, 40, 7), (70, 30, 10), (2, 3000, 1400), (5, 40, 0)])
def test_copy_pages(w, caches, pages, n):  # noqa: F811
    say(f"copy caches={caches} pages={pages} n={n}")
    r = np.random.default_rng(n)
    order = r.permutation(pages)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 6:
        src[1] = src[0]  # copied twice
        src[2], dst[3], src[4], dst[5] = -1, pages, 1 << 30, -7  # left out
        src[6] = dst[6]  # onto itself
    got = pools(caches, pages, 1)
    before = [c.cpu().numpy() for c in got]
    w.qmm_kv_copy_pages(got, i32(src), i32(dst))
    for c, b in zip(got, before):
        assert np.array_equal(c.cpu().numpy(), co.copy_pages(b, src, dst))


def test_copy_pages_of_16_bit_caches(w):  # noqa: F811
    k, v = (randn((9, 2, 7, 64), "bf16", i) for i in (1, 2))
    want = [t.clone() for t in (k, v)]
    for t in want:
        t[[8, 0]] = t[[3, 3]].clone()
    w.qmm_kv_copy_pages([k, v], i32(np.array([3, 3])), i32(np.array([8, 0])))
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def _table(B, pages, live, stride, page, seed, shared=0):
    r = np.random.default_rng(seed)
    per = r.multinomial(live, np.full(B, 1 / B)) if B else np.zeros(0, int)
    per = np.minimum(per, stride)
    order = r.permutation(pages)
    table = r.integers(-5, pages + 5, (B, stride)).astype(np.int32)  # what lies behind a sequence's pages may be anything
    at = 0
    for b in range(B):
        table[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
        n = min(shared, per[b])
        table[b, :n] = table[0, :n]
    lens = per * page - r.integers(0, page, B)
    return table, np.where(per > 0, lens, 0)


@pytest.mark.parametrize("B,pages,live,stride,page,shared,caches", [
    (1, 1, 1, 1, 16, 0, 1), (3, 64, 20, 12, 16, 0, 2), (4, 64, 64, 64, 8, 0, 2), (5, 100, 60, 30, 7, 3, 5), (2, 33, 0, 4, 16, 0, 1),
    (40, 5000, 3100, 200, 16, 2, 3), (64, 70001, 40000, 1000, 24, 0, 1), (3, 300, 40, 20, 16, 0, 70)])
def test_compact(w, B, pages, live, stride, page, shared, caches):  # noqa: F811
    say(f"compact B={B} pages={pages} live={live} stride={stride} shared={shared} caches={caches}")
    table, lens = _table(B, pages, live, stride, page, pages + live, shared)
    got = [device(np.random.default_rng(3).integers(0, 256, (pages, 16)).astype(np.uint8))] if pages > 10000 else pools(caches, pages, 1)
    before = [c.cpu().numpy() for c in got]
    new, moved_to, n = w.qmm_kv_compact(got, i32(table), i32(lens), page)
    want, to, count, high, free = co.compact(pages, table, lens, page)
    assert int(n) == count
    assert np.array_equal(moved_to.cpu().numpy(), to)
    assert np.array_equal(new.cpu().numpy(), want)
    for c, b in zip(got, before):
        assert np.array_equal(c.cpu().numpy(), co.copy_pages(b, high, free))


def test_compact_odd_tables(w):  # noqa: F811
    """Entries outside the cache in use, lengths below 0 and past the table, the same page in every place."""
    pages, page = 50, 16
    table = np.array([[-3, 40, 50, 7], [40, 41, 1 << 30, 44], [9, 9, 9, 9], [1, 2, 3, 4]], np.int32)
    lens = np.array([64, 10**6, 33, -5], np.int32)
    got = pools(1, pages, 1)
    before = got[0].cpu().numpy()
    new, moved_to, n = w.qmm_kv_compact(got, i32(table), i32(lens), page)
    want, to, count, high, free = co.compact(pages, table, lens, page)
    assert count == 5 and int(n) == 5
    assert np.array_equal(moved_to.cpu().numpy(), to) and np.array_equal(new.cpu().numpy(), want)
    assert np.array_equal(got[0].cpu().numpy(), co.copy_pages(before, high, free))


def test_compact_most_pages(w):  # noqa: F811
    """The most pages of a call, every other one in use."""
    pages = 1 << 20
    table = np.arange(1, pages, 2, dtype=np.int32).reshape(8, -1)
    cache = torch.arange(pages * 4, device=DEV, dtype=torch.int32).view(pages, 4)
    new, moved_to, n = w.qmm_kv_compact([cache], i32(table), i32(np.full(8, table.shape[1] * 32)), 32)
    assert int(n) == pages // 2
    # odd pages below the middle stay; the odd ones above it go to the even ones below, in order
    middle = pages // 2
    high = torch.arange(middle + 1, pages, 2, device=DEV)
    assert torch.equal(moved_to[high], torch.arange(0, middle, 2, device=DEV, dtype=torch.int32))
    low = torch.arange(1, middle, 2, device=DEV)
    assert torch.equal(moved_to[low], low.int())
    assert torch.equal(cache[moved_to[high].long()][:, 0], high.int() * 4)
    assert bool((moved_to[0::2] == -1).all())
    assert torch.equal(new, moved_to[i32(table).long()])


def test_compact_twice_changes_nothing_more(w):  # noqa: F811
    table, lens = _table(6, 200, 120, 40, 16, 5)
    got = pools(2, 200, 1)
    new, _, n = w.qmm_kv_compact(got, i32(table), i32(lens), 16)
    kept = [c.clone() for c in got]
    again, moved_to, m = w.qmm_kv_compact(got, new, i32(lens), 16)
    assert torch.equal(again, new) and int(n) == int(m)
    assert all(torch.equal(a, b) for a, b in zip(got, kept))
    assert torch.equal(moved_to[:int(m)], torch.arange(int(m), device=DEV, dtype=torch.int32)) and bool((moved_to[int(m):] == -1).all())


def test_attention_is_the_same_after_fork_and_compaction(w):  # noqa: F811
    """Sequences that are appended to, forked, dropped and packed, in both kinds of cache: their attention stays."""
    from cache_cases import paged4
    D, page, group, Hkv, Hq = 64, 16, 32, 2, 4
    lens = [100, 37, 70]
    k4, v4, table = paged4(lens, Hkv, D, page, group, 1, spare=20)
    k4, v4 = device(k4), device(v4)
    pages = len(k4)
    k16, v16 = (randn((pages, Hkv, page, D), "bf16", i) for i in (1, 2))
    q = randn((3, Hq, D), "bf16", 3)
    starts = i32(np.arange(4))
    free = [p for p in range(pages) if p not in {int(p) for row, n in zip(table, lens) for p in row[:-(-n // page)]}]

    def attend(table, lens, q=q):
        rest = (table, lens, starts[:len(q) + 1], 1, 112)
        return w.qmm_kv4_attention(q, k4, v4, *rest, group), w.qmm_attention(q, k16, v16, *rest)

    kv = i32(np.array(lens))
    before = attend(i32(table), kv)
    # Sequence 0 forked in place of 1: its last page copied to a free one.
    forked = table.copy()
    forked[1] = table[0]
    forked[1, 6] = free[3]
    w.qmm_kv_copy_pages([k4, v4, k16, v16], i32(table[0, 6:7]), i32(np.array(free[3:4])))
    kv2 = i32(np.array([100, 100, 70]))
    both = attend(i32(forked), kv2, q[[0, 0, 2]])
    for a, b in zip(both, before):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[0]) and torch.equal(a[2], b[2])
    new, moved_to, live = w.qmm_kv_compact([k4, v4, k16, v16], i32(forked), kv2, page)
    assert int(live) == 7 + 1 + 5
    after = attend(new, kv2, q[[0, 0, 2]])
    for a, b in zip(after, both):
        assert torch.equal(a, b)
    # The fork goes on to write its own last page: the other sequence keeps its keys.
    fresh = randn((1, Hkv, D), "bf16", 9)
    slot = new[1, 6].long().view(1) * page + 100 % page
    w.qmm_kv4_append(fresh, fresh, fresh, None, None, None, slot, k4, v4, group)
    kv3 = i32(np.array([100, 101, 70]))
    last = attend(new, kv3, q[[0, 0, 2]])[0]
    assert torch.equal(last[0], after[0][0]) and not torch.equal(last[1], after[0][1]) and torch.equal(last[2], after[0][2])


def test_pages_in_a_graph_and_on_another_stream(w):  # noqa: F811
    table, lens = _table(5, 100, 60, 30, 16, 7)
    src, dst = i32(np.array([1, 1, 5])), i32(np.array([9, 12, 30]))
    got = pools(3, 100, 2)
    kept = [c.clone() for c in got]
    t, n = i32(table), i32(lens)

    def step():
        w.qmm_kv_copy_pages(got, src, dst)
        return w.qmm_kv_compact(got, t, n, 16)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        new, more = _table(5, 100, 40 + 10 * seed, 30, 16, seed)
        t.copy_(i32(new))
        n.copy_(i32(more))
        for c, k in zip(got, kept):
            c.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        result = [x.clone() for x in (*out, *got)]
        for c, k in zip(got, kept):
            c.copy_(k)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            want = step()
        s.synchronize()
        for a, b in zip(result, (*want, *got)):
            assert torch.equal(a, b), seed


def test_refusals_on_tensors(w):  # noqa: F811
    a, b = pools(2, 10, 1)
    i = i32(np.array([1, 2]))
    for caches in ([], a, [a, b[:5]], [a, a.cpu()], [a, a[:, :, ::2]], [a[:0]]):
        with pytest.raises(ValueError):
            w.qmm_kv_copy_pages(caches, i, i + 3)
    with pytest.raises(TypeError):
        w.qmm_kv_copy_pages([a, None], i, i + 3)
    with pytest.raises(TypeError):
        w.qmm_kv_copy_pages([a], i.long(), i + 3)
    with pytest.raises(ValueError):
        w.qmm_kv_copy_pages([a], i, i32(np.array([1])))
    with pytest.raises(w.QmmError):  # pages of 24 bytes
        w.qmm_kv_copy_pages([torch.zeros((4, 24), dtype=torch.uint8, device=DEV)], i, i + 3)
    with pytest.raises(w.QmmError):
        w.qmm_kv_compact([a], i32(np.zeros((2, 3))), i, 0)
    with pytest.raises(ValueError):
        w.qmm_kv_compact([a], i32(np.zeros((3, 3))), i, 16)
