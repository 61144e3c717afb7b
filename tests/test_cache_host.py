"""The 4-bit cache and the care of pages without a GPU: exported symbols, refusals before any launch, sizes, and pins
of their oracle.

The pointers of the refused calls are fake and never dereferenced; a call that got past validation would report
QMM_ERR_HIP on a machine without a GPU.
"""
import ctypes
import math
import os
import re

import numpy as np
import pytest

from oracle import cache_oracle as co
from test_layer_host import A, ALIGN, FLAGS, GROUP, MIS, NULL, ROOT, SHAPE, WORKSPACE, _lib, lib  # noqa: F401


def test_exports():
    import weight_only_group_amd as w
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qmm_cache.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(qmm_[a-z0-9_]+)\s*\(", text))
    assert declared == set(w.cache.EXPORTS)
    _lib()
    raw = ctypes.CDLL(w.LIB_PATH)
    for name in declared:
        assert getattr(raw, name) is not None


def test_page_bytes():
    lib = _lib()
    for D in (64, 128, 256):
        for group in (32, 64, 128):
            for page in (8, 16, 24, 128):
                want = page * (D // 2 + 4 * D // group) if group <= D else 0
                assert lib.qmm_kv4_page_bytes(page, D, group) == want
                assert want == 0 or want == page // 8 * co.block_bytes(D, group)
    for bad in ((0, 128, 32), (-8, 128, 32), (12, 128, 32), (16, 96, 32), (16, 128, 16), (16, 128, 256), (16, 128, 0)):
        assert lib.qmm_kv4_page_bytes(*bad) == 0, bad


def _append(lib, **kw):  # noqa: F811
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, T=3, Hq=8, Hkv=2, D=128, gs=64, cos=A, sin=A, R=64, P=10, pos=A, slots=A,
             out=A, kc=A, vc=A, pages=4, page=16, fl=0)
    a.update(kw)
    return lib.qmm_kv4_append(*a.values(), None)


APPEND = [(dict(T=-1), SHAPE), (dict(T=2**31 - 1), SHAPE), (dict(Hq=7), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=96), SHAPE),
          (dict(R=40), SHAPE), (dict(R=144), SHAPE), (dict(R=-16), SHAPE), (dict(P=0), SHAPE), (dict(qs=1020), SHAPE),
          (dict(qs=1016), SHAPE), (dict(ks=128), SHAPE), (dict(vs=-256), SHAPE), (dict(pages=0), SHAPE), (dict(page=0), SHAPE),
          (dict(page=12), SHAPE), (dict(page=-16), SHAPE), (dict(pages=2**27, page=16), SHAPE), (dict(gs=16), GROUP),
          (dict(gs=256), GROUP), (dict(gs=0), GROUP), (dict(gs=-1), GROUP), (dict(gs=128, D=64), GROUP),
          (dict(fl=2), FLAGS), (dict(q=None), NULL), (dict(cos=None), NULL), (dict(pos=None), NULL), (dict(slots=None), NULL),
          (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(out=MIS), ALIGN), (dict(v=MIS), ALIGN), (dict(kc=MIS), ALIGN),
          (dict(sin=MIS), ALIGN), (dict(slots=MIS), ALIGN)]


@pytest.mark.parametrize("kw,want", APPEND, ids=str)
def test_append_refuses(lib, kw, want):  # noqa: F811
    assert _append(lib, **kw) == want, lib.qmm_last_error()
    assert lib.qmm_last_error()


def _gather(lib, **kw):  # noqa: F811
    a = dict(kc=A, vc=A, pages=4, Hkv=2, page=16, D=128, gs=64, slots=A, T=3, fl=0, k=A, v=A)
    a.update(kw)
    return lib.qmm_kv4_gather(*a.values(), None)


GATHER = [(dict(T=-1), SHAPE), (dict(T=2**31 - 1), SHAPE), (dict(Hkv=0), SHAPE), (dict(Hkv=5000), SHAPE), (dict(D=32), SHAPE),
          (dict(page=20), SHAPE), (dict(pages=0), SHAPE), (dict(gs=48), GROUP), (dict(fl=8), FLAGS), (dict(kc=None), NULL),
          (dict(vc=None), NULL), (dict(slots=None), NULL), (dict(k=None), NULL), (dict(v=MIS), ALIGN), (dict(slots=MIS), ALIGN),
          (dict(vc=MIS), ALIGN)]


@pytest.mark.parametrize("kw,want", GATHER, ids=str)
def test_gather_refuses(lib, kw, want):  # noqa: F811
    assert _gather(lib, **kw) == want, lib.qmm_last_error()


def _attention(lib, **kw):  # noqa: F811
    a = dict(q=A, qs=1024, T=3, Hq=8, Hkv=2, D=128, gs=32, kc=A, vc=A, pages=4, page=16, table=A, ts=4, kv=A, starts=A, B=2,
             max_q=2, max_kv=64, first=None, end=None, scale=0.1, cap=0.0, slopes=None, fl=0, out=A, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.qmm_kv4_attention(*a.values(), None)


ATTENTION = [(dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(max_q=-1), SHAPE), (dict(Hq=9), SHAPE),
             (dict(D=80), SHAPE), (dict(max_kv=65), SHAPE), (dict(max_kv=-1), SHAPE), (dict(ts=0), SHAPE),
             (dict(ts=2**28, page=8), SHAPE), (dict(qs=1000), SHAPE), (dict(scale=math.nan), SHAPE), (dict(cap=-1.0), SHAPE),
             (dict(cap=math.inf), SHAPE), (dict(page=20), SHAPE), (dict(gs=16), GROUP), (dict(gs=256), GROUP), (dict(fl=2), FLAGS),
             (dict(q=None), NULL), (dict(table=None), NULL), (dict(kv=None), NULL), (dict(starts=None), NULL), (dict(out=None), NULL),
             (dict(kc=None), NULL), (dict(q=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(first=A + 2), ALIGN),
             (dict(slopes=A + 1), ALIGN), (dict(pages=0), SHAPE), (dict(T=2**30), SHAPE),
             (dict(ws=None, max_kv=2**20, ts=2**20), WORKSPACE), (dict(ws=MIS, max_kv=2**20, ts=2**20), ALIGN),
             (dict(B=65535, T=2**20, max_q=2**20), SHAPE)]


@pytest.mark.parametrize("kw,want", ATTENTION, ids=str)
def test_attention_refuses(lib, kw, want):  # noqa: F811
    assert _attention(lib, **kw) == want, lib.qmm_last_error()


def _pools(n=2, size=4096, at=A):
    return (ctypes.c_void_p * max(n, 1))(*[at] * max(n, 1)), (ctypes.c_int64 * max(n, 1))(*[size] * max(n, 1)), n


def _copy(lib, pools=None, **kw):  # noqa: F811
    a = dict(pages=10, src=A, dst=A, n=3)
    a.update(kw)
    return lib.qmm_kv_copy_pages(*(pools or _pools()), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(pools=_pools(-1)), SHAPE), (dict(pools=_pools(4097)), SHAPE), (dict(pools=(None, _pools()[1], 2)), NULL),
    (dict(pools=(_pools()[0], None, 2)), NULL), (dict(pools=_pools(at=None)), NULL), (dict(pools=_pools(at=MIS)), ALIGN),
    (dict(pools=_pools(size=0)), SHAPE), (dict(pools=_pools(size=24)), SHAPE), (dict(pools=_pools(size=2**31)), SHAPE),
    (dict(pages=0), SHAPE), (dict(n=-1), SHAPE), (dict(src=None), NULL), (dict(dst=None), NULL), (dict(dst=A + 2), ALIGN)], ids=str)
def test_copy_refuses(lib, kw, want):  # noqa: F811
    assert _copy(lib, **kw) == want, lib.qmm_last_error()


def _compact(lib, pools=None, **kw):  # noqa: F811
    a = dict(pages=10, table=A, ts=4, kv=A, B=2, page=16, new=A, moved=A, live=A, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.qmm_kv_compact(*(pools or _pools()), *a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(pools=_pools(-1)), SHAPE), (dict(pools=_pools(at=None)), NULL), (dict(pools=_pools(size=8)), SHAPE),
    (dict(pages=0), SHAPE), (dict(pages=2**20 + 1), SHAPE), (dict(B=-1), SHAPE), (dict(ts=0), SHAPE), (dict(B=2**16, ts=2**15), SHAPE),
    (dict(page=0), SHAPE), (dict(table=None), NULL), (dict(kv=None), NULL), (dict(new=None), NULL), (dict(moved=None), NULL),
    (dict(live=None), NULL), (dict(live=A + 1), ALIGN), (dict(moved=A + 2), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(wsb=64), WORKSPACE), (dict(ws=MIS), ALIGN)], ids=str)
def test_compact_refuses(lib, kw, want):  # noqa: F811
    assert _compact(lib, **kw) == want, lib.qmm_last_error()


def test_calls_without_work(lib):  # noqa: F811
    assert _append(lib, T=0, kc=None) == 0
    assert _gather(lib, T=0, kc=None) == 0
    assert _attention(lib, T=0) == 0 and _attention(lib, B=0) == 0 and _attention(lib, max_q=0) == 0
    assert _copy(lib, n=0, src=None) == 0 and _copy(lib, pools=(None, None, 0)) == 0


def test_workspace_sizes():
    lib = _lib()
    n = lib.qmm_kv4_attention_workspace_bytes(1, 1, 32, 8, 128, 1, 8192)
    assert n > 128 << 10
    for bad in ((0, 1, 32, 8, 128, 1, 8192), (1, 0, 32, 8, 128, 1, 8192), (1, 1, 32, 7, 128, 1, 8192), (1, 1, 32, 8, 100, 1, 8192)):
        assert lib.qmm_kv4_attention_workspace_bytes(*bad) == 0
    assert lib.qmm_kv_compact_workspace_bytes(1000) >= (128 << 10) + 4000
    assert lib.qmm_kv_compact_workspace_bytes(0) == lib.qmm_kv_compact_workspace_bytes(2**20 + 1) == 0


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    import weight_only_group_amd as w
    _lib()
    c = torch.zeros((4, 2, w.kv4_page_bytes(16, 64, 32)), dtype=torch.uint8)
    q = torch.zeros((1, 4, 64), dtype=torch.float16)
    slots, i = torch.zeros(1, dtype=torch.int64), torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_kv4_append(q, q[:, :2], q[:, :2], None, None, None, slots, c, c, 32)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_kv4_gather(c, c, slots, 64, 32)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_kv4_attention(q, c, c, i, i[0, :1], i[0], 1, 16, 32)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_kv_copy_pages([c], i[0], i[0])
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_kv_compact([c], i, i[0, :1], 16)
    with pytest.raises(ValueError):
        w.qmm_kv_copy_pages([], i[0], i[0])
    with pytest.raises(ValueError, match="multiple of 8"):
        w.kv4_page_bytes(12, 64, 32)


# ---- pins of the oracle ------------------------------------------------------------------

def test_places_are_a_permutation():
    for D in (64, 128, 256):
        for place in (co.key_place, co.value_place):
            every = {place(t, d, D) for t in range(8) for d in range(D)}
            assert every == {(byte, half) for byte in range(4 * D) for half in range(2)}
        for group in (32, 64, 128):
            if group > D:
                continue
            for keys in (True, False):
                at = sorted(p for t in range(8) for g in range(D // group) for p in co.scale_places(t, g, D, group, keys))
                assert at == list(range(4 * D, co.block_bytes(D, group), 2))


@pytest.mark.parametrize("scale", [1e-7, 1e-3, 1.0, 300.0, 9000.0, 1e6])
def test_codes_are_the_nearest(scale):
    """A value is at most half a step off what its code stands for; a step and a half at the group's ends, where the
    8 bits of the scale and the rounded middle leave the range a little short; and what is past the limit is cut."""
    r = np.random.default_rng(1)
    x = (r.standard_normal((50, 128)) * scale + r.standard_normal((50, 1)) * scale).astype(np.float32)
    s, m, c = co.quantise(x, 32)
    assert c.min() >= 0 and c.max() <= 15
    step = np.repeat(s.astype(np.float64), 32, axis=1)
    held = np.repeat(m.astype(np.float64), 32, axis=1) + step * (c - 8)
    want = np.clip(x.astype(np.float64), -co.LARGEST, co.LARGEST)
    # half a step; at the ends the scale's rounding times 8 (2^-8 8 / 2 steps), the middle's and fp16's smallest step
    room = 0.5 * step + 8 * step * 2.0**-8 + np.abs(np.repeat(m.astype(np.float64), 32, axis=1)) * 2.0**-11 + 8 * 2.0**-24
    assert (np.abs(held - want) <= room).all()
    bits = np.frexp(s.astype(np.float64))[0] * 256
    assert (bits == np.rint(bits)).all()  # 8 significant bits


def test_constant_groups_and_nan():
    x = np.full((1, 64), 3.25, np.float32)
    s, m, c = co.quantise(x, 32)
    assert (s == 0).all() and (m == 3.25).all() and (c == 8).all()
    x[0, 40] = np.nan
    s, m, c = co.quantise(x, 32)
    assert np.isnan(s[0, 1]) and np.isnan(m[0, 1]) and s[0, 0] == 0 and m[0, 0] == 3.25


def test_what_is_put_is_read_back():
    r = np.random.default_rng(2)
    for D, group in ((64, 32), (128, 128), (256, 64)):
        for keys in (True, False):
            cache = r.integers(0, 256, (2, 2, 16 * (D // 2 + 4 * D // group))).astype(np.uint8)
            before = [p.copy() for p in co.parts(cache, D, group, keys)]
            s, m, c = co.quantise(r.standard_normal(D), group)
            co.put(cache, 1, 0, 11, s, m, c, group, keys)
            step, middle = co.parts(cache, D, group, keys)
            assert np.array_equal(step[1, 0, 11], np.repeat(s, group).astype(float) * (c - 8))
            assert np.array_equal(middle[1, 0, 11], np.repeat(m, group).astype(float))
            step[1, 0, 11], middle[1, 0, 11] = before[0][1, 0, 11], before[1][1, 0, 11]
            assert np.array_equal(step, before[0], equal_nan=True) and np.array_equal(middle, before[1], equal_nan=True)


def test_codes_times_scales_are_halves():
    """s (c - 8) and 24 s are fp16 numbers for every scale that the append can give."""
    e = np.ldexp(1.0, np.arange(-24, 8))
    s = np.unique((e[:, None] * np.arange(1, 256)).astype(np.float16).astype(np.float64))
    s = s[(s <= 2192) & (np.frexp(s)[0] * 256 == np.rint(np.frexp(s)[0] * 256))]
    for c in [*range(-8, 8), 24]:
        assert np.array_equal((s * c).astype(np.float16).astype(np.float64), s * c)


# ---- the bound on the attention's error has teeth -------------------------------------------

@pytest.mark.parametrize("mistake", [None, "middle_of_a_group_lost", "one_code_off", "last_key_lost", "query_in_4_bits", "next_scale"])
def test_planted_mistakes_pass_no_bound(mistake):
    r = np.random.default_rng(4)
    D, group, page, n = 64, 32, 16, 40
    q = r.standard_normal((1, 1, D)).astype(np.float16).astype(np.float64)
    x = r.standard_normal((2, 3, 1, page, D)) + 0.5
    held = []
    for keys in (0, 1):
        s, m, c = co.quantise(x[keys], group)
        held.append((np.repeat(s, group, -1).astype(float) * (c - 8), np.repeat(m, group, -1).astype(float)))
    table = np.array([[2, 0, 1]])
    args = lambda q, k, v, n: (q, k, v, table, [n], [0, 1], D**-0.5, group)  # noqa: E731
    want, bound = co.attention(*args(q, *held, n))
    (ks, km), (vs, vm) = ([p.copy() for p in h] for h in held)
    if mistake == "middle_of_a_group_lost":
        km[2, 0, 3, :32] = 0
    elif mistake == "one_code_off":
        vs[0, 0, 5, 7] += vs[0, 0, 5][vs[0, 0, 5] > 0].min()
    elif mistake == "last_key_lost":
        n -= 1
    elif mistake == "query_in_4_bits":
        q = np.ldexp(np.rint(np.frexp(q)[0] * 16), np.frexp(q)[1] - 4)
    elif mistake == "next_scale":
        ks[2, 0, 3] *= 1.3
    got = co.attention(*args(q, (ks, km), (vs, vm), n))[0].astype(np.float16).astype(np.float64)
    assert (np.abs(got - want) <= bound).all() == (mistake is None)
