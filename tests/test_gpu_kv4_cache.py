"""qmm_kv4_append and qmm_kv4_gather against their definition. The bytes of the cache are equal to the oracle's: its
steps are fp32 operations, correctly rounded, on keys that are rotated in float64 and rounded once. The rotated
query errs by at most 3 fp32 roundings of |a c| + |b s| and one of the data type; a gathered value by one fp32 rounding
of the value and one of the data type."""
import numpy as np
import pytest
import torch

from cache_cases import device, filled
from layer_cases import DEV, TYPES, check, f64, i32, randn, say
from oracle import cache_oracle as co
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required")
    import weight_only_group_amd as mod
    mod.library()
    return mod


def _case(T, Hq, Hkv, D, R, page, group, dtype, seed, fused, P=50, scale=1.0):
    r = np.random.default_rng(seed)
    if fused:
        rows = randn((T, (Hq + 2 * Hkv) * D + 8), dtype, seed, scale)
        q, k, v = (t.unflatten(1, (-1, D)) for t in rows[:, :-8].split([Hq * D, Hkv * D, Hkv * D], dim=1))
    else:
        q, k, v = (randn((T, h, D), dtype, seed + i, scale) for i, h in enumerate((Hq, Hkv, Hkv)))
    angle = r.uniform(0, 6.28, (P, R // 2))
    cos, sin = (torch.from_numpy(f(angle).astype(np.float32)).to(DEV) for f in (np.cos, np.sin))
    pages = T // page + 3
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    caches = [r.integers(0, 256, (pages, Hkv, page * (D // 2 + 4 * D // group))).astype(np.uint8) for _ in range(2)]
    return q, k, v, cos, sin, r.integers(0, P, T).astype(np.int32), slots, *caches


def _append(w, T, Hq, Hkv, D, R, page, group, dtype, adjacent, fused, scale=1.0, change=None):
    say(f"kv4 append T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} page={page} group={group} {dtype} adjacent={adjacent} fused={fused}")
    q, k, v, cos, sin, pos, slots, kc, vc = _case(T, Hq, Hkv, D, R, page, group, dtype, T + D + R, fused, scale=scale)
    if change:
        change(k, v, slots, len(kc) * page)
    dk, dv = device(kc), device(vc)
    out = w.qmm_kv4_append(q, k, v, cos if R else None, sin if R else None, i32(pos), device(slots), dk, dv, group, adjacent=adjacent)
    cs, sn = (f64(cos), f64(sin)) if R else (None, None)
    want, size = co.append(f64(q), f64(k), f64(v), cs, sn, pos, slots, kc, vc, group, page, adjacent)
    u, tiny = lo.ROUNDOFF[dtype], lo.TINY[dtype]
    rot = np.arange(D) < R
    check(out, want, np.where(rot, u * np.abs(want) + (1 + u) * 3 * lo.F32 * size + tiny, 0), "q")
    assert np.array_equal(dk.cpu().numpy(), kc), "k_cache"
    assert np.array_equal(dv.cpu().numpy(), vc), "v_cache"


CASES = [(1, 1, 1, 64, 64, 8, 32), (1, 8, 2, 128, 128, 16, 32), (7, 32, 8, 128, 64, 16, 64), (13, 5, 1, 256, 256, 24, 32),
         (3, 6, 3, 64, 16, 8, 64), (130, 4, 4, 128, 96, 64, 128), (2, 3, 3, 256, 112, 104, 64), (5, 2, 1, 128, 0, 8, 32),
         (40, 2, 2, 256, 128, 16, 128)]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("adjacent", [True, False])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,group", CASES)
def test_append(w, T, Hq, Hkv, D, R, page, group, dtype, adjacent, fused):
    def skip(k, v, slots, most):
        if T > 2:
            slots[1], slots[2] = -1, most  # the second one past the cache

    _append(w, T, Hq, Hkv, D, R, page, group, dtype, adjacent, fused, change=skip)


@pytest.mark.parametrize("scale", [1e-6, 3e-4, 100.0, 12000.0])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_sizes(w, dtype, scale):
    _append(w, 20, 2, 2, 128, 64, 16, 32, dtype, False, True, scale=scale)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_consecutive_and_special_values(w, dtype):
    """Runs of slots that fill blocks and end inside them; equal values, zeros, infinities and NaN."""
    def special(k, v, slots, most):
        slots[:] = np.concatenate([np.arange(5, 5 + 30), np.arange(40, 40 + len(slots) - 30)])
        for t in (k, v):
            t[3, 0, :64] = 2.5
            t[4] = 0
            t[5, 0, 7] = float("inf")
            t[6, 1, 70] = float("-inf")
            t[7, 1, 127] = float("nan")
            t[8, 0, :32] = -0.0

    _append(w, 90, 2, 2, 128, 0, 16, 32, dtype, False, False, change=special)
    _append(w, 90, 2, 2, 128, 0, 16, 128, dtype, False, True, change=special)


def test_append_positions_are_cut_to_the_table(w):
    q, k, v, cos, sin, pos, slots, kc, vc = _case(4, 2, 1, 64, 64, 8, 32, "fp16", 3, False)
    bad = np.array([-5, 10**9, 2, 49], np.int32)
    call = lambda p, c: w.qmm_kv4_append(q, k, v, cos, sin, i32(p), device(slots), c, c.clone(), 32)  # noqa: E731
    a, b = device(kc), device(kc)
    assert torch.equal(call(bad, a), call(np.clip(bad, 0, 49), b)) and torch.equal(a, b)


def test_append_nothing_and_other_stream(w):
    q, k, v, cos, sin, pos, slots, kc, vc = _case(9, 2, 1, 128, 64, 8, 64, "bf16", 4, True)
    dk, dv = device(kc), device(vc)
    assert w.qmm_kv4_append(q[:0], k[:0], v[:0], cos, sin, i32(pos[:0]), device(slots[:0]), dk, dv, 64).shape == (0, 2, 128)
    assert np.array_equal(dk.cpu().numpy(), kc)
    first = w.qmm_kv4_append(q, k, v, cos, sin, i32(pos), device(slots), dk, dv, 64)
    other = device(kc), device(vc)
    args = i32(pos), device(slots)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = w.qmm_kv4_append(q, k, v, cos, sin, *args, *other, 64)
    s.synchronize()
    assert torch.equal(first, again) and torch.equal(dk, other[0]) and torch.equal(dv, other[1])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hkv,D,page,group", [(1, 1, 64, 8, 32), (37, 2, 128, 16, 128), (100, 3, 256, 24, 32), (5, 5, 64, 64, 64),
                                                (300, 1, 128, 8, 32)])
def test_gather(w, T, Hkv, D, page, group, dtype):
    say(f"kv4 gather T={T} Hkv={Hkv} D={D} page={page} group={group} {dtype}")
    pages = 6
    kc, vc = (filled(pages, Hkv, page, D, group, keys, T + D, 2.0) for keys in (True, False))
    slots = np.random.default_rng(T).integers(0, pages * page, T)  # some of them twice
    if T > 2:
        slots[1], slots[2] = -3, pages * page
    got = w.qmm_kv4_gather(device(kc), device(vc), device(slots), D, group, dtype=TYPES[dtype])
    inside = ((slots >= 0) & (slots < pages * page))[:, None, None]
    at = np.clip(slots, 0, pages * page - 1)
    u, tiny = lo.ROUNDOFF[dtype], lo.TINY[dtype]
    for t, cache, keys in zip(got, (kc, vc), (True, False)):
        step, middle = co.parts(cache, D, group, keys)
        want = (step + middle)[at // page, :, at % page] * inside
        check(t, want, np.abs(want) * (u + (1 + u) * lo.F32) + tiny, "keys" if keys else "values")


def test_gather_bad_groups(w):
    """Scales or middles that are not finite: the whole group is NaN, and nothing else."""
    D, group, page = 64, 32, 8
    kc, vc = (filled(1, 1, page, D, group, keys, 5) for keys in (True, False))
    for cache, keys in ((kc, True), (vc, False)):
        for t, g, which, v in ((1, 0, 0, np.inf), (2, 1, 1, -np.inf), (3, 0, 1, np.nan), (4, 1, 0, np.nan)):
            at = co.scale_places(t, g, D, group, keys)[which]
            cache[0, 0, at:at + 2] = np.frombuffer(np.float16(v).tobytes(), np.uint8)
    got = w.qmm_kv4_gather(device(kc), device(vc), torch.arange(8, device=DEV), D, group)
    for t, cache, keys in zip(got, (kc, vc), (True, False)):
        want = sum(co.parts(cache, D, group, keys))[0, 0][:, None]
        assert np.isnan(want).sum() == 4 * 32
        check(t, want, np.abs(want) * 2.0**-10 + 2.0**-25, "bad groups")


def test_large_cache_offsets(w):
    """A cache of more than 2^32 bytes: the last slots land where they should and are read from there."""
    Hkv, D, page, group = 8, 256, 128, 64
    size = w.kv4_page_bytes(page, D, group)
    pages = (1 << 32) // (Hkv * size) + 5
    kc = torch.zeros((pages, Hkv, size), dtype=torch.uint8, device=DEV)
    vc = torch.zeros_like(kc)
    k, v = randn((2, Hkv, D), "fp16", 1), randn((2, Hkv, D), "fp16", 2)
    slots = torch.tensor([pages * page - 1, 3], device=DEV)
    w.qmm_kv4_append(k, k, v, None, None, None, slots, kc, vc, group)
    near = [torch.zeros((2, Hkv, size), dtype=torch.uint8, device=DEV) for _ in range(2)]
    w.qmm_kv4_append(k, k, v, None, None, None, torch.tensor([2 * page - 1, 3], device=DEV), *near, group)
    for far, n in zip((kc, vc), near):
        assert torch.equal(far[-1], n[1]) and torch.equal(far[0], n[0])
        assert int(torch.count_nonzero(far)) == int(torch.count_nonzero(n))
    a = w.qmm_kv4_gather(kc, vc, slots, D, group)
    b = w.qmm_kv4_gather(*near, torch.tensor([2 * page - 1, 3], device=DEV), D, group)
    assert all(torch.equal(x, y) and x.any() for x, y in zip(a, b))


def test_refusals_on_tensors(w):
    q, k, v, cos, sin, pos, slots, kc, vc = _case(4, 2, 1, 64, 64, 8, 32, "fp16", 3, False)
    dk, dv, sl = device(kc), device(vc), device(slots)
    good = (q, k, v, cos, sin, i32(pos), sl, dk, dv, 32)
    w.qmm_kv4_append(*good)

    def refused(error, call, **change):
        with pytest.raises(error):
            call(*[change.get(i, a) for i, a in zip("q k v cos sin pos slots kc vc group".split(), good)])

    refused(ValueError, w.qmm_kv4_append, group=16)
    refused(ValueError, w.qmm_kv4_append, kc=dk[:, :, :-8].contiguous(), vc=dv[:, :, :-8].contiguous())
    refused(TypeError, w.qmm_kv4_append, kc=dk.view(torch.int8), vc=dv.view(torch.int8))
    refused(ValueError, w.qmm_kv4_append, vc=dv[:1])
    refused(ValueError, w.qmm_kv4_append, kc=dk[:, :, ::2])
    refused(ValueError, w.qmm_kv4_append, k=torch.cat([k, k], 1), v=torch.cat([v, v], 1))
    refused(TypeError, w.qmm_kv4_append, k=k.bfloat16())
    refused(TypeError, w.qmm_kv4_append, slots=sl.int())
    with pytest.raises(TypeError):
        w.qmm_kv4_gather(dk, dv, sl, 64, 32, dtype=torch.float32)
    with pytest.raises(ValueError):
        w.qmm_kv4_gather(dk, dv, sl, 96, 32)
    with pytest.raises(TypeError):
        w.qmm_kv4_gather(dk, dv, sl.int(), 64, 32)
