"""qmm_kv_append against float64: an fp32 rotation errs by at most 3 roundings
(2^-24 each) of |a c| + |b s|, then one rounding to the data type."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, TYPES, check, f64, i32, randn, say
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required")
    import weight_only_group_amd as mod
    mod.library()
    return mod


def _case(T, Hq, Hkv, D, R, page, dtype, seed, fused, P=50):
    r = np.random.default_rng(seed)
    if fused:
        rows = randn((T, (Hq + 2 * Hkv) * D + 8), dtype, seed)
        q, k, v = (t.unflatten(1, (-1, D)) for t in rows[:, :-8].split([Hq * D, Hkv * D, Hkv * D], dim=1))
    else:
        q, k, v = (randn((T, h, D), dtype, seed + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    angle = r.uniform(0, 6.28, (P, R // 2))
    cos, sin = (torch.from_numpy(f(angle).astype(np.float32)).to(DEV) for f in (np.cos, np.sin))
    pages = T // page + 3
    slots = r.permutation(pages * page)[:T].astype(np.int64)
    kc, vc = (randn((pages, Hkv, page, D), dtype, seed + 5 + i) for i in range(2))
    return q, k, v, cos, sin, r.integers(0, P, T).astype(np.int32), slots, kc, vc


CASES = [(1, 1, 1, 64, 64, 1), (1, 8, 2, 128, 128, 16), (7, 32, 8, 128, 64, 16), (13, 5, 1, 256, 256, 24),
         (3, 6, 3, 64, 16, 5), (130, 4, 4, 128, 96, 64), (2, 3, 3, 256, 112, 100), (5, 2, 1, 128, 0, 7)]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("adjacent", [True, False])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,page", CASES)
def test_append(w, T, Hq, Hkv, D, R, page, dtype, adjacent, fused):
    say(f"append T={T} Hq={Hq} Hkv={Hkv} D={D} R={R} page={page} {dtype} adjacent={adjacent} fused={fused}")
    q, k, v, cos, sin, pos, slots, kc, vc = _case(T, Hq, Hkv, D, R, page, dtype, T + D + R, fused)
    if T > 2:
        slots[1] = -1
        slots[2] = kc.shape[0] * page  # one past the cache
    cs, sn = (f64(cos), f64(sin)) if R else (None, None)
    want = lo.kv_append(f64(q), f64(k), f64(v), cs, sn, pos, slots, f64(kc), f64(vc), adjacent)
    out = w.qmm_kv_append(q, k, v, cos if R else None, sin if R else None, i32(pos), torch.from_numpy(slots).to(DEV), kc,
                          vc, adjacent=adjacent)
    u, tiny = lo.ROUNDOFF[dtype], lo.TINY[dtype]
    # What R leaves alone, other slots and all values are copies: equal bits.
    rot = np.arange(D) < R
    check(out, want[0], np.where(rot, u * np.abs(want[0]) + (1 + u) * 3 * lo.F32 * want[3] + tiny, 0), "q")
    moved = want[4] * rot
    check(kc, want[1], np.where(moved > 0, u * np.abs(want[1]) + (1 + u) * 3 * lo.F32 * moved + tiny, 0), "k_cache")
    check(vc, want[2], np.zeros(want[2].shape), "v_cache")


def test_append_positions_are_cut_to_the_table(w):
    q, k, v, cos, sin, pos, slots, kc, vc = _case(4, 2, 1, 64, 64, 8, "fp16", 3, False)
    bad = np.array([-5, 10**9, 2, 49], np.int32)
    sl = torch.from_numpy(slots).to(DEV)
    out = w.qmm_kv_append(q, k, v, cos, sin, i32(bad), sl, kc.clone(), vc.clone())
    same = w.qmm_kv_append(q, k, v, cos, sin, i32(np.clip(bad, 0, 49)), sl, kc.clone(), vc.clone())
    assert torch.equal(out, same)


def test_append_nothing_and_non_finite(w):
    q, k, v, cos, sin, pos, slots, kc, vc = _case(3, 2, 1, 128, 64, 8, "bf16", 4, True)
    sl = torch.from_numpy(slots).to(DEV)
    before = kc.clone()
    assert w.qmm_kv_append(q[:0], k[:0], v[:0], cos, sin, i32(pos[:0]), sl[:0], kc, vc).shape == (0, 2, 128)
    assert torch.equal(kc, before)
    k[1, 0, 100] = float("inf")
    k[1, 0, 101] = float("nan")
    w.qmm_kv_append(q, k, v, cos, sin, i32(pos), sl, kc, vc)
    row = kc[slots[1] // 8, 0, slots[1] % 8]
    assert torch.isinf(row[100]) and torch.isnan(row[101]) and torch.isfinite(row[:100]).all()


def test_append_large_cache_offsets(w):
    """A cache of more than 2^32 bytes: the last slots land where they should."""
    Hkv, D, page = 8, 256, 128
    pages = (1 << 32) // (Hkv * D * page * 2) + 5
    kc = torch.zeros((pages, Hkv, page, D), dtype=torch.float16, device=DEV)
    vc = torch.zeros_like(kc)
    k, v = randn((2, Hkv, D), "fp16", 1), randn((2, Hkv, D), "fp16", 2)
    slots = torch.tensor([pages * page - 1, 3], device=DEV)
    w.qmm_kv_append(k, k, v, None, None, None, slots, kc, vc)
    assert torch.equal(kc[-1, :, -1], k[0]) and torch.equal(vc[-1, :, -1], v[0])
    assert torch.equal(kc[0, :, 3], k[1]) and torch.equal(vc[0, :, 3], v[1])
    assert int(torch.count_nonzero(kc)) == int(torch.count_nonzero(k))
