"""Groups of the 4-bit cache whose scale is finite and so large that they stand for NaN, and of the largest scales that
stand for numbers: read back, and attended to by each of the kernels. Expected values and bounds are the oracle's."""
import numpy as np
import pytest
import torch

from cache_cases import device, filled, paged4
from layer_cases import DEV, check, f64, i32, randn, say
from oracle import cache_oracle as co
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# name: sequences, new tokens of each, query heads, key heads, bound of the keys, head sizes
KERNELS = {
    "a_token": (1, 1, 16, 4, 300, (64, 128, 256)),
    "a_tile": (1, 8, 8, 4, 300, (64, 128, 256)),
    "two_tiles": (5, 40, 256, 128, 300, (64, 128)),
    "parts_of_a_token": (1, 1, 16, 4, 4200, (64, 128, 256)),
    "parts_of_tiles": (1, 30, 8, 4, 4200, (64, 128, 256)),
    "blocks": (1, 100, 336, 168, 300, (64, 128, 256)),
}
CASES = [(name, D) for name, kernel in KERNELS.items() for D in kernel[5]]
GROUPS = {64: 32, 128: 128, 256: 64}
KV, PAGE = 300, 16


def put_scale(cache, page, head, key, D, group, keys, s):
    block = cache[page, head].reshape(PAGE // 8, -1)[key % PAGE // 8]
    for g in range(D // group):
        at = co.scale_places(key % 8, g, D, group, keys)[0]
        if s[g] is not None:
            block[at:at + 2] = np.frombuffer(np.float16(s[g]).tobytes(), np.uint8)


def attend(w, name, D, places, s, first=None, end=None):  # noqa: F811
    """Results before and after the scales of `places` (keys?, key head, key) become s, with the expected ones, for the query
    heads of the first five key heads (the fifth keeps its scales) and the tokens of the last sequence."""
    B, T, Hq, Hkv, max_kv, _ = KERNELS[name]
    group, G = GROUPS[D], Hq // Hkv
    say(f"kv4 large scales {name} D={D} s={s}")
    k, v, table = paged4([KV] * B, Hkv, D, PAGE, group, 1)
    if max_kv > table.shape[1] * PAGE:
        table = np.pad(table, ((0, 0), (0, -(-max_kv // PAGE) - table.shape[1])))
    q = randn((B * T, Hq, D), "bf16", 2)
    dev = lambda a: None if a is None else i32(np.tile(a, B))  # noqa: E731
    rest = (i32(table), i32(np.full(B, KV)), i32(np.arange(B + 1) * T), T, max_kv, group)
    call = lambda: w.qmm_kv4_attention(q, device(k), device(v), *rest, scale=0.02, first=dev(first), end=dev(end))[-T:, :5 * G]  # noqa: E731
    before = call()
    for keys, head, key in places:
        put_scale(k if keys else v, table[B - 1, key // PAGE], head, key, D, group, keys, s)
    got = call()
    part = lambda c, keys: [x[:, :min(5, Hkv)] for x in co.parts(c, D, group, keys)]  # noqa: E731
    want, bound = co.attention(f64(q)[-T:, :5 * G], part(k, True), part(v, False), table[-1:], [KV], [0, T], 0.02, group, first=first,
                               end=end, dtype="bf16")
    check(got, want, bound, "out")
    return before, got, want


@pytest.mark.parametrize("s", [3000.0, -3000.0, 60000.0, 2736.0])
@pytest.mark.parametrize("name,D", CASES)
def test_such_a_group_is_nan_to_the_queries_that_see_it(w, name, D, s):  # noqa: F811
    """Keys that the last query alone sees, and keys that all see; a key and a value of each."""
    T, G = KERNELS[name][1], KERNELS[name][2] // KERNELS[name][3]
    scales = [None] * (D // GROUPS[D] - 1) + [s]  # the last group's
    places = [(True, 0, KV - 1), (False, 1, KV - 1), (True, 2, 40), (False, 3, 41)]
    before, got, want = attend(w, name, D, places, scales)
    assert np.isnan(want[-1, 0]).all() and np.isnan(want[:, 2 * G]).all() and np.isnan(want[:, 3 * G, -1]).all()
    assert np.isfinite(want[:-1, :2 * G]).all() and (D == GROUPS[D] or np.isfinite(want[:, 3 * G, 0]).all())
    assert torch.equal(got[:T - 1, :2 * G], before[:T - 1, :2 * G])


@pytest.mark.parametrize("s", [3000.0, 60000.0, float("nan")])
@pytest.mark.parametrize("name,D", CASES)
def test_keys_that_no_query_sees_have_no_part(w, name, D, s):  # noqa: F811
    """Between the keys that a tile's queries see, and next to the ends of them."""
    T = KERNELS[name][1]
    first, end = np.where(np.arange(T) % 2 == 0, 10, 200), np.where(np.arange(T) % 2 == 0, 100, 290)
    places = [(keys, head, key) for keys, head in ((True, 0), (False, 1), (True, 2), (False, 2)) for key in (9, 100, 150, 199, 290)]
    before, got, want = attend(w, name, D, places, [s] * (D // GROUPS[D]), first, end)
    assert np.isfinite(want).all() and torch.equal(got, before)


@pytest.mark.parametrize("s", [2720.0, -2720.0, 2192.0])
@pytest.mark.parametrize("name,D", CASES)
def test_the_largest_scales_stand_for_numbers(w, name, D, s):  # noqa: F811
    _, got, want = attend(w, name, D, [(True, 0, KV - 1), (False, 1, KV - 1), (True, 2, 40), (False, 3, 41)], [s] * (D // GROUPS[D]))
    assert np.isfinite(want).all()


@pytest.mark.parametrize("D,group", [(64, 32), (128, 128), (256, 64)])
def test_reading_back(w, D, group):  # noqa: F811
    """As the attention takes them."""
    caches = [filled(1, 1, PAGE, D, group, keys, 5) for keys in (True, False)]
    for t, s in enumerate((2720.0, -2720.0, 2728.0, 2730.0, -2736.0, 3000.0, 60000.0)):
        for cache, keys in zip(caches, (True, False)):
            put_scale(cache, 0, 0, t, D, group, keys, [s] + [None] * (D // group - 1))
    got = w.qmm_kv4_gather(*map(device, caches), torch.arange(PAGE, device=DEV), D, group, torch.bfloat16)
    for t, cache, keys in zip(got, caches, (True, False)):
        want = sum(co.parts(cache, D, group, keys))[0, 0][:, None]
        assert np.isnan(want).sum() == 4 * group
        check(t, want, np.abs(want) * (2.0**-8 + 2.0**-24) + 2.0**-133, "read back")
