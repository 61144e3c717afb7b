"""qmm_attention on prompts enough to fill the CUs with blocks of 128 rows: the
same checks as for the split kernel, on shapes that take the other one."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, check, f64, i32, paged, randn, say
from oracle import layer_oracle as lo
from test_gpu_attention import run, w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# 16 sequences: lengths around the steps of 32, 64 and 128, some with a context before the prompt.
KV = [130, 1, 64, 65, 127, 128, 129, 63, 200, 33, 90, 2, 150, 96, 31, 70]
FULL = list(KV)
PART = [130, 1, 10, 65, 100, 3, 129, 60, 73, 33, 90, 1, 68, 40, 31, 70]
SHAPES = [(6, 6, 64, 16), (8, 4, 128, 24), (6, 6, 128, 64), (3, 3, 256, 7), (10, 2, 64, 1), (12, 3, 256, 128)]


@pytest.mark.parametrize("q_lens", [FULL, PART], ids=["full", "part"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("Hq,Hkv,D,page", SHAPES)
def test_prompts(w, Hq, Hkv, D, page, dtype, q_lens):  # noqa: F811
    run(w, KV, q_lens, Hq, Hkv, D, page, dtype)


@pytest.mark.parametrize("softcap,slopes", [(20.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cap_and_distance(w, D, softcap, slopes):  # noqa: F811
    kw = {"softcap": softcap}
    if slopes:
        kw["slopes"] = 2.0 ** -np.arange(1, 7)
    run(w, KV, PART, 6, 6, D, 16, "bf16" if D == 64 else "fp16", q_scale=4.0, **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["window", "documents", "prefix", "any"])
def test_masks(w, kind, D):  # noqa: F811
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(KV, PART)])
    first, end = np.zeros_like(pos), pos + 1
    r = np.random.default_rng(5)
    if kind == "window":
        first = pos + 1 - 20
    elif kind == "documents":
        first = pos // 37 * 37
    elif kind == "prefix":
        end = np.maximum(end, 50)
    else:
        first, end = r.integers(-50, 220, len(pos)), r.integers(-50, 220, len(pos))
    out = run(w, KV, PART, 6, 6, D, 24, "fp16", first=first, end=end)
    kv = np.repeat(KV, PART)
    assert not f64(out)[np.maximum(first, 0) >= np.minimum(end, kv)].any()


@pytest.mark.parametrize("kv,q_lens", [(KV, PART), ([200, 33], [3, 1])], ids=["tiles", "split"])
def test_ranges_at_the_ends_of_32_bits(w, kv, q_lens):  # noqa: F811
    T = sum(q_lens)
    r = np.random.default_rng(6)
    first = r.choice([-2**31, -1, 0, 5, 40, 2**31 - 1], T)
    end = r.choice([-2**31, -2**31 + 1, -7, 0, 60, 2**31 - 1], T)
    run(w, kv, q_lens, 6, 6, 64, 16, "fp16", first=first, end=end)


def test_all_rows_empty(w):  # noqa: F811
    T = sum(PART)
    out = run(w, KV, PART, 6, 6, 128, 16, "fp16", first=np.full(T, 30), end=np.full(T, 30))
    assert not out.any()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), 60000.0])
def test_places_past_the_end_have_no_part(w, fill, D):  # noqa: F811
    run(w, KV, PART, 6, 6, D, 32, "fp16", fill=fill)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_value_reaches_only_queries_that_see_it(w, bad, D):  # noqa: F811
    say(f"a bad value in tiles D={D} {bad}")
    kv, page, H = 200, 16, 96
    k, v, table = paged(1, [kv], H, D, page, "bf16", 1)
    q = randn((kv, H, D), "bf16", 2)
    args = (i32(table), i32(np.array([kv])), i32(np.array([0, kv])), kv, kv)
    clean = w.qmm_attention(q, k, v, *args)
    k[table[0, 147 // page], 0, 147 % page, 3] = bad
    v[table[0, 146 // page], 1, 146 % page, 37] = bad
    got = w.qmm_attention(q, k, v, *args)
    assert torch.equal(got[:146], clean[:146])
    assert torch.equal(got[:, 2:], clean[:, 2:])
    assert torch.equal(got[:147, 0], clean[:147, 0])
    seen = got[146:, 1]
    assert not torch.isfinite(seen[:, 37]).any()
    rest = [d for d in range(D) if d != 37]
    near, want = f64(seen[:, rest]), f64(clean[146:, 1][:, rest])
    assert np.isfinite(near).all() and np.abs(near - want).max() < 2.0**-6


def test_huge_scores(w):  # noqa: F811
    run(w, KV, PART, 6, 6, 128, 16, "fp16", q_scale=300.0)
    run(w, KV, PART, 6, 6, 64, 16, "bf16", q_scale=3000.0)


def test_views_and_lengths_below_the_bounds(w):  # noqa: F811
    run(w, KV, PART, 6, 6, 128, 16, "fp16", view=True, max_kv=208)


def test_sequences_without_keys_or_queries(w):  # noqa: F811
    D, page, H = 128, 16, 40
    say("tiles with empty sequences")
    k, v, table = paged(4, [90, 1, 40, 70], H, D, page, "fp16", 1)
    kv = np.array([90, 0, 40, 70])
    starts = np.array([0, 80, 90, 90, 130])
    q = randn((130, H, D), "fp16", 2)
    out = w.qmm_attention(q, k, v, i32(table), i32(kv), i32(starts), 80, 90)
    want, bound = lo.attention(f64(q), f64(k), f64(v), table, kv, starts, D**-0.5)
    check(out, want, bound, "out")
    assert not out[80:90].any()


def test_equal_bits_and_a_long_prompt(w):  # noqa: F811
    """A prompt of some thousand tokens against the same rows asked for one by one (the split kernel)."""
    n, H, Hkv, D, page = 3001, 8, 2, 128, 48
    say("a long prompt")
    k, v, table = paged(1, [n], Hkv, D, page, "bf16", 1)
    q = randn((n, H, D), "bf16", 2)
    args = (k, v, i32(table), i32(np.array([n])), i32(np.array([0, n])), n, n)
    out = w.qmm_attention(q, *args, softcap=30.0)
    assert torch.equal(out, w.qmm_attention(q, *args, softcap=30.0))
    at = [0, 1, 127, 128, 1500, 2999, 3000]
    one = w.qmm_attention(q[at].contiguous(), k, v, i32(np.repeat(table, len(at), axis=0)), i32(np.array(at) + 1),
                          i32(np.arange(len(at) + 1)), 1, n, softcap=30.0)
    a, b = f64(out[at]), f64(one)
    # Each is within three roundings of sum p |v| of the formula; |v| is below 6 here.
    assert np.abs(a - b).max() < 6 * 6 * 2.0**-8
    assert np.linalg.norm(a - b) < 2 * 2.0**-8 * np.linalg.norm(b)


def test_large_cache_offsets(w):  # noqa: F811
    Hkv, D, page = 8, 256, 128
    pages = (1 << 32) // (Hkv * D * page * 2) + 5
    k = torch.zeros((pages, Hkv, page, D), dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    for c, s in ((k, 1), (v, 2)):
        c[-2:] = randn((2, Hkv, page, D), "fp16", s)
    B, n = 11, 90
    q = randn((B * n, 8, D), "fp16", 3)
    rest = (i32(np.full(B, 200)), i32(np.arange(B + 1) * n), n, 200)
    out = w.qmm_attention(q, k, v, i32(np.repeat([[pages - 1, pages - 2]], B, axis=0)), *rest)
    near = w.qmm_attention(q, k[-2:].contiguous(), v[-2:].contiguous(), i32(np.repeat([[1, 0]], B, axis=0)), *rest)
    assert torch.equal(out, near) and out.any()
