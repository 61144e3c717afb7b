"""The cap on scores from far below them to far above, in both attention kernels.
A cap far above the scores must leave them as they are: its error goes with the
score, not with the cap. The bound is the oracle's."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, check, f64, i32, paged, randn, say
from oracle import layer_oracle as lo
from test_gpu_attention import run, w  # noqa: F401  (the fixture)
from test_gpu_attention_tiles import KV, PART

pytestmark = pytest.mark.gpu

CAPS = [1e-39, 1e-30, 0.5, 64.0, 64.5, 1e3, 1e5, 1e7, 1e30, 3e38]


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_caps_on_single_tokens(w, dtype, softcap):  # noqa: F811
    run(w, [33, 700, 140], [1, 1, 3], 4, 2, 128, 16, dtype, softcap=softcap)
    run(w, [33, 700, 140], [1, 1, 3], 4, 2, 64, 16, dtype, softcap=softcap, scale=-0.2)


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("D,dtype", [(64, "bf16"), (128, "fp16"), (256, "fp16")])
def test_caps_on_prompts(w, D, dtype, softcap):  # noqa: F811
    run(w, KV, PART, 6, 6, D, 16, dtype, softcap=softcap)


@pytest.mark.parametrize("softcap", [1e3, 1e7])
def test_large_caps_with_a_distance_bias(w, softcap):  # noqa: F811
    slopes = 2.0 ** -np.arange(1, 7)
    run(w, KV, PART, 6, 6, 64, 16, "fp16", q_scale=4.0, softcap=softcap, slopes=slopes)
    run(w, [90, 333], [1, 2], 6, 6, 128, 16, "fp16", q_scale=4.0, softcap=softcap, slopes=slopes)


@pytest.mark.parametrize("softcap", [100.0, 1e4])
def test_scores_around_and_above_a_large_cap(w, softcap):  # noqa: F811
    """Both ways of taking the cap within one row: scores from a hundredth of it to several times it."""
    run(w, [90, 200], [1, 90], 4, 2, 128, 16, "fp16", q_scale=softcap * 1.5)
    run(w, [90, 200], [1, 2], 4, 2, 128, 16, "bf16", q_scale=softcap * 1.5, softcap=softcap)
    run(w, KV, PART, 6, 6, 64, 16, "bf16", q_scale=softcap * 1.5, softcap=softcap)


@pytest.mark.parametrize("T", [3, 130])
def test_a_large_cap_keeps_bad_values_to_their_queries(w, T):  # noqa: F811
    say(f"a bad value under a large cap, T={T}")
    H, D, page = 40 if T > 100 else 2, 64, 16
    k, v, table = paged(1, [T], H, D, page, "bf16", 1)
    q = randn((T, H, D), "bf16", 2)
    at = T - 1
    v[table[0, at // page], 0, at % page, 5] = float("inf")
    args = (i32(table), i32(np.array([T])), i32(np.array([0, T])), T, T)
    got = w.qmm_attention(q, k, v, *args, softcap=1e6)
    v[table[0, at // page], 0, at % page, 5] = 0
    clean = w.qmm_attention(q, k, v, *args, softcap=1e6)
    assert torch.equal(got[:-1], clean[:-1])
    assert not torch.isfinite(got[-1, 0, 5])
    want, bound = lo.attention(f64(q), f64(k), f64(v), table, [T], [0, T], D**-0.5, softcap=1e6, dtype="bf16")
    check(clean, want, bound, "out")
    assert clean.device == torch.device(DEV)
