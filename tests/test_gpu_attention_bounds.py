"""Sequences with more queries or keys than the call's bounds: the rows and keys
within them are what they are without the cut."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, check, f64, i32, paged, randn, say
from oracle import layer_oracle as lo
from test_gpu_attention import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def cut(w, kv_lens, q_lens, max_q, max_kv, H, D, slopes, first=None, dtype="fp16"):  # noqa: F811
    B, T, page = len(kv_lens), sum(q_lens), 16
    say(f"attention cut: kv={kv_lens} q={q_lens} max_q={max_q} max_kv={max_kv} H={H} D={D} slopes={slopes}")
    k, v, table = paged(B, kv_lens, H, D, page, dtype, 1)
    q = randn((T, H, D), dtype, 2)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    slope = 2.0 ** -np.arange(2, 2 + H) if slopes else None
    out = w.qmm_attention(q, k, v, i32(table), i32(np.array(kv_lens)), i32(starts), max_q, max_kv,
                          slopes=None if slope is None else torch.from_numpy(slope).float().to(DEV),
                          first=None if first is None else i32(first))
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])
    want, bound = lo.attention(f64(q), f64(k), f64(v), table, kv_lens, starts, D**-0.5,
                               slopes=None if slope is None else slope.astype(np.float32), first=first,
                               end=np.minimum(pos + 1, max_kv), dtype=dtype)
    kept = np.concatenate([np.arange(m) < max_q for m in q_lens])
    check(out[torch.from_numpy(kept).to(DEV)], want[kept], bound[kept], "out")
    return out, kept


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_more_than_the_bounds_few_rows(w, D, slopes):  # noqa: F811
    cut(w, [100, 40], [5, 1], 2, 100, 4, D, slopes)
    cut(w, [100, 40, 700], [5, 1, 3], 3, 64, 4, D, slopes)
    cut(w, [700], [1], 1, 650, 4, D, slopes)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("D", [64, 256])
def test_more_than_the_bounds_prompts(w, D, slopes):  # noqa: F811
    kv, q = [130, 200, 90, 150, 96, 128], [130, 73, 90, 68, 40, 120]
    cut(w, kv, q, 70, 200, 15, D, slopes)
    cut(w, kv, q, 130, 100, 15, D, slopes)
    cut(w, kv, q, 100, 120, 15, D, slopes, first=np.concatenate([np.arange(n - m, n) for n, m in zip(kv, q)]) - 20)
