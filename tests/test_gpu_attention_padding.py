"""Tokens that belong to no sequence, or to none within the call's bounds, get 0:
a batch padded to a fixed number of tokens reads nothing stale."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, i32, paged, randn, say
from test_gpu_attention import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def padded(w, starts, kv_lens, max_q, T, H, Hkv, D, dtype="bf16"):  # noqa: F811
    """The call on T tokens into a result full of ones, against the same sequences without the padding."""
    say(f"attention padding: starts={starts} kv={kv_lens} max_q={max_q} T={T} H={H}/{Hkv} D={D}")
    k, v, table = paged(len(kv_lens), kv_lens, Hkv, D, 16, dtype, 1)
    q = randn((T, H, D), dtype, 2)
    rest = (k, v, i32(table), i32(np.array(kv_lens)))
    out = torch.ones_like(q)
    w.qmm_attention(q, *rest, i32(np.array(starts)), max_q, max(kv_lens), out=out)
    of_none = np.ones(T, bool)
    for a, b in zip(starts, starts[1:]):
        of_none[a:min(b, a + max_q)] = False
    none = torch.from_numpy(of_none).to(DEV)
    assert not out[none].any()
    first, last = starts[0], starts[-1]
    alone = w.qmm_attention(q[first:last].contiguous(), *rest, i32(np.array(starts) - first), max_q, max(kv_lens))
    assert torch.equal(out[~none], alone[~none[first:last]])
    assert out[~none].any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_tokens_padded(w, D):  # noqa: F811
    padded(w, [0, 1, 2, 3], [700, 5, 33], 1, 16, 8, 2, D)
    padded(w, [2, 3, 4, 5], [70, 5, 33], 1, 6, 4, 4, D)
    padded(w, [0, 5, 6, 9], [70, 5, 33], 2, 11, 4, 1, D)
    padded(w, [3, 3, 4], [70, 5], 1, 4, 4, 4, D)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_prompts_padded(w, D):  # noqa: F811
    padded(w, [7, 137, 137, 237, 300], [130, 4, 150, 90], 130, 400, 24, 24, D)
    padded(w, [0, 130, 230, 300], [130, 150, 90], 80, 301, 60, 30, D)


def test_no_sequences_at_all(w):  # noqa: F811
    q = randn((5, 4, 64), "fp16", 1)
    k = torch.zeros((2, 2, 16, 64), dtype=torch.float16, device=DEV)
    out = torch.ones_like(q)
    w.qmm_attention(q, k, k, i32(np.zeros((0, 4))), i32(np.zeros(0)), i32(np.zeros(1)), 1, 16, out=out)
    assert not out.any()
    out.fill_(1)
    w.qmm_attention(q, k, k, i32(np.zeros((1, 4))), i32(np.ones(1)), i32(np.array([0, 5])), 0, 16, out=out)
    assert not out.any()
