"""Keys at the end of the range that the call takes, just below 2^31: a small cache
whose one page stands for the whole sequence, and queries that see its last keys."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, check, f64, i32, randn, say
from oracle import layer_oracle as lo
from test_gpu_attention import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
PAGE, ENTRIES = 49981, 42966
KV = PAGE * ENTRIES  # 2^31 - 2


@pytest.mark.parametrize("bad", [None, float("inf")])
@pytest.mark.parametrize("q_lens,Hkv", [([1], 1), ([3, 1], 2), ([130], 43)], ids=["one", "few", "prompt"])
def test_keys_up_to_the_end_of_31_bits(w, q_lens, Hkv, bad):  # noqa: F811
    say(f"attention far keys q={q_lens} Hkv={Hkv} bad={bad}")
    B, T, D = len(q_lens), sum(q_lens), 64
    k, v = (randn((1, Hkv, PAGE, D), "fp16", s) for s in (1, 2))
    q = randn((T, Hkv, D), "fp16", 3)
    kv_lens = [KV, KV - 40][:B]
    table = np.zeros((B, ENTRIES), np.int32)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])
    first = pos - 150
    end = np.minimum(pos + 1, KV - 1)
    if bad is not None:  # the last key of all, which no query sees
        v[0, :, (KV - 1) % PAGE] = bad
    slopes = 2.0 ** -np.arange(5, 5 + Hkv)
    out = w.qmm_attention(q, k, v, i32(table), i32(np.array(kv_lens)), i32(starts), max(q_lens), KV, first=i32(first),
                          end=i32(end), slopes=torch.from_numpy(slopes).float().to(DEV))
    want, bound = lo.attention(f64(q), f64(k), f64(v), table, kv_lens, starts, D**-0.5,
                               slopes=slopes.astype(np.float32), first=first, end=end)
    check(out, want, bound, "out")
