"""Keys of a 4-bit cache at the end of the range that the call takes, just below 2^31: a small cache whose one page stands
for the whole sequence, and queries that see its last keys."""
import numpy as np
import pytest
import torch

from cache_cases import device, filled
from layer_cases import DEV, check, f64, i32, randn, say
from oracle import cache_oracle as co
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)


pytestmark = pytest.mark.gpu
PAGE, ENTRIES = 43688, 49155
KV = PAGE * ENTRIES  # 2^31 - 8


@pytest.mark.parametrize("bad", [None, float("inf")])
@pytest.mark.parametrize("q_lens,Hq,Hkv", [([1], 1, 1), ([3, 1], 8, 2), ([130], 256, 32)], ids=["one", "few", "prompt"])
def test_keys_up_to_the_end_of_31_bits(w, q_lens, Hq, Hkv, bad):  # noqa: F811
    say(f"kv4 attention far keys q={q_lens} Hkv={Hkv} bad={bad}")
    B, T, D, group = len(q_lens), sum(q_lens), 64, 64
    k, v = (filled(1, Hkv, PAGE, D, group, keys, 1 + keys) for keys in (True, False))
    q = randn((T, Hq, D), "fp16", 3)
    kv_lens = [KV, KV - 40][:B]
    table = np.zeros((B, ENTRIES), np.int32)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])
    first = pos - 150
    end = np.minimum(pos + 1, KV - 1)
    if bad is not None:  # the last key of all, which no query sees
        at = co.scale_places(7, 0, D, group, False)[0]
        v[0].reshape(Hkv, PAGE // 8, -1)[:, -1, at:at + 2] = np.frombuffer(np.float16(bad).tobytes(), np.uint8)
    slopes = 2.0 ** -np.linspace(5, 12, Hq)
    in_blocks = w.library().qmm_kv4_attention_workspace_bytes(B, T, Hq, Hkv, D, max(q_lens), KV) == 0
    assert in_blocks == (T == 130)
    out = w.qmm_kv4_attention(q, device(k), device(v), i32(table), i32(np.array(kv_lens)), i32(starts), max(q_lens), KV, group,
                              first=i32(first), end=i32(end), slopes=torch.from_numpy(slopes).float().to(DEV))
    # The oracle on a page of the last keys alone: positions count from its start.
    near = PAGE - 400
    part = [np.ascontiguousarray(c.reshape(1, Hkv, PAGE // 8, -1)[:, :, near // 8:]).reshape(1, Hkv, -1) for c in (k, v)]
    off = KV - 400
    want, bound = co.attention(f64(q), co.parts(part[0], D, group, True), co.parts(part[1], D, group, False), np.zeros((B, 1), np.int32),
                               [n - off for n in kv_lens], starts, D**-0.5, group, slopes=slopes.astype(np.float32), first=first - off,
                               end=end - off)
    check(out, want, bound, "out")
