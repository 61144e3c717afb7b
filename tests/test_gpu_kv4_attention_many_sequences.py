"""qmm_kv4_attention in parts of the keys with more sequences than a wave has lanes, with more tiles than blocks run at a
time, and with more chunks than a tile has parts. Against float64 and at the bounds of the other tests."""
import numpy as np
import pytest

from test_gpu_kv4_attention import run
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


def parts(w, kv_lens, q_lens, Hq, Hkv, D, max_kv, group=64, **kw):  # noqa: F811
    p = w.kv4_attention_plan_info(len(kv_lens), int(sum(q_lens)), Hq, Hkv, D, int(max(q_lens)), max_kv)
    assert p["kernel"] == "parts"
    run(w, [int(n) for n in kv_lens], [int(n) for n in q_lens], Hq, Hkv, D, 16, group, "bf16", max_kv=max_kv, **kw)
    return p


@pytest.mark.parametrize("B,Hq,Hkv,D,max_kv,max_q", [(65, 4, 1, 128, 4200, 1), (130, 4, 2, 64, 4200, 1), (130, 2, 2, 256, 4200, 3),
                                                     (513, 2, 1, 64, 4200, 1), (1000, 2, 2, 64, 8200, 1), (1024, 3, 1, 128, 4200, 2)])
def test_ragged_lengths(w, B, Hq, Hkv, D, max_kv, max_q):  # noqa: F811
    """Some without keys, some without queries, a few far longer than the rest."""
    r = np.random.default_rng(B + D)
    kv = np.exp(r.uniform(0, np.log(150), B)).astype(int)
    kv[r.integers(0, B, 3)] = (max_kv - 7, 3000, 1111)
    q = r.integers(1, max_q + 1, B)
    q[r.random(B) < 0.1] = 0
    kv = np.maximum(kv, q)
    kv[r.random(B) < 0.05] = 0
    p = parts(w, kv, q, Hq, Hkv, D, max_kv)
    if B * Hkv > p["resident"]:
        assert p["blocks"] == B * Hkv + p["parts"]  # no shares make as few blocks as run at a time


@pytest.mark.parametrize("q_lens", [[1], [7]])
def test_more_chunks_than_parts(w, q_lens):  # noqa: F811
    """40000 keys are 313 times the fewest chunks of a part; a tile has 256 parts at most."""
    parts(w, [40000], q_lens, 2, 1, 64, 40000)


def test_even_lengths(w):  # noqa: F811
    parts(w, [300] * 200, [1] * 200, 2, 1, 64, 4200)
    parts(w, [100] * 90, [5] * 90, 4, 1, 128, 4200)
