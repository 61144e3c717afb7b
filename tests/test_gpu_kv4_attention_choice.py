"""Which kernel of qmm_kv4_attention takes a call: sizes decide, not whether a mask is given."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import i32, randn, say
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,n,B", [(24, 24, 500, 4), (24, 24, 1500, 1), (32, 8, 300, 4), (4, 4, 60, 2), (64, 16, 1, 3)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_mask_of_the_default_gives_the_same_bits(w, D, Hq, Hkv, n, B):  # noqa: F811
    say(f"kv4 attention with the default mask given, D={D} Hq={Hq} Hkv={Hkv} n={n} B={B}")
    k, v, table = paged4([n] * B, Hkv, D, 16, 64, 1)
    q = randn((B * n, Hq, D), "bf16", 2)
    args = (q, device(k), device(v), i32(table), i32(np.full(B, n)), i32(np.arange(B + 1) * n), n, n, 64)
    pos = np.tile(np.arange(n), B)
    out = w.qmm_kv4_attention(*args)
    for masks in ({"end": pos + 1}, {"first": 0 * pos}, {"first": 0 * pos - 5, "end": pos + 1}):
        assert torch.equal(out, w.qmm_kv4_attention(*args, **{name: i32(a) for name, a in masks.items()})), masks.keys()
