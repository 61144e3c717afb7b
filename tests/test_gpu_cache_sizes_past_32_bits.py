"""Sizes past 32 bits given to the calls on tensors: refused, not cut to their low bits."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import DEV, i32, randn
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [2**31, 2**32 + 1, 2**32 + 40, -2**32 + 40])
def test_bounds_of_the_attention(w, n):  # noqa: F811
    k, v, table = paged4([40], 1, 64, 16, 32, 1)
    q = randn((1, 2, 64), "fp16", 2)
    k16 = torch.zeros((len(k), 1, 16, 64), dtype=torch.float16, device=DEV)
    rest = (i32(table), i32(np.array([40])), i32(np.array([0, 1])))
    for bounds in ((n, 40), (1, n)):
        with pytest.raises(ValueError, match="2\\^31"):
            w.qmm_kv4_attention(q, device(k), device(v), *rest, *bounds, 32)
        with pytest.raises(ValueError, match="2\\^31"):
            w.qmm_attention(q, k16, k16, *rest, *bounds)


def test_groups_and_pages(w):  # noqa: F811
    k, v, table = paged4([40], 1, 64, 16, 32, 1)
    dk, dv, q = device(k), device(v), randn((1, 1, 64), "fp16", 2)
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    group = 2**32 + 32
    for call in (lambda: w.qmm_kv4_gather(dk, dv, slots, 64, group), lambda: w.qmm_kv4_gather(dk, dv, slots, 2**32 + 64, 32),
                 lambda: w.qmm_kv4_append(q, q, q, None, None, None, slots, dk, dv, group),
                 lambda: w.qmm_kv4_attention(q, dk, dv, i32(table), i32(np.array([40])), i32(np.array([0, 1])), 1, 40, group),
                 lambda: w.qmm_kv_compact([dk, dv], i32(table), i32(np.array([40])), 2**32 + 16)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()
