"""The experts' layer at sizes as they are used, by the norm of its error: the
oracle's limit is little more than the rounding of the result itself, so that a
sum in fewer bits, a bias of the products or a lost part of the intermediate shows."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, expert_planes, f64, gen, randn, say
from oracle import layer_oracle as lo
from test_gpu_moe import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

SIZES = [  # T, H, I, E, k, gs
    (5, 4096, 1056, 4, 2, 32), (5, 4096, 1056, 4, 2, -1), (56, 864, 2528, 5, 1, -1), (2, 2048, 1024, 8, 8, 128),
    (33, 1024, 512, 3, 2, 64),
]


@pytest.mark.parametrize("bits", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H,I,E,k,gs", SIZES)
def test_moe_error_norm(w, T, H, I, E, k, gs, dtype, bits):  # noqa: F811
    strips = (T + bits) % 2 == 0
    x = randn((T, H), dtype, 3 * T + H)
    gu, gu_np = expert_planes(E, H, 2 * I, bits, gs, dtype, strips, seed=21 + bits)
    dn, dn_np = expert_planes(E, I, H, bits, gs, dtype, strips, seed=22 + bits)
    g = gen(T + k)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32)
    weights = torch.rand((T, k), generator=g)
    y = f64(w.qmm_moe(x, ids.to(DEV), weights.to(DEV), gu, dn, bits, gs, strips=strips))
    want, limit = lo.moe_norm(f64(x), ids.numpy(), f64(weights), gu_np, dn_np, bits, gs, dtype)
    error = np.linalg.norm(y - want) / np.linalg.norm(want)
    own = np.linalg.norm(lo.rounded(want, dtype) - want) / np.linalg.norm(want)
    say(f"moe T={T} H={H} I={I} E={E} k={k} bits={bits} gs={gs} {dtype}: error {error:.3e}, rounding {own:.3e}, limit {limit:.3e}")
    assert error <= limit
