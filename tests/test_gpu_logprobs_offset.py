"""Log probabilities of logits far from zero: they depend on differences alone, so
an offset that all logits of a row share must not cost accuracy. The bound is that
of logits around zero: 2^-19 for the sum and two roundings of the result."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, TYPES, check, f64, gen, say
from oracle import layer_oracle as lo
from test_gpu_logprobs import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("offset", [0.0, 300.0, -1e4, 1e4, 2.0**20])
@pytest.mark.parametrize("M,V,top", [(1, 32000, 5), (3, 1000, 20), (600, 257, 2), (2, 7, 7)])
def test_an_offset_costs_nothing(w, M, V, top, offset):  # noqa: F811
    say(f"logprobs M={M} V={V} top={top} offset={offset}")
    logits = (3 * torch.randn((M, V), generator=gen(V)) + offset).to(DEV)
    targets = torch.randint(0, V, (M,), generator=gen(V + 1)).to(DEV)
    got = w.qmm_logprobs(logits, targets, top=top)
    want = lo.logprobs(f64(logits), targets.cpu().numpy(), top)
    assert np.array_equal(got[3].cpu().numpy(), want[3])
    for at, name in ((0, "logprob"), (2, "top_logprobs")):
        check(got[at], want[at], 2.0**-19 + 2 * lo.F32 * np.abs(want[at]), name)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_a_certain_token(w, dtype):  # noqa: F811
    """One logit above all others by far more or less than a rounding of its size."""
    V = 5000
    logits = torch.zeros((3, V)).to(TYPES[dtype])
    logits[0] = 8192
    logits[0, 17] = 8192 + 64
    logits[1] = -8192
    logits[1, 4999] = -8192 + 128
    logits[2] = 1000
    logits[2, 3] = 1016
    logits = logits.to(DEV)
    targets = torch.tensor([17, 4999, 0], device=DEV)
    got = w.qmm_logprobs(logits, targets, top=2)
    want = lo.logprobs(f64(logits), targets.cpu().numpy(), 2)
    assert np.array_equal(got[3].cpu().numpy(), want[3])
    assert (got[0] <= 0).all() and (got[2] <= 0).all()
    check(got[0], want[0], 2.0**-19 + 2 * lo.F32 * np.abs(want[0]), "logprob")
    check(got[2], want[2], 2.0**-19 + 2 * lo.F32 * np.abs(want[2]), "top_logprobs")
