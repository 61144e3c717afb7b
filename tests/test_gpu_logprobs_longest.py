"""The longest rows that the call takes, with the type's lowest value as a mask."""
import math

import pytest
import torch

from layer_cases import DEV, say
from test_gpu_logprobs import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [0, 2])
@pytest.mark.parametrize("runs", [1 << 24, 2049 << 13, 3])
def test_a_row_of_two_to_the_thirty(w, runs, top):  # noqa: F811
    """Runs of masked and of equal logits in turn: half the tokens share all the probability."""
    V = 1 << 30
    say(f"logprobs V={V} runs of {runs} top={top}")
    lowest = torch.finfo(torch.bfloat16).min
    logits = torch.full((1, V), lowest, dtype=torch.bfloat16, device=DEV)
    if runs == 3:  # one token in three
        logits[0, 1::3] = 2.0
        first, live = 1, (V + 1) // 3
    else:
        # (2049 << 13: what one of 64 blocks takes, so that whole blocks are masked)
        starts = range(runs, V, 2 * runs)
        for at in starts:
            logits[0, at:at + runs] = 2.0
        first, live = runs, sum(min(runs, V - at) for at in starts)
    targets = torch.tensor([first], device=DEV)
    logprob, entropy, top_logprobs, ids = w.qmm_logprobs(logits, targets, top=top)
    # fp32 sums of equal terms of one sign, up to 2^30 / 2^14 of them in a thread: 2^16 roundings of 2^-24 at most
    assert abs(logprob.item() + math.log(live)) < 2.0**-8
    assert abs(entropy.item() - math.log(live)) < 2.0**-8
    if top:
        step = 3 if runs == 3 else 1
        assert ids[0].tolist() == [first, first + step]
        assert (top_logprobs + math.log(live)).abs().max() < 2.0**-8
