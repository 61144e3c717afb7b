"""More rows of logits than one launch has threads for."""
import pytest
import torch

from layer_cases import DEV, say
from test_gpu_logprobs import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_targets", [True, False])
@pytest.mark.parametrize("M", [(1 << 22) + 1, (1 << 24) + 5])
def test_many_rows(w, M, with_targets):  # noqa: F811
    say(f"logprobs M={M} V=2 targets={with_targets}")
    g = torch.Generator(device=DEV).manual_seed(1)
    logits = (3 * torch.randn((M, 3), generator=g, device=DEV)).half()[:, :2]
    targets = torch.randint(0, 2, (M,), generator=g, device=DEV) if with_targets else None
    logprob, entropy, top, ids = w.qmm_logprobs(logits, targets, top=1)
    want = torch.log_softmax(logits.double(), dim=1)
    # 2^-19 for the sum (as for every row of logits), the results are below 40 in size
    near = lambda a, b: float((a.double() - b).abs().max()) < 2.0**-19 + 40 * 2.0**-23  # noqa: E731
    assert near(entropy, -(want.exp() * want).sum(dim=1))
    assert torch.equal(ids[:, 0], (logits[:, 1] > logits[:, 0]).to(torch.int32))
    assert near(top[:, 0], want.amax(dim=1))
    if with_targets:
        assert near(logprob, want.gather(1, targets[:, None])[:, 0])
