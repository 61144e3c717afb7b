"""qmm_logprobs against float64. Ids have to be equal. The sums are fp32 over V
terms of one sign: with the exponentials good to 2^-20 (arguments of up to 30
carry their rounding into the result), lse errs by at most 2^-19 plus a few
roundings of its size; the entropy by that and the same of the mean of |l - m|."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, TYPES, check, f64, gen, say
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required")
    import weight_only_group_amd as mod
    mod.library()
    return mod


def compare(w, logits, targets, top):
    got = w.qmm_logprobs(logits, targets, top=top)
    l = f64(logits)
    want = lo.logprobs(l, None if targets is None else targets.cpu().numpy(), top)
    assert np.array_equal(got[3].cpu().numpy(), want[3]), "ids differ"
    finite = np.where(np.isfinite(l), l, 0)
    size = np.abs(finite).max(axis=1)
    slack = 2.0**-19 + 8 * lo.F32 * size
    if targets is not None:
        check(got[0], want[0], slack + 2 * lo.F32 * np.where(np.isfinite(want[0]), np.abs(want[0]), 0), "logprob")
    else:
        assert got[0] is None
    with np.errstate(all="ignore"):
        p = np.exp(l - l.max(axis=1, keepdims=True))
        spread = np.nan_to_num((p * np.abs(np.where(p > 0, finite - finite.max(axis=1, keepdims=True), 0))).sum(axis=1) / p.sum(axis=1))
    check(got[1], want[1], slack + 2.0**-18 * (1 + spread), "entropy")
    check(got[2], want[2], slack[:, None] + 2 * lo.F32 * np.where(np.isfinite(want[2]), np.abs(want[2]), 0), "top_logprobs")
    return got


CASES = [(1, 1, 1), (2, 2, 2), (3, 7, 7), (1, 33, 32), (5, 64, 5), (4, 255, 20), (3, 1000, 1), (2, 4097, 20), (1, 32000, 5),
         (17, 511, 3), (2, 50257, 32), (3, 9000, 0), (1, 200003, 20)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("M,V,top", CASES)
def test_logprobs(w, M, V, top, dtype):
    say(f"logprobs M={M} V={V} top={top} {dtype}")
    logits = (3 * torch.randn((M, V), generator=gen(M + V))).to(TYPES[dtype]).to(DEV)
    targets = torch.randint(0, V, (M,), generator=gen(V)).to(DEV)
    compare(w, logits, targets, top)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("pad", [1, 3, 8, 63])
def test_strided_rows(w, dtype, pad):
    M, V = 6, 1003
    rows = torch.full((M, V + pad), 1e4).to(TYPES[dtype]).to(DEV)  # what lies between the rows is larger than all
    for start in {0, pad // 2, pad}:
        view = rows[:, start:start + V]
        rows.fill_(1e4)
        view.copy_(torch.randn((M, V), generator=gen(pad)))
        compare(w, view, torch.arange(M, device=DEV) * 100, 9)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_ties_go_to_the_lower_index(w, dtype):
    for V in (40, 5000, 70000):
        logits = torch.zeros((4, V), dtype=TYPES[dtype], device=DEV)  # row 0: all equal
        logits[1] = torch.arange(V, device=DEV) % 7
        logits[2] = -0.0
        logits[2, 1::2] = 0.0
        logits[3] = torch.arange(V - 1, -1, -1, device=DEV) // 3
        compare(w, logits, torch.full((4,), V - 1, device=DEV), 32)


@pytest.mark.parametrize("order", ["rising", "falling", "organ"])
def test_sorted_rows(w, order):
    V = 60000
    l = torch.linspace(-20, 20, V)
    l = {"rising": l, "falling": l.flip(0), "organ": torch.cat([l[::2], l.flip(0)[::2]])}[order]
    compare(w, l[None].repeat(2, 1).to(DEV).contiguous(), torch.tensor([0, V - 1], device=DEV), 32)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_non_finite_logits(w, dtype):
    V = 3001
    logits = torch.randn((8, V), generator=gen(1)).to(TYPES[dtype])
    inf, nan = float("inf"), float("nan")
    logits[0, torch.arange(V) % 3 > 0] = -inf
    logits[1] = -inf
    logits[2] = -inf
    logits[2, 2999] = 1.0
    logits[3, 17] = inf
    logits[4, 2000] = nan
    logits[5, 2000:2003] = -nan
    logits[6] = torch.finfo(TYPES[dtype]).min
    logits[7, 5] = torch.finfo(TYPES[dtype]).max / 2
    targets = torch.tensor([0, 1, 2999, 17, 5, 6, 7, 8], device=DEV)
    got = compare(w, logits.to(DEV), targets, 20)
    assert got[1][2].item() == 0 and got[0][2].item() == 0
    assert abs(got[1][6].item() - np.log(V)) < 1e-4


def test_targets_outside(w):
    logits = torch.randn((5, 100), generator=gen(1)).to(DEV)
    targets = torch.tensor([-1, -100, 100, 1 << 40, 99], device=DEV)
    got = compare(w, logits, targets, 2)
    assert got[0][:2].tolist() == [0.0, 0.0] and torch.isnan(got[0][2:4]).all()
    compare(w, logits, None, 3)


def test_many_rows_and_none(w):
    logits = torch.randn((3000, 130), generator=gen(2)).half().to(DEV)
    compare(w, logits, torch.zeros(3000, dtype=torch.int64, device=DEV), 4)
    got = w.qmm_logprobs(logits[:0], torch.zeros(0, dtype=torch.int64, device=DEV), top=3)
    assert [tuple(t.shape) for t in got] == [(0,), (0,), (0, 3), (0, 3)]


def test_offsets_past_32_bits(w):
    """Rows that lie more than 2^32 bytes apart."""
    rows = torch.zeros((3, (1 << 31) + 7), dtype=torch.float16, device=DEV)
    logits = rows[:, :5000]
    logits.copy_(torch.randn((3, 5000), generator=gen(3)))
    compare(w, logits, torch.tensor([1, 2, 3], device=DEV), 5)


def test_equal_bits_and_graph(w):
    logits = torch.randn((2, 150000), generator=gen(4)).to(torch.bfloat16).to(DEV)
    targets = torch.tensor([5, 77], device=DEV)
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)
    first = w.qmm_logprobs(logits, targets, top=20, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w.qmm_logprobs(logits, targets, top=20, workspace=ws)
    for i in range(4):
        if i:
            logits.copy_(torch.randn(logits.shape, generator=gen(4 + i)))
            first = w.qmm_logprobs(logits, targets, top=20, workspace=ws)
            torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(first, out):
            assert torch.equal(a, b), i
