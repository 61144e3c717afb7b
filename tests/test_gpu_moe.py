"""The mixture-of-experts layer (qmm_moe_route, qmm_moe) against float64.

Bounds are those of the oracle: fp32 sums, the intermediate kept to 16 bits,
one rounding of the result. Logits and weights: an fp32 sum of H exact products
errs by at most H 2^-24 of the sum of their sizes; a weight by twice the
logits' error plus a few roundings.
"""
import numpy as np
import pytest
import torch

from layer_cases import DEV, check, expert_planes, f64, gen, randn, say
from oracle import layer_oracle as lo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    if not torch.cuda.is_available():
        pytest.fail("a GPU is required")
    import weight_only_group_amd as mod
    mod.library()
    return mod


ROUTE = [(1, 32, 1, 1), (1, 2048, 64, 8), (3, 96, 5, 5), (16, 256, 17, 4), (17, 512, 128, 16), (64, 1056, 130, 2),
         (33, 4096, 256, 8), (64, 64, 1024, 16), (2, 128, 1000, 1)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H,E,k", ROUTE)
def test_route(w, T, H, E, k, dtype, renorm):
    say(f"route T={T} H={H} E={E} k={k} {dtype} renorm={renorm}")
    x, r = randn((T, H), dtype, T + H), randn((E, H), dtype, E, 1 / np.sqrt(H))
    ids, weights, logits = w.qmm_moe_route(x, r, k, renormalize=renorm)
    _, _, want = lo.moe_route(f64(x), f64(r), k, renorm)
    bound = (H + 4) * lo.F32 * (np.abs(f64(x)) @ np.abs(f64(r)).T)
    check(logits, want, bound, "logits")
    # The choice and the weights, from the call's own logits: exact, ties to the lower expert.
    got = f64(logits)
    want_ids, want_w, _ = _of_logits(got, k, renorm)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    check(weights, want_w, 1e-6 * want_w + 1e-12, "weights")


def _of_logits(logits, k, renorm):
    ids = np.array([lo.largest(row, k) for row in logits], np.int32).reshape(len(logits), k)
    e = np.exp(logits - logits.max(axis=1, keepdims=True))
    chosen = np.take_along_axis(e, ids, axis=1)
    return ids, chosen / (chosen if renorm else e).sum(axis=1, keepdims=True), logits


def test_route_ties_go_to_the_lower_expert(w):
    x = torch.ones((5, 64), dtype=torch.float16, device=DEV)
    r = torch.zeros((40, 64), dtype=torch.float16, device=DEV)
    r[[7, 9, 33]] = 1.0
    r[20] = -0.0
    ids, weights, _ = w.qmm_moe_route(x, r, 6)
    assert ids.cpu().tolist() == [[7, 9, 33, 0, 1, 2]] * 5
    assert torch.equal(weights[:, 0], weights[:, 2])


def test_route_nan_and_infinite_logits(w):
    x = torch.zeros((3, 32), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    x[1, 1] = 1
    r = torch.zeros((8, 32), dtype=torch.bfloat16, device=DEV)
    r[:, 0] = torch.arange(8)
    r[5, 1] = float("-inf")
    r[3, 2] = float("nan")  # 0 * NaN: NaN for every token
    ids, weights, logits = w.qmm_moe_route(x, r, 2)
    assert torch.isnan(logits[:, 3]).all() and torch.isnan(weights).all()
    assert ids[:, 0].cpu().tolist() == [3, 3, 3]
    r[3, 2] = 0
    x[0, 1] = 1e-3
    ids, weights, logits = w.qmm_moe_route(x, r, 2)
    assert logits[1, 5].item() == float("-inf")
    assert ids.cpu().tolist()[1] == [7, 6]
    assert torch.isfinite(weights[1]).all()


MOE = [
    # T, H, I, E, k, bits, gs
    (1, 32, 32, 1, 1, 4, -1), (1, 256, 128, 4, 2, 4, 128), (2, 288, 96, 3, 3, 4, 32), (5, 128, 64, 8, 2, 8, 64),
    (7, 256, 128, 4, 2, 3, 64), (9, 128, 160, 2, 2, 2, 32), (16, 64, 64, 6, 4, 1, 64), (17, 512, 256, 4, 1, 4, -1),
    (33, 96, 192, 3, 2, 3, 96), (64, 128, 64, 2, 2, 4, 64), (64, 64, 32, 40, 16, 8, -1), (4, 1024, 512, 8, 2, 4, 128),
    (40, 160, 96, 1, 1, 2, 32), (12, 96, 544, 5, 3, 4, 32),
]


@pytest.mark.parametrize("strips", [True, False])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,H,I,E,k,bits,gs", MOE)
def test_moe(w, T, H, I, E, k, bits, gs, dtype, strips):
    say(f"moe T={T} H={H} I={I} E={E} k={k} bits={bits} gs={gs} {dtype} strips={strips}")
    x = randn((T, H), dtype, 11 * T + H)
    gu, gu_np = expert_planes(E, H, 2 * I, bits, gs, dtype, strips, seed=1 + bits, zeros="fraction")
    dn, dn_np = expert_planes(E, I, H, bits, gs, dtype, strips, seed=2 + bits)
    g = gen(T + k)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).to(DEV)
    weights = torch.rand((T, k), generator=g).to(DEV)
    y = w.qmm_moe(x, ids, weights, gu, dn, bits, gs, strips=strips)
    want, bound = lo.moe(f64(x), ids.cpu().numpy(), f64(weights), gu_np, dn_np, bits, gs, dtype)
    check(y, want, bound, "y")
    again = w.qmm_moe(x, ids, weights, gu, dn, bits, gs, strips=strips)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16)), "two calls differ"


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_moe_all_tokens_to_one_expert_and_dropped_ids(w, dtype):
    T, H, I, E, k, bits, gs = 64, 128, 96, 5, 3, 4, 32
    x = randn((T, H), dtype, 5)
    gu, gu_np = expert_planes(E, H, 2 * I, bits, gs, dtype, True, seed=8)
    dn, dn_np = expert_planes(E, I, H, bits, gs, dtype, True, seed=9)
    ids = torch.full((T, k), -1, dtype=torch.int32)
    ids[:, 1] = 4
    ids[3] = torch.tensor([E, 1 << 30, -7])  # nothing: row 3 is zero
    ids[9, 2] = 0
    weights = torch.rand((T, k), generator=gen(1)).to(DEV)
    y = w.qmm_moe(x, ids.to(DEV), weights, gu, dn, bits, gs, strips=True)
    want, bound = lo.moe(f64(x), ids.numpy(), f64(weights), gu_np, dn_np, bits, gs, dtype)
    check(y, want, bound, "y")
    assert not y[3].any()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_moe_non_finite_tokens_stay_alone(w, dtype):
    """A token with a NaN or an infinity gives none to the tokens that share its expert."""
    T, H, I, E, k, bits, gs = 6, 64, 64, 3, 2, 4, 32
    x = randn((T, H), dtype, 6)
    x[2, 5] = float("nan")
    x[4, 7] = float("inf")
    gu, _ = expert_planes(E, H, 2 * I, bits, gs, dtype, True, seed=3)
    dn, _ = expert_planes(E, I, H, bits, gs, dtype, True, seed=4)
    ids = torch.tensor([[0, 1]] * T, dtype=torch.int32, device=DEV)
    weights = torch.full((T, k), 0.5, device=DEV)
    y = w.qmm_moe(x, ids, weights, gu, dn, bits, gs, strips=True)
    clean = x.clone()
    clean[2, 5] = clean[4, 7] = 0
    y0 = w.qmm_moe(clean, ids, weights, gu, dn, bits, gs, strips=True)
    rest = [0, 1, 3, 5]
    assert torch.equal(y[rest], y0[rest])
    assert torch.isnan(y[2]).all()
    assert not torch.isfinite(y[4]).all()


def test_moe_large_intermediate_keeps_its_range(w):
    """fp16 data whose intermediate passes the fp16 range: the result stays finite and right."""
    T, H, I, E, bits, gs = 2, 64, 64, 2, 8, -1
    x = randn((T, H), "fp16", 7, 30.0)
    gu, gu_np = expert_planes(E, H, 2 * I, bits, gs, "fp16", False, seed=5)
    gu = (gu[0], gu[1], gu[2], gu[3] * 30)
    gu_np = (gu_np[0], gu_np[1], gu_np[2], f64(gu[3]))
    dn, dn_np = expert_planes(E, I, H, bits, gs, "fp16", False, seed=6)
    dn = (dn[0], dn[1], dn[2], dn[3] / 64)
    dn_np = (dn_np[0], dn_np[1], dn_np[2], f64(dn[3]))
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device=DEV)
    weights = torch.full((T, 1), 1 / 64, device=DEV)
    y = w.qmm_moe(x, ids, weights, gu, dn, bits, gs)
    want, bound = lo.moe(f64(x), ids.cpu().numpy(), f64(weights), gu_np, dn_np, bits, gs, "fp16")
    check(y, want, bound, "y")


def test_moe_on_another_stream_and_empty(w):
    T, H, I, E, k, bits, gs = 8, 256, 128, 8, 2, 4, 64
    x = randn((T, H), "bf16", 1)
    r = randn((E, H), "bf16", 2)
    gu, _ = expert_planes(E, H, 2 * I, bits, gs, "bf16", True, seed=1)
    dn, _ = expert_planes(E, I, H, bits, gs, "bf16", True, seed=2)
    ids, weights, _ = w.qmm_moe_route(x, r, k)
    y = w.qmm_moe(x, ids, weights, gu, dn, bits, gs, strips=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ids2, weights2, _ = w.qmm_moe_route(x, r, k)
        y2 = w.qmm_moe(x, ids2, weights2, gu, dn, bits, gs, strips=True)
    s.synchronize()
    assert torch.equal(ids, ids2) and torch.equal(y, y2)
    e_ids, e_w, e_l = w.qmm_moe_route(x[:0], r, k)
    assert e_ids.shape == (0, k) and e_l.shape == (0, E)
    assert w.qmm_moe(x[:0], e_ids, e_w, gu, dn, bits, gs, strips=True).shape == (0, H)


def test_moe_in_a_graph(w):
    """Route and experts captured once, replayed on new inputs, against eager calls."""
    T, H, I, E, k, bits, gs = 4, 256, 128, 8, 2, 4, 64
    x = randn((T, H), "fp16", 1)
    r = randn((E, H), "fp16", 2)
    gu, _ = expert_planes(E, H, 2 * I, bits, gs, "fp16", True, seed=1)
    dn, _ = expert_planes(E, I, H, bits, gs, "fp16", True, seed=2)
    ws = torch.zeros(8 << 20, dtype=torch.uint8, device=DEV)

    def step():
        ids, weights, _ = w.qmm_moe_route(x, r, k, workspace=ws)
        return w.qmm_moe(x, ids, weights, gu, dn, bits, gs, strips=True, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in range(4):
        x.copy_(randn((T, H), "fp16", 100 + seed))
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got, want), seed
