"""The workspace of calls that are given none, across graph captures and growth:
a graph keeps memory of its own, an eager call never takes over what a capture
only recorded, and a given workspace is checked."""
import numpy as np
import pytest
import torch

from layer_cases import DEV, expert_planes, gen, i32, paged, randn, say
from test_gpu_attention import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


class Attend:
    """Single tokens on long contexts (keys split over blocks, joined by arrival counters)."""

    def __init__(self, w, kv, seed, H=8, Hkv=2, D=128):  # noqa: F811
        self.w, B = w, len(kv)
        self.k, self.v, table = paged(B, kv, Hkv, D, 16, "fp16", seed)
        self.q = randn((B, H, D), "fp16", seed)
        self.rest = (i32(table), i32(np.array(kv)), i32(np.arange(B + 1)), 1, max(kv))
        self.seed = seed

    def __call__(self):
        return self.w.qmm_attention(self.q, self.k, self.v, *self.rest)

    def change(self, n):
        self.q.copy_(randn(self.q.shape, "fp16", 1000 * self.seed + n))


def capture(call):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


def replay(graph, out, call, n):
    call.change(n)
    graph.replay()
    torch.cuda.synchronize()
    got = out.clone()
    want = call()
    torch.cuda.synchronize()
    assert torch.equal(got, want), n


def test_a_graph_outlives_the_growth_of_the_workspace(w):  # noqa: F811
    say("graph, then larger eager calls")
    small, large = Attend(w, [700], 1), Attend(w, [3000] * 40, 2)
    small()
    torch.cuda.synchronize()
    graph, out = capture(small)
    for n in range(4):
        large()
        # what the stream's old buffer was may be another tensor now
        filler = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
        replay(graph, out, small, n)
        assert all(bool((f == 255).all()) for f in filler)


def test_captures_without_a_call_before(w):  # noqa: F811
    say("two graphs, the second replayed first")
    calls = [Attend(w, [900], 3), Attend(w, [400, 1500], 4)]
    graphs = [capture(c) for c in calls]
    for n in range(3):
        for i in (1, 0, 1):
            replay(*graphs[i], calls[i], 10 * n + i)


def test_a_capture_leaves_the_streams_workspace_alone(w):  # noqa: F811
    say("capture on a stream that has a workspace")
    call = Attend(w, [800], 5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    key = (0, stream.cuda_stream)
    ws = w._workspaces[key]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = call()
        again = call()  # the same capture: the same workspace, one behind the other
    assert w._workspaces[key] is ws and w._captured[key][1] is not ws
    for n in range(3):
        call.change(n)
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        assert torch.equal(out, want) and torch.equal(again, want)
    torch.cuda.synchronize()
    assert not ws[:w.WORKSPACE_HEADER].any()


def test_a_whole_layer_captured_without_workspaces(w):  # noqa: F811
    say("route, experts and log probabilities in one graph")
    T, H, I, E, k, bits, gs = 5, 256, 128, 8, 2, 4, 64
    x, r = randn((T, H), "bf16", 1), randn((E, H), "bf16", 2)
    gu, _ = expert_planes(E, H, 2 * I, bits, gs, "bf16", True, seed=1)
    dn, _ = expert_planes(E, I, H, bits, gs, "bf16", True, seed=2)
    big = randn((2, 200000), "bf16", 3)

    def step():
        ids, weights, _ = w.qmm_moe_route(x, r, k)
        return [w.qmm_moe(x, ids, weights, gu, dn, bits, gs, strips=True), *w.qmm_logprobs(big, top=20)[1:]]

    graph, out = capture(step)
    for n in range(3):
        x.copy_(randn((T, H), "bf16", 10 + n))
        big.copy_(randn(big.shape, "bf16", 20 + n))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, step()):
            assert torch.equal(a, b), n


def test_the_decode_product_captured_without_a_workspace(w):  # noqa: F811
    K, N, bits, gs = 8192, 256, 4, 128
    assert w.workspace_bytes(1, K, N, bits, gs) > 0
    r = torch.randint(0, 16, (K, N), generator=gen(1)).to(torch.uint8).to(DEV)
    qw, _ = w.qmm_pack(r, bits)
    z = torch.full((K // gs, N), 7.0, dtype=torch.float16, device=DEV)
    s = torch.full((K // gs, N), 0.01, dtype=torch.float16, device=DEV)
    x = randn((1, K), "fp16", 1)
    graph, out = capture(lambda: w.qmm_gemv(x, qw, None, z, s, bits, gs))
    for n in range(4):
        x.copy_(randn((1, K), "fp16", 5 + n))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, w.qmm_gemv(x, qw, None, z, s, bits, gs)), n


def test_given_workspaces_are_checked(w):  # noqa: F811
    q = randn((1, 4, 64), "fp16", 1)
    k = torch.zeros((2, 2, 16, 64), dtype=torch.float16, device=DEV)
    attend = lambda ws: w.qmm_attention(q, k, k, i32(np.zeros((1, 2))), i32(np.ones(1)), i32(np.arange(2)), 1, 16, workspace=ws)  # noqa: E731
    x, r = randn((2, 64), "fp16", 1), randn((4, 64), "fp16", 2)
    qw, _ = w.qmm_pack(torch.zeros((64, 16), dtype=torch.uint8, device=DEV), 4)
    one = torch.ones((1, 16), dtype=torch.float16, device=DEV)
    calls = [attend, lambda ws: w.qmm_moe_route(x, r, 1, workspace=ws), lambda ws: w.qmm_logprobs(x, workspace=ws),
             lambda ws: w.qmm_gemv(x, qw, None, one, one, 4, -1, workspace=ws)]
    for call in calls:
        with pytest.raises(ValueError, match="on cuda"):
            call(torch.zeros(4 << 20, dtype=torch.uint8))
        with pytest.raises(ValueError, match="contiguous"):
            call(torch.zeros((4, 1 << 20), dtype=torch.uint8, device=DEV)[:, ::2])
        with pytest.raises(TypeError):
            call(1 << 20)
        call(torch.zeros(4 << 20, dtype=torch.uint8, device=DEV))
    with pytest.raises(w.QmmError):
        w.qmm_moe_route(x, r, 1, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
