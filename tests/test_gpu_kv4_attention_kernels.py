"""Each kernel of qmm_kv4_attention, named by qmm_kv4_attention_plan_info before the call, against float64 at the bounds of
the other tests; the workspace that calls in parts of the keys share, in graphs and passed round."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import DEV, i32, randn, say
from test_gpu_kv4_attention import run
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

HEADER = 128 << 10  # bytes of counters at a workspace's start


def kernel(w, kv_lens, q_lens, Hq, Hkv, D, max_kv=None, biased=False):  # noqa: F811
    return w.kv4_attention_plan_info(len(kv_lens), sum(q_lens), Hq, Hkv, D, max(q_lens), max_kv or max(kv_lens), biased)["kernel"]


CASES = [("tile", [1, 700, 33], [1, 1, 1], 8, 2), ("tile", [40, 700, 9], [3, 16, 1], 2, 2), ("pair", [40, 200, 30, 9], [40, 8, 1, 9], 256, 128),
         ("parts", [1300, 1, 133], [1, 1, 1], 8, 2), ("parts", [1100, 7, 150], [3, 7, 20], 6, 2), ("blocks", [139, 1, 66, 133], [139, 1, 65, 70], 128, 64)]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 64), (256, 128)])
@pytest.mark.parametrize("name,kv_lens,q_lens,Hq,Hkv", CASES)
def test_the_kernel_named(w, name, kv_lens, q_lens, Hq, Hkv, D, group, dtype):  # noqa: F811
    max_kv = {"parts": 4200, "tile": 600 if D == 256 else 700}.get(name, max(kv_lens))
    kv_lens = [min(n, max_kv) for n in kv_lens]
    want = "tile" if name == "pair" and D == 256 else name  # heads of 256 have no pairs
    assert kernel(w, kv_lens, q_lens, Hq, Hkv, D, max_kv) == want
    run(w, kv_lens, q_lens, Hq, Hkv, D, 16, group, dtype, max_kv=max_kv)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("kv", [1, 17, 700, 4099])
def test_one_sequence_in_parts(w, kv, dtype):  # noqa: F811
    assert kernel(w, [kv], [1], 8, 2, 128, 4200) == "parts"
    run(w, [kv], [1], 8, 2, 128, 16, 64, dtype, max_kv=4200)


def long_call(lens, seed, q=1, max_kv=4200, D=128):
    """Arguments of a call in parts, its lengths on the device among them."""
    k, v, table = paged4(lens, 2, D, 16, 64, seed)
    table = np.pad(table, ((0, 0), (0, -(-max_kv // 16) - table.shape[1])))
    return [randn((len(lens) * q, 8, D), "bf16", seed + 1), device(k), device(v), i32(table), i32(np.array(lens)),
            i32(np.arange(len(lens) + 1) * q), q, max_kv, 64]


def test_equal_bits_and_other_stream_in_parts(w):  # noqa: F811
    assert kernel(w, [2000, 300], [1, 1], 8, 2, 128, 4200) == "parts"
    args = long_call([2000, 300], 1)
    a = w.qmm_kv4_attention(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b = w.qmm_kv4_attention(*args)
    s.synchronize()
    assert torch.equal(a, b)
    for _ in range(5):
        assert torch.equal(a, w.qmm_kv4_attention(*args))


def test_a_workspace_passed_round_in_parts(w):  # noqa: F811
    """One zeroed buffer for calls of several kinds, which leave its counters at zero."""
    args = long_call([2000, 300], 1)
    few = long_call([3000, 1], 2, q=20, D=64)
    need = [w.library().qmm_kv4_attention_workspace_bytes(2, 2 * q, 8, 2, D, q, 4200) for q, D in ((1, 128), (20, 64))]
    assert min(need) > HEADER
    k16, v16 = w.qmm_kv4_gather(*args[1:3], torch.arange(len(args[1]) * 16, device=DEV), 128, 64, torch.bfloat16)
    k16, v16 = (t.unflatten(0, (len(args[1]), 16)).transpose(1, 2).contiguous() for t in (k16, v16))
    logits = randn((2, 5000), "bf16", 3)
    kinds = [lambda ws: w.qmm_kv4_attention(*args, workspace=ws), lambda ws: w.qmm_attention(args[0], k16, v16, *args[3:8], workspace=ws),
             lambda ws: w.qmm_kv4_attention(*few, workspace=ws),
             lambda ws: w.qmm_kv_compact([args[1].clone(), args[2].clone()], args[3], args[4], 16, workspace=ws)[0],
             lambda ws: w.qmm_logprobs(logits, torch.tensor([3, 7], device=DEV), top=2, workspace=ws)[0]]
    want = [f(None) for f in kinds]
    ws = torch.zeros(max(*need, 1 << 24), dtype=torch.uint8, device=DEV)
    for i in range(3):
        for j, (f, x) in enumerate(zip(kinds, want)):
            assert torch.equal(f(ws), x), (i, j)
            assert not ws[:HEADER].any(), (i, j)


def test_a_workspace_of_just_the_size(w):  # noqa: F811
    """And of a byte less, which is refused."""
    args = long_call([4000, 3], 1)
    need = w.library().qmm_kv4_attention_workspace_bytes(2, 2, 8, 2, 128, 1, 4200)
    room = torch.zeros(need + 4096, dtype=torch.uint8, device=DEV)
    room[need:] = 77
    assert torch.equal(w.qmm_kv4_attention(*args, workspace=room[:need]), w.qmm_kv4_attention(*args))
    assert (room[need:] == 77).all()
    with pytest.raises((w.QmmError, ValueError)):
        w.qmm_kv4_attention(*args, workspace=room[:need - 1])


def test_a_graph_of_a_decoding_step_in_parts(w):  # noqa: F811
    """Append, attention and the care of the pages in one graph, replayed for other tokens, against the same calls made eagerly."""
    Hq, Hkv, D, page, group, B, bound = 8, 2, 128, 16, 64, 3, 4208
    lens = [3000, 301, 64]
    assert kernel(w, lens, [1] * B, Hq, Hkv, D, bound) == "parts"
    k4, v4, table = paged4(lens, Hkv, D, page, group, 1, spare=8)
    tdev = i32(np.pad(table, ((0, 0), (0, bound // page - table.shape[1]))))
    caches, other = ([device(c) for c in (k4, v4)] for _ in range(2))
    q, k, v = (randn((B, h, D), "bf16", h + i) for i, h in enumerate((Hq, Hkv, Hkv)))
    kv, slots, starts = i32(np.array(lens)), torch.zeros(B, dtype=torch.int64, device=DEV), i32(np.arange(B + 1))
    src, dst = i32(np.array([-1])), i32(np.array([0]))

    def step(caches):
        got = w.qmm_kv4_append(q, k, v, None, None, None, slots, *caches, group)
        out = w.qmm_kv4_attention(got, *caches, tdev, kv, starts, 1, bound, group)
        w.qmm_kv_copy_pages(caches, src, dst)
        return out, *w.qmm_kv_compact(caches, tdev, kv, page)

    def inputs(i):
        now = np.array(lens) - i
        slots.copy_(device(np.array([table[b, (n - 1) // page] * page + (n - 1) % page for b, n in enumerate(now)], np.int64)))
        kv.copy_(i32(now))
        for t in (q, k, v):
            t.copy_(randn(t.shape, "bf16", 7 * i + t.shape[1]))

    inputs(0)
    for c in (caches, other):
        step(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches)
    for i in (1, 2, 3):
        say(f"replay {i}")
        inputs(i)
        for c, o, a in zip(caches, other, (k4, v4)):
            c.copy_(device(a))
            o.copy_(device(a))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, *caches)]
        for a, b in zip(got, (*step(other), *other)):
            assert torch.equal(a, b), i
