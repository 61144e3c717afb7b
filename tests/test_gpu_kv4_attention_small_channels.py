"""Channels of a query far smaller than its largest one, in qmm_kv4_attention: down to 2^-14 of it (bf16: 2^-17) they count in
full. The keys are 0 in the largest channel and thousands in the others, so that the small ones make the scores; bounds are the
oracle's for the query without its largest channel, which has no part in them."""
import numpy as np
import pytest
import torch

from cache_cases import device, paged4
from layer_cases import DEV, TYPES, check, f64, i32, say
from oracle import cache_oracle as co
from test_gpu_kv4_cache import w  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

KERNELS = [("tile", 1, 1, 16, 4, 300), ("tile", 1, 8, 8, 4, 300), ("pair", 5, 40, 256, 128, 300), ("parts", 1, 1, 16, 4, 4200),
           ("parts", 1, 30, 8, 4, 4200), ("blocks", 1, 100, 336, 168, 300)]
CASES = [(*kernel, *size) for kernel in KERNELS for size in ((64, 32), (128, 32), (128, 64), (256, 64))
         if (kernel[0], size[0]) != ("pair", 256)]  # heads of 256 have no pairs of tiles
KV, PAGE = 300, 16


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("name,B,T,Hq,Hkv,max_kv,D,group", CASES)
def test_they_count_in_full(w, name, B, T, Hq, Hkv, max_kv, D, group, dtype):  # noqa: F811
    assert w.kv4_attention_plan_info(B, B * T, Hq, Hkv, D, T, max_kv)["kernel"] == name
    say(f"kv4 small channels {name} T={T} D={D} group={group} {dtype}")
    k, v, table = paged4([KV] * B, Hkv, D, PAGE, group, 1)
    r = np.random.default_rng(2)
    blocks = k.reshape(len(k), Hkv, PAGE // 8, -1)
    for t in range(8):
        for g in range(D // group):
            s = np.float16(r.integers(128, 256, blocks.shape[:-1]) * (g > 0))
            m = np.float16(r.uniform(-8000, 8000, blocks.shape[:-1]) * (g > 0))
            for at, x in zip(co.scale_places(t, g, D, group, True), (s, m)):
                blocks[..., at:at + 2] = np.ascontiguousarray(x)[..., None].view(np.uint8)
    steps = 1024 if dtype == "fp16" else 128  # values with all the bits their type has
    q = (1 + r.integers(0, steps, (B * T, Hq, D)) / steps) * 2.0 ** (-14 if dtype == "fp16" else -17) * r.choice([-1, 1], (B * T, Hq, D))
    q[..., 0] = 1
    if max_kv > table.shape[1] * PAGE:
        table = np.pad(table, ((0, 0), (0, -(-max_kv // PAGE) - table.shape[1])))
    dq = torch.from_numpy(q).to(TYPES[dtype]).to(DEV)
    assert (f64(dq) == q).all()
    G = Hq // Hkv
    scale = 1.0 if dtype == "fp16" else 8.0
    out = w.qmm_kv4_attention(dq, device(k), device(v), i32(table), i32(np.full(B, KV)), i32(np.arange(B + 1) * T), T, max_kv, group,
                              scale=scale)[-T:, :4 * G]
    q[..., 0] = 0
    part = lambda c, keys: [x[:, :4] for x in co.parts(c, D, group, keys)]  # noqa: E731
    want, bound = co.attention(q[-T:, :4 * G], part(k, True), part(v, False), table[-1:], [KV], [0, T], scale, group, dtype=dtype)
    check(out, want, bound, "out")
    # Small enough that the channels' last bits show: without them the results are elsewhere.
    less = np.ldexp(np.trunc(np.ldexp(q, 24)) // 4 * 4, -24)
    other = co.attention(less[-T:, :4 * G], part(k, True), part(v, False), table[-1:], [KV], [0, T], scale, group, dtype=dtype)[0]
    assert (np.abs(other - want) > bound).any()
