"""A small decoder on the library's operators: quantised projections and experts,
a paged key/value cache, a prompt taken at once and tokens decoded one by one.

    python examples/decoder_layers.py

Weights are random (there is nothing to load), so the text means nothing; what
the run shows is how the calls fit together, and that decoding a token gives the
log probabilities that the prompt gave for it.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_group_amd as qmm  # noqa: E402

BITS, GROUP = 4, 64
PAGE = 16


class Linear:
    """A quantised projection: packed once, in 16-column strips; few rows take the decode product."""

    def __init__(self, K, N, gen, dtype):
        codes = torch.randint(0, 1 << BITS, (K, N), generator=gen, device="cuda", dtype=torch.uint8)
        words, self.lo = qmm.qmm_pack(codes, BITS)
        self.words = qmm.qmm_to_strips(words)
        self.zeros = torch.full((K // GROUP, N), 7.5, device="cuda", dtype=dtype)
        self.scales = torch.full((K // GROUP, N), 0.2 / K**0.5, device="cuda", dtype=dtype)

    def __call__(self, x):
        product = qmm.qmm_gemv if x.shape[0] <= qmm.GEMV_MAX_M else qmm.qmm_gemm
        return product(x, self.words, self.lo, self.zeros, self.scales, BITS, GROUP, strips=True)


def experts(E, K, N, gen, dtype):
    """E projections behind one another, as qmm_moe takes them."""
    each = [Linear(K, N, gen, dtype) for _ in range(E)]
    return tuple(None if getattr(each[0], n) is None else torch.stack([getattr(e, n) for e in each])
                 for n in ("words", "lo", "zeros", "scales"))


def norm(x):
    return torch.nn.functional.rms_norm(x, x.shape[-1:])


class Layer:
    def __init__(self, m, gen):
        self.m = m
        self.qkv = Linear(m.H, (m.Hq + 2 * m.Hkv) * m.D, gen, m.dtype)
        self.out = Linear(m.Hq * m.D, m.H, gen, m.dtype)
        self.router = torch.randn((m.E, m.H), generator=gen, device="cuda").to(m.dtype)
        self.gate_up, self.down = experts(m.E, m.H, 2 * m.I, gen, m.dtype), experts(m.E, m.I, m.H, gen, m.dtype)
        self.k_cache = torch.zeros((m.pages, m.Hkv, PAGE, m.D), device="cuda", dtype=m.dtype)
        self.v_cache = torch.zeros_like(self.k_cache)

    def __call__(self, x, batch):
        m = self.m
        q, k, v = (t.unflatten(1, (-1, m.D)) for t in
                   self.qkv(norm(x)).split([m.Hq * m.D, m.Hkv * m.D, m.Hkv * m.D], dim=1))  # views: no copies
        q = qmm.qmm_kv_append(q, k, v, m.cos, m.sin, batch["positions"], batch["slots"], self.k_cache, self.v_cache)
        a = qmm.qmm_attention(q, self.k_cache, self.v_cache, batch["table"], batch["kv_lens"], batch["q_starts"],
                              batch["max_q"], batch["max_kv"], softcap=30.0)
        x = x + self.out(a.flatten(1))
        h = norm(x)
        return x + torch.cat([self.moe(part) for part in h.split(qmm.layer.MOE_MAX_TOKENS)])

    def moe(self, h):
        ids, weights, _ = qmm.qmm_moe_route(h, self.router, self.m.k)
        return qmm.qmm_moe(h, ids, weights, self.gate_up, self.down, BITS, GROUP, strips=True)


class Decoder:
    H, Hq, Hkv, D, E, k, I, V, layers_n, longest = 512, 8, 2, 64, 8, 2, 256, 1000, 2, 512

    def __init__(self, sequences, dtype=torch.float16, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = dtype
        per = -(-self.longest // PAGE)
        self.pages = sequences * per
        # Pages in any order: a cache that has been in use for a while.
        self.table = torch.randperm(self.pages, generator=gen, device="cuda").to(torch.int32).view(sequences, per)
        angle = torch.arange(self.longest, device="cuda")[:, None] * 10000.0 ** (-torch.arange(self.D // 2, device="cuda") * 2 / self.D)
        self.cos, self.sin = angle.cos(), angle.sin()
        self.embed = torch.randn((self.V, self.H), generator=gen, device="cuda").to(dtype)
        self.layers = [Layer(self, gen) for _ in range(self.layers_n)]
        self.head = Linear(self.H, self.V, gen, dtype)

    def batch(self, kv_lens, q_lens):
        """What the calls need to know of a step: sequence b's last q_lens[b] of kv_lens[b] tokens are new."""
        seq = torch.repeat_interleave(torch.arange(len(kv_lens)), torch.tensor(q_lens))
        pos = torch.cat([torch.arange(n - m, n) for n, m in zip(kv_lens, q_lens)])
        page = self.table.cpu()[seq, pos // PAGE].long()
        dev = lambda t, d=torch.int32: t.to(d).cuda()  # noqa: E731
        return dict(positions=dev(pos), slots=dev(page * PAGE + pos % PAGE, torch.int64), table=self.table,
                    kv_lens=dev(torch.tensor(kv_lens)), q_starts=dev(torch.tensor([0, *q_lens]).cumsum(0)), max_q=max(q_lens),
                    max_kv=max(kv_lens))

    def __call__(self, tokens, kv_lens, q_lens, targets, top=3):
        """New tokens of all sequences, one behind another -> log probabilities of `targets`, entropy, alternatives."""
        batch = self.batch(kv_lens, q_lens)
        x = self.embed[tokens]
        for layer in self.layers:
            x = layer(x, batch)
        return qmm.qmm_logprobs(self.head(norm(x)), targets, top=top)


def main(prompts=(150, 37, 91), steps=5):
    model = Decoder(len(prompts))
    gen = torch.Generator(device="cuda").manual_seed(1)
    tokens = [torch.randint(0, model.V, (n,), generator=gen, device="cuda") for n in prompts]
    lens = list(prompts)
    # The prompts at once: every token's successor is scored, the last one's drawn below.
    after = [torch.cat([t[1:], t.new_tensor([-1])]) for t in tokens]
    logprob, entropy, _, ids = model(torch.cat(tokens), lens, lens, torch.cat(after))
    print(f"prompts of {list(prompts)} tokens: mean log probability {logprob.sum().item() / (sum(lens) - len(lens)):.4f}, "
          f"mean entropy {entropy.mean().item():.4f}")
    last = ids[torch.tensor(lens).cumsum(0) - 1, 0].long()
    taken = []
    for step in range(steps):
        lens = [n + 1 for n in lens]
        logprob, entropy, top, ids = model(last, lens, [1] * len(lens), torch.full_like(last, -1))
        taken.append(last)
        print(f"step {step}: tokens {last.tolist()}, next {ids[:, 0].tolist()} at {[round(v, 4) for v in top[:, 0].tolist()]}")
        last = ids[:, 0].long()
    # The same tokens as one prompt give the same log probabilities for the next one.
    whole = [torch.cat([t, torch.stack(taken)[:, i]]) for i, t in enumerate(tokens)]
    check = model(torch.cat(whole), lens, lens, torch.full((sum(lens),), -1, device="cuda"))
    at = torch.tensor(lens).cumsum(0) - 1
    difference = (check[2][at, 0] - top[:, 0]).abs().max().item()
    print(f"decoded step by step against one prompt: log probabilities differ by {difference:.2e} at most")
    return difference


if __name__ == "__main__":
    main()
