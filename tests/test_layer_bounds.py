"""The limit on the norm of the experts' error has teeth: a result with a mistake
planted in it (on the CPU, in float64) passes it only without the mistake."""
import numpy as np
import pytest

from oracle import layer_oracle as lo

CASES = [(4, 1024, 512, 4, 2, 4, 128), (9, 2048, 1024, 2, 1, 4, 128), (24, 864, 1504, 2, 1, 1, -1), (6, 1024, 992, 2, 2, 2, 32)]


def data(T, H, I, E, k, bits, gs, dtype, seed=5):
    r = np.random.default_rng(seed)

    def planes(K, N):
        groups = 1 if gs == -1 else K // gs
        words = r.integers(-2**31, 2**31, (E, K * bits // 32, N), dtype=np.int64).astype(np.int32)
        scales = r.uniform(0.5, 1.5, (E, groups, N)) / np.sqrt((4.0**bits - 1) / 6 * K)
        return words, None, r.integers(0, 2**bits, scales.shape).astype(np.float64), lo.rounded(scales, dtype)

    x = lo.rounded(r.standard_normal((T, H)), dtype)
    ids = np.array([r.permutation(E)[:k] for _ in range(T)], np.int32)
    return x, ids, r.uniform(0, 1, (T, k)), planes(H, 2 * I), planes(I, H)


def in_bits(v, bits):
    """v to `bits` significant bits."""
    m, e = np.frexp(v)
    return np.ldexp(np.round(m * 2.0**bits) / 2.0**bits, e)


def result(x, ids, weights, gate_up, down, bits, gs, dtype, mistake):
    xs = x.copy()
    if mistake == "unit_of_x_lost":
        xs[:, -32:] = 0
    h, _ = lo.moe_hidden(xs, ids, gate_up, bits, gs)
    if mistake == "low_part_lost":
        h = in_bits(h, 8)
    elif mistake == "five_bits":
        h = in_bits(h, 5)
    elif mistake == "unit_of_h_lost":
        h[..., -32:] = 0
    else:
        h = in_bits(h, 16)
    wt = lo.rounded(weights, "bf16") if mistake == "weights_in_8_bits" else weights
    y, _ = lo.moe_down(h, ids, wt, down, bits, gs)
    if mistake == "rounded_twice":
        y = in_bits(y, 8 if dtype == "bf16" else 11) * (1 + 2.0**-11 * np.random.default_rng(1).choice([-1, 1], y.shape))
    if mistake == "scaled":
        y = y * 1.004
    return lo.rounded(y, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_planted_mistakes_pass_no_norm(case, dtype):
    args = data(*case, dtype)
    bits, gs = case[5:]
    want, limit = lo.moe_norm(*args, bits, gs, dtype)
    error = lambda m: np.linalg.norm(result(*args, bits, gs, dtype, m) - want) / np.linalg.norm(want)  # noqa: E731
    assert error(None) < limit
    mistakes = ["unit_of_x_lost", "unit_of_h_lost", "low_part_lost", "five_bits", "scaled", "weights_in_8_bits"]
    if dtype == "fp16":  # (in bf16 far below the result's own rounding)
        mistakes.append("rounded_twice")
    passed = [m for m in mistakes if error(m) <= limit]
    assert not passed, (passed, limit)


def test_the_norms_result_is_the_bounds():
    """Both oracles of the layer agree, ids outside included."""
    x, ids, weights, gu, dn = data(5, 128, 96, 3, 2, 4, 32, "fp16")
    ids[2] = [-1, 3]
    ids[4, 0] = 1 << 30
    y, _ = lo.moe(x, ids, weights, gu, dn, 4, 32, "fp16")
    again, limit = lo.moe_norm(x, ids, weights, gu, dn, 4, 32, "fp16")
    assert np.allclose(y, again, rtol=1e-12, atol=1e-12 * np.abs(y).max()) and not again[2].any() and 0 < limit < 1e-3


@pytest.mark.parametrize("softcap", [1e5, 1e6, 1e8])
def test_a_cap_with_cancellation_passes_no_bound(softcap):
    """cap - 2 cap / (1 + e^2x) in fp32, for scores far below the cap."""
    r = np.random.default_rng(2)
    D, n = 64, 300
    q, k, v = lo.rounded(1.5 * r.standard_normal((1, 1, D)), "fp16"), *(
        lo.rounded(r.standard_normal((1, 1, n, D)), "fp16") for _ in range(2))
    want, bound = lo.attention(q, k, v, np.zeros((1, 1), int), [n], [0, 1], D**-0.5, softcap=softcap)
    s = (k[0, 0] @ q[0, 0] * D**-0.5).astype(np.float32)
    c, one, two = np.float32(softcap), np.float32(1), np.float32(2)
    t = c - two * c / (one + np.exp(two * s / c))
    p = np.exp(t.astype(np.float64) - t.max())
    assert (np.abs(p @ v[0, 0] / p.sum() - want[0, 0]) > bound[0, 0]).any()
    s = s.astype(np.float64)
    p = np.exp(s - s.max())
    assert (np.abs(p @ v[0, 0] / p.sum() - want[0, 0]) <= bound[0, 0]).all()
