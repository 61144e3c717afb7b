"""The largest scale of a group of the 4-bit cache that stands for numbers: as the header, the binding and the oracle have
it, and as fp16 arithmetic gives it. Without a GPU."""
import os
import re

import numpy as np

from oracle import cache_oracle as co
from test_layer_host import ROOT


def test_header_binding_and_oracle_agree():
    import weight_only_group_amd as w
    text = open(os.path.join(ROOT, "include", "qmm_cache.h")).read()
    assert int(re.search(r"#define QMM_KV4_LARGEST_SCALE (\d+)", text)[1]) == w.cache.LARGEST_SCALE == co.LARGEST_SCALE


def test_24_times_a_scale_is_a_number_up_to_the_limit_only():
    """So is 16 + 15 times it less that; scales of 8 bits are then exact."""
    s = np.arange(2**15, dtype=np.uint16).view(np.float16)
    s = s[np.isfinite(s)]
    with np.errstate(over="ignore"):
        assert np.array_equal(np.isfinite(s * np.float16(24)), s <= co.LARGEST_SCALE)
    mantissa = np.frexp(s.astype(np.float64))[0] * 256
    eight = s[(mantissa == np.rint(mantissa)) & (s <= co.LARGEST_SCALE)].astype(np.float64)
    assert eight.max() == 2720
    for c in [*range(-8, 8), 24]:
        assert np.array_equal((eight * c).astype(np.float16).astype(np.float64), eight * c)


def test_the_append_stays_below_it():
    x = np.array([[-1e30, 1e30] * 16, [-16384, 16384] * 16], np.float32)
    assert (co.quantise(x, 32)[0] == 2192).all()


def test_parts_are_nan_beyond_it():
    D, group = 64, 32
    for s, bad in ((2728.0, False), (2730.0, True), (-2728.0, False), (-3000.0, True), (65504.0, True)):
        for keys in (True, False):
            cache = np.zeros((1, 1, co.block_bytes(D, group)), np.uint8)
            co.put(cache, 0, 0, 3, [np.float16(s), np.float16(1)], np.zeros(2, np.float16), np.full(D, 9), group, keys)
            step, middle = (p[0, 0, 3] for p in co.parts(cache, D, group, keys))
            for p, want in ((step, s), (middle, 0.0)):
                assert np.isnan(p[:32]).all() if bad else (p[:32] == want).all()
            assert (step[32:] == 1).all() and (middle[32:] == 0).all()


def test_scales_of_more_bits_are_off_by_a_64th():
    """What the attention's decoding makes of such a scale: 24 s and the sum, each rounded to fp16."""
    s = np.arange(2**15, dtype=np.uint16).view(np.float16)
    s = s[np.isfinite(s) & (s <= co.LARGEST_SCALE) & (s >= 2.0**-14)]
    down = (s * np.float16(-24)).astype(np.float64)  # rounded
    for c in range(-8, 8):
        held = ((24.0 + c) * s.astype(np.float64) + down).astype(np.float16).astype(np.float64)  # one rounding, as of a multiply-add
        assert (np.abs(held - c * s.astype(np.float64)) <= s.astype(np.float64) / 64).all()
