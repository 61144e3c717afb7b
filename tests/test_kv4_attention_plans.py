"""Which kernel qmm_kv4_attention takes for which sizes, as qmm_kv4_attention_plan_info says, and the sizes it refuses. Host
only; the figures of sizes are for 256 CUs, which a machine without a GPU counts on."""
import ctypes

import pytest

from test_layer_host import NULL, SHAPE, _lib


def plan(*sizes, biased=False):
    import weight_only_group_amd as w
    _lib()
    return w.kv4_attention_plan_info(*sizes, biased=biased)


def need_256_cus():
    if plan(1, 1, 1, 1, 64, 1, 1)["cus"] != 256:
        pytest.skip("sizes for 256 CUs")


# B, T, Hq, Hkv, D, max_q, max_kv, kernel
SIZES = [
    # the sizes that the GPU tests of each kernel are made for
    (4, 4, 8, 2, 128, 1, 4200, "parts"), (4, 31, 6, 2, 64, 20, 4200, "parts"), (2, 70, 8, 4, 256, 40, 4200, "parts"),
    (4, 88, 256, 128, 64, 40, 200, "pair"), (6, 126, 256, 128, 128, 21, 90, "pair"), (5, 200, 256, 128, 64, 40, 40, "pair"),
    (4, 275, 128, 64, 64, 139, 139, "blocks"), (4, 275, 128, 64, 256, 139, 139, "blocks"), (2, 136, 256, 128, 128, 101, 101, "blocks"),
    (2, 220, 160, 80, 128, 130, 200, "blocks"), (2, 350, 96, 96, 128, 200, 210, "blocks"), (2, 170, 200, 100, 256, 100, 100, "blocks"),
    (2, 100, 352, 88, 64, 70, 77, "blocks"), (1, 100, 336, 168, 128, 100, 100, "blocks"), (1, 90, 384, 192, 128, 90, 90, "blocks"),
    (4, 400, 120, 60, 64, 110, 150, "blocks"), (1, 3000, 32, 8, 128, 3000, 3000, "blocks"), (2, 205, 160, 80, 64, 139, 139, "blocks"),
    (1, 200, 168, 8, 256, 200, 200, "blocks"), (1, 3, 32, 8, 128, 3, 3000, "parts"), (1, 3, 336, 168, 128, 3, 200, "tile"),
    # both sides of each rule
    (1, 1, 32, 8, 64, 1, 1536, "tile"), (1, 1, 32, 8, 64, 1, 1537, "parts"), (1, 1, 32, 8, 128, 1, 1024, "tile"),
    (1, 1, 32, 8, 128, 1, 1025, "parts"), (1, 1, 32, 8, 256, 1, 614, "tile"), (1, 1, 32, 8, 256, 1, 615, "parts"),
    (512, 512, 32, 8, 128, 1, 16384, "tile"), (512, 512, 32, 8, 128, 1, 16385, "parts"), (513, 513, 32, 8, 128, 1, 1 << 20, "tile"),
    (1024, 1024, 2, 1, 128, 1, 8192, "parts"), (1025, 1025, 2, 1, 128, 1, 8192, "tile"),
    (1, 128, 4, 4, 128, 128, 1024, "pair"), (1, 129, 4, 4, 128, 129, 513, "parts"), (1, 129, 4, 4, 128, 129, 512, "pair"),
    (1, 129, 4, 4, 256, 129, 307, "tile"), (1, 16, 4, 4, 128, 16, 100, "tile"), (1, 17, 4, 4, 128, 17, 100, "pair"),
    (1, 4064, 32, 8, 128, 4064, 4064, "blocks"), (1, 1017, 32, 8, 128, 1017, 1017, "blocks"), (1, 1016, 32, 8, 128, 1016, 1016, "parts"),
    (33, 1055, 32, 8, 128, 32, 500, "pair"), (33, 1056, 32, 8, 128, 32, 500, "blocks"),
    # one query head a key head: of heads of 64 prompts of few tiles only
    (1, 2000, 32, 32, 64, 2000, 2000, "blocks"), (1, 4000, 32, 32, 64, 4000, 4000, "pair"), (1, 4000, 32, 32, 128, 4000, 4000, "blocks"),
    (1, 4000, 32, 32, 256, 4000, 4000, "blocks"),
]


@pytest.mark.parametrize("case", SIZES, ids=str)
def test_kernel(case):
    need_256_cus()
    *sizes, kernel = case
    assert plan(*sizes)["kernel"] == kernel


def test_distances_count_for_heads_of_256_only():
    need_256_cus()
    for D, Hq, Hkv, kernel in ((64, 32, 32, "pair"), (128, 32, 32, "blocks"), (256, 32, 32, "tile"), (256, 32, 8, "blocks")):
        assert plan(1, 8000, Hq, Hkv, D, 8000, 8000, biased=True)["kernel"] == kernel


@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_workspace_goes_with_parts(D):
    """The bytes of all blocks' sums, for calls with slopes and without."""
    lib = _lib()
    for B in (1, 3, 40, 513, 1024):
        for Hq, Hkv in ((8, 2), (4, 4), (32, 1)):
            for q in (1, 9, 300, 4000):
                for kv in (q, 700, 2000, 9000, 200000):
                    sizes = (B, B * q, Hq, Hkv, D, q, kv)
                    need = lib.qmm_kv4_attention_workspace_bytes(*sizes)
                    for biased in (False, True):
                        p = plan(*sizes, biased=biased)
                        assert p["rows"] == {"tile": 16, "pair": 32, "parts": 16, "blocks": 128 if D == 256 else 256}[p["kernel"]]
                        assert (p["parts"] > 0) == (p["resident"] > 0) == (p["kernel"] == "parts")
                        if p["kernel"] == "parts":
                            assert need == (128 << 10) + p["blocks"] * 16 * (D + 2) * 4


def test_refusals():
    lib = _lib()
    info = (ctypes.c_int32 * 6)()
    call = lib.qmm_kv4_attention_plan_info
    good = (1, 1, 8, 2, 128, 1, 100, 0)
    assert call(*good, info, 6) == 0 and call(*good, None, 0) == 0 and call(*good, None, 6) == NULL
    for at, bad in ((0, 0), (0, 65536), (1, 0), (2, 7), (3, 0), (4, 96), (5, 0), (6, -1)):
        assert call(*good[:at], bad, *good[at + 1:], info, 6) == SHAPE
    assert call(65535, 1 << 20, 8, 2, 128, 1 << 20, 100, 0, info, 6) == SHAPE  # more blocks than a launch has
    info[2] = -7
    assert call(*good, info, 2) == 0 and info[2] == -7
