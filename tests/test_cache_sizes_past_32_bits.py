"""Sizes past 32 bits given to the 4-bit cache's calls, the care of pages and the attention: refused by name, not cut to
their low bits. Without a GPU; the calls on tensors are held to it in test_gpu_cache_sizes_past_32_bits.py."""
import pytest

from test_layer_host import _lib

PAST = [2**31, 2**32 + 16, -2**31 - 1000, -2**32 + 16, 2**64 + 16]


@pytest.mark.parametrize("n", PAST)
def test_page_bytes(n):
    import weight_only_group_amd as w
    _lib()
    assert w.kv4_page_bytes(16, 64, 32) == 640
    for sizes in ((n, 64, 32), (16, n + 48, 32), (16, 64, n + 16)):
        with pytest.raises(ValueError, match="2\\^31"):
            w.kv4_page_bytes(*sizes)


@pytest.mark.parametrize("n", PAST)
def test_plan(n):
    import weight_only_group_amd as w
    _lib()
    good = dict(B=1, T=16, Hq=16, Hkv=16, D=64, max_q=16, max_kv=16)
    w.kv4_attention_plan_info(**good)
    for name in good:
        with pytest.raises(ValueError, match=name):
            w.kv4_attention_plan_info(**good | {name: n})


@pytest.mark.parametrize("n", PAST)
def test_compaction(n):
    import weight_only_group_amd as w
    with pytest.raises(ValueError, match="page_size"):
        w.qmm_kv_compact([], None, None, n)
