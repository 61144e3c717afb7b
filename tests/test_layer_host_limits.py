"""Refusals of calls larger than a launch, without a GPU: the pointers are fake and
never dereferenced."""
import pytest

from test_layer_host import SHAPE, _attention, lib  # noqa: F401  (the fixture)


@pytest.mark.parametrize("kw", [dict(B=65535, Hq=4096, Hkv=4096, qs=4096 * 128, max_q=1), dict(B=65535, Hq=64, Hkv=8, qs=64 * 128, max_q=1024),
                                dict(B=4096, Hq=64, Hkv=64, qs=64 * 128, max_q=1 << 24)], ids=str)
def test_attention_grids_past_a_launch(lib, kw):  # noqa: F811
    assert _attention(lib, **kw) == SHAPE, lib.qmm_last_error()
    assert b"call of their own" in lib.qmm_last_error()
