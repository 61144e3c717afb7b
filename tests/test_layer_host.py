"""The layer operators without a GPU: exported symbols, refusals before any
launch, workspace sizes, and pins of their float64 oracle.

The pointers of the refused calls are fake and never dereferenced; a call that
got past validation would report QMM_ERR_HIP on a machine without a GPU.
"""
import ctypes
import math
import os
import re

import numpy as np
import pytest

from oracle import layer_oracle as lo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, MIS = 0x10000, 0x10004
NULL, BITS, SHAPE, GROUP, ALIGN, WORKSPACE, FLAGS = 1, 2, 3, 4, 5, 6, 8


def _lib():
    import weight_only_group_amd as w
    if not os.path.exists(w.LIB_PATH):
        from weight_only_group_amd import build
        build.build()
    return w.library()


@pytest.fixture
def lib():
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-validation tests use fake pointers; run them where no GPU is visible")
    return _lib()


def test_exports():
    import weight_only_group_amd as w
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qmm_layer.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b(qmm_[a-z0-9_]+)\s*\(", text))
    assert declared == set(w.layer.EXPORTS)
    _lib()
    raw = ctypes.CDLL(w.LIB_PATH)
    for name in declared:
        assert getattr(raw, name) is not None


def _route(lib, **kw):
    a = dict(x=A, T=4, H=256, r=A, E=16, k=2, fl=0, ids=A, wt=A, lg=A, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.qmm_moe_route(*a.values(), None)


ROUTE = [(dict(T=65), SHAPE), (dict(T=-1), SHAPE), (dict(H=48), SHAPE), (dict(H=0), SHAPE), (dict(E=0), SHAPE),
         (dict(E=1025), SHAPE), (dict(k=0), SHAPE), (dict(k=17), SHAPE), (dict(E=1, k=2), SHAPE), (dict(fl=2), FLAGS),
         (dict(fl=1 << 31), FLAGS), (dict(x=None), NULL), (dict(r=None), NULL), (dict(ids=None), NULL), (dict(wt=None), NULL),
         (dict(lg=None), NULL), (dict(x=MIS), ALIGN), (dict(r=MIS), ALIGN), (dict(ids=A + 2), ALIGN), (dict(ws=None), WORKSPACE),
         (dict(wsb=16), WORKSPACE), (dict(ws=MIS), ALIGN), (dict(H=2**31 - 32), SHAPE)]


@pytest.mark.parametrize("kw,want", ROUTE, ids=str)
def test_route_refuses(lib, kw, want):
    assert _route(lib, **kw) == want, lib.qmm_last_error()
    assert lib.qmm_last_error()


def _moe(lib, gu=None, dn=None, **kw):
    import weight_only_group_amd as w
    a = dict(x=A, T=4, H=256, I=128, E=16, k=2, ids=A, wt=A, gu=(A,) * 4, dn=(A,) * 4, bits=4, gs=64, fl=0, y=A, ws=A,
             wsb=1 << 30)
    a.update(kw)
    for n, given in (("gu", gu), ("dn", dn)):
        planes = dict(zip(("qw", "lo", "z", "s"), a[n])) | (given or {})
        a[n] = ctypes.byref(w.layer.Experts(*planes.values()))
    return lib.qmm_moe(*a.values(), None)


MOE = [(dict(bits=5), BITS), (dict(T=65), SHAPE), (dict(T=-1), SHAPE), (dict(H=40), SHAPE), (dict(I=40), SHAPE), (dict(I=0), SHAPE),
       (dict(E=0), SHAPE), (dict(k=17), SHAPE), (dict(k=0), SHAPE), (dict(gs=48), GROUP), (dict(gs=0), GROUP),
       (dict(gs=256), GROUP), (dict(H=1 << 20, I=1 << 16, gs=-1), SHAPE), (dict(fl=4), FLAGS), (dict(x=None), NULL),
       (dict(ids=None), NULL), (dict(wt=None), NULL), (dict(y=None), NULL), (dict(gu=dict(qw=None)), NULL),
       (dict(dn=dict(s=None)), NULL), (dict(dn=dict(lo=None), bits=3), NULL), (dict(gu=dict(z=MIS)), ALIGN),
       (dict(dn=dict(lo=MIS), bits=3), ALIGN), (dict(x=MIS), ALIGN), (dict(y=MIS), ALIGN), (dict(ids=A + 1), ALIGN),
       (dict(ws=None), WORKSPACE), (dict(wsb=1024), WORKSPACE), (dict(ws=MIS), ALIGN)]


@pytest.mark.parametrize("kw,want", MOE, ids=str)
def test_moe_refuses(lib, kw, want):
    assert _moe(lib, **kw) == want, lib.qmm_last_error()


def _append(lib, **kw):
    a = dict(q=A, qs=1024, k=A, ks=256, v=A, vs=256, T=3, Hq=8, Hkv=2, D=128, cos=A, sin=A, R=64, P=10, pos=A, slots=A, out=A,
             kc=A, vc=A, pages=4, page=16, fl=0)
    a.update(kw)
    return lib.qmm_kv_append(*a.values(), None)


APPEND = [(dict(T=-1), SHAPE), (dict(T=2**31 - 1), SHAPE), (dict(Hq=7), SHAPE), (dict(Hkv=0), SHAPE), (dict(D=96), SHAPE),
          (dict(R=40), SHAPE), (dict(R=144), SHAPE), (dict(R=-16), SHAPE), (dict(P=0), SHAPE), (dict(qs=1020), SHAPE),
          (dict(qs=1016), SHAPE), (dict(ks=128), SHAPE), (dict(vs=-256), SHAPE), (dict(pages=0), SHAPE), (dict(page=0), SHAPE),
          (dict(fl=2), FLAGS), (dict(q=None), NULL), (dict(cos=None), NULL), (dict(pos=None), NULL), (dict(slots=None), NULL),
          (dict(vc=None), NULL), (dict(out=MIS), ALIGN), (dict(v=MIS), ALIGN), (dict(kc=MIS), ALIGN), (dict(sin=MIS), ALIGN),
          (dict(slots=MIS), ALIGN)]


@pytest.mark.parametrize("kw,want", APPEND, ids=str)
def test_append_refuses(lib, kw, want):
    assert _append(lib, **kw) == want, lib.qmm_last_error()


def _attention(lib, **kw):
    a = dict(q=A, qs=1024, T=3, Hq=8, Hkv=2, D=128, kc=A, vc=A, pages=4, page=16, table=A, ts=4, kv=A, starts=A, B=2, max_q=2,
             max_kv=64, first=None, end=None, scale=0.1, cap=0.0, slopes=None, fl=0, out=A, ws=A, wsb=1 << 40)
    a.update(kw)
    return lib.qmm_attention(*a.values(), None)


ATTENTION = [(dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(max_q=-1), SHAPE), (dict(Hq=9), SHAPE),
             (dict(D=80), SHAPE), (dict(max_kv=65), SHAPE), (dict(max_kv=-1), SHAPE), (dict(ts=0), SHAPE),
             (dict(ts=2**30, page=2), SHAPE), (dict(qs=1000), SHAPE), (dict(scale=math.nan), SHAPE), (dict(cap=-1.0), SHAPE),
             (dict(cap=math.inf), SHAPE), (dict(fl=2), FLAGS), (dict(q=None), NULL), (dict(table=None), NULL),
             (dict(kv=None), NULL), (dict(starts=None), NULL), (dict(out=None), NULL), (dict(kc=None), NULL),
             (dict(q=MIS), ALIGN), (dict(out=MIS), ALIGN), (dict(first=A + 2), ALIGN), (dict(slopes=A + 1), ALIGN),
             (dict(pages=0), SHAPE), (dict(T=2**30), SHAPE)]


@pytest.mark.parametrize("kw,want", ATTENTION, ids=str)
def test_attention_refuses(lib, kw, want):
    assert _attention(lib, **kw) == want, lib.qmm_last_error()


def _logprobs(lib, **kw):
    a = dict(l=A, stride=100, M=3, V=100, t=A, top=2, fl=0, lp=A, en=A, tl=A, ti=A, ws=A, wsb=1 << 30)
    a.update(kw)
    return lib.qmm_logprobs(*a.values(), None)


LOGPROBS = [(dict(M=-1), SHAPE), (dict(V=0), SHAPE), (dict(V=2**31 - 1), SHAPE), (dict(top=33), SHAPE), (dict(top=-1), SHAPE),
            (dict(V=1, top=2, stride=1), SHAPE), (dict(stride=99), SHAPE), (dict(fl=1 | 16), FLAGS), (dict(fl=2), FLAGS),
            (dict(l=None), NULL), (dict(en=None), NULL), (dict(lp=None), NULL), (dict(t=None), NULL), (dict(ti=None), NULL),
            (dict(l=A + 1), ALIGN), (dict(l=A + 2, fl=16), ALIGN), (dict(t=MIS), ALIGN), (dict(tl=A + 2), ALIGN)]


@pytest.mark.parametrize("kw,want", LOGPROBS, ids=str)
def test_logprobs_refuses(lib, kw, want):
    assert _logprobs(lib, **kw) == want, lib.qmm_last_error()


def test_empty_calls_do_nothing(lib):
    assert _route(lib, T=0, x=None, ids=None) == 0
    assert _moe(lib, T=0, x=None) == 0
    assert _append(lib, T=0, q=None) == 0
    assert _attention(lib, T=0, q=None) == 0
    assert _attention(lib, B=0, q=None) == 0
    assert _logprobs(lib, M=0, l=None) == 0
    assert lib.qmm_last_error() == b""


def test_workspace_sizes(lib):
    assert lib.qmm_moe_workspace_bytes(0, 256, 128, 4, 2) == 0
    assert lib.qmm_moe_workspace_bytes(8, 250, 128, 4, 2) == 0
    assert lib.qmm_moe_workspace_bytes(8, 256, 128, 4, 2) >= 8 * 2 * 128 * 4
    assert lib.qmm_moe_workspace_bytes(64, 256, 128, 4, 2) > lib.qmm_moe_workspace_bytes(8, 256, 128, 4, 2)
    assert lib.qmm_attention_workspace_bytes(1, 1, 8, 2, 100, 1, 100) == 0
    assert lib.qmm_logprobs_workspace_bytes(1, 0, 0) == 0
    assert lib.qmm_logprobs_workspace_bytes(1, 10, 33) == 0


def test_binding_refuses():
    import torch
    import weight_only_group_amd as w
    h = torch.zeros((2, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_moe_route(h, h, 1)
    with pytest.raises(TypeError):
        w.qmm_moe_route(h.float(), h, 1)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_moe(h, h, h, (), (), 4, 32)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_kv_append(h.view(2, 1, 64), h.view(2, 1, 64), h.view(2, 1, 64), None, None, None, None, None, None)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_attention(h.view(2, 1, 64), h, h, h, h, h, 1, 1)
    with pytest.raises(ValueError, match="GPU"):
        w.qmm_logprobs(h)
    with pytest.raises(TypeError):
        w.qmm_logprobs(h.to(torch.int32))


# ---- pins of the oracle ------------------------------------------------------------

def test_pin_route():
    x = np.array([[1.0, 2.0], [0.0, 1.0]])
    r = np.array([[1.0, 0.0], [0.0, 1.0], [1.0, 0.5]])  # logits 1, 2, 2 and 0, 1, 0.5
    ids, wt, logits = lo.moe_route(x, r, 2, True)
    assert logits.tolist() == [[1, 2, 2], [0, 1, 0.5]]
    assert ids.tolist() == [[1, 2], [1, 2]]
    assert wt[0].tolist() == [0.5, 0.5]
    _, wt, _ = lo.moe_route(x, r, 2, False)
    assert wt[1, 0] == pytest.approx(math.e / (1 + math.e + math.exp(0.5)), rel=1e-14)


def test_pin_moe_by_hand():
    # One expert, H = I = 32, all codes 1 with zero 0 and scale 1: g = u = sum(x); y = w * 32 * silu(s) * s.
    words = np.full((1, 4, 64), 0x11111111, np.int32)
    one, nil = np.ones((1, 1, 64)), np.zeros((1, 1, 64))
    down = (np.full((1, 4, 32), 0x11111111, np.int32), None, nil[..., :32], one[..., :32])
    x = np.zeros((1, 32))
    x[0, 3] = 2.0
    y, bound = lo.moe(x, np.array([[0]]), np.array([[0.25]]), (words, None, nil, one), down, 4, -1, "fp16")
    want = 0.25 * 32 * 2 / (1 + math.exp(-2)) * 2
    assert np.allclose(y, want, rtol=1e-14) and (bound > 0).all() and (bound < 0.01 * want).all()
    y, _ = lo.moe(x, np.array([[-1]]), np.array([[0.25]]), (words, None, nil, one), down, 4, -1, "fp16")
    assert not y.any()


def test_pin_rotation_is_a_rotation():
    r = np.random.default_rng(0)
    x, angle = r.standard_normal(64), r.uniform(0, 6, 16)
    for adjacent in (True, False):
        y, _ = lo.rotate(x, np.cos(angle), np.sin(angle), adjacent)
        assert np.linalg.norm(y) == pytest.approx(np.linalg.norm(x), rel=1e-12)
        assert np.array_equal(y[32:], x[32:])
        back, _ = lo.rotate(y, np.cos(angle), -np.sin(angle), adjacent)
        assert np.allclose(back, x, atol=1e-14)
    quarter, _ = lo.rotate(np.arange(4.0), np.array([0.0, 0.0]), np.array([1.0, 1.0]), True)
    assert quarter.tolist() == [-1, 0, -3, 2]
    quarter, _ = lo.rotate(np.arange(4.0), np.array([0.0, 0.0]), np.array([1.0, 1.0]), False)
    assert quarter.tolist() == [-2, -3, 0, 1]


def _attn(**kw):
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((3, 2, 4)), r.standard_normal((3, 1, 4, 4)), r.standard_normal((3, 1, 4, 4))
    args = dict(q=q, k_cache=k, v_cache=v, table=np.array([[2, 0]]), kv_lens=[6], q_starts=[0, 3], scale=0.5)
    args.update(kw)
    return lo.attention(**args)[0], q, k, v


def test_pin_attention():
    out, q, k, v = _attn()
    keys, values = (np.concatenate([c[2, 0], c[0, 0]])[:6] for c in (k, v))
    e = [math.exp(0.5 * sum(q[1, 1, d] * keys[j, d] for d in range(4))) for j in range(5)]  # query 1 is at position 4
    want = [sum(e[j] * values[j, d] for j in range(5)) / sum(e) for d in range(4)]
    assert np.allclose(out[1, 1], want, rtol=1e-13)
    only, *_ = _attn(first=np.array([2, 2, 2]), end=np.array([3, 3, 3]))  # one key: its value
    assert np.allclose(only, values[2])
    none, *_ = _attn(first=np.array([3, 3, 3]), end=np.array([3, 0, -4]))
    assert not none.any()
    near, *_ = _attn(slopes=np.array([1e6, 1e6]))  # all weight on the query's own position
    assert np.allclose(near[:, 0], values[3:])
    flat, *_ = _attn(softcap=1e-9)  # all scores alike: the mean
    assert np.allclose(flat[2, 0], values.mean(axis=0))
    assert np.allclose(_attn(softcap=1e9)[0], out, rtol=1e-9)


def test_pin_logprobs():
    l = np.log(np.array([[1.0, 2.0, 4.0, 1.0], [1, 1, 1, 1]]))
    lp, en, top, ids = lo.logprobs(l, np.array([2, -1]), 3)
    assert lp[0] == pytest.approx(math.log(0.5)) and lp[1] == 0
    assert en[0] == pytest.approx(0.5 * math.log(2) + 0.25 * math.log(4) + 0.25 * math.log(8))
    assert en[1] == pytest.approx(math.log(4))
    assert ids.tolist() == [[2, 1, 0], [0, 1, 2]]
    assert np.allclose(np.exp(top[0]), [0.5, 0.25, 0.125])
    lp, en, top, ids = lo.logprobs(np.array([[0.0, -np.inf, np.nan]]), np.array([0]), 2)
    assert np.isnan([lp[0], en[0]]).all() and ids.tolist() == [[2, 0]]


@pytest.mark.parametrize("plant", ["softmax_over_all", "half_turn", "window_off_by_one", "scale_after_cap", "entropy_sign"])
def test_planted_mistakes_show(plant, monkeypatch):
    """A mistake planted in the oracle moves some pin."""
    pins = {"softmax_over_all": test_pin_route, "half_turn": test_pin_rotation_is_a_rotation,
            "window_off_by_one": test_pin_attention, "scale_after_cap": test_pin_attention, "entropy_sign": test_pin_logprobs}
    route, rotate, attention, logprobs = lo.moe_route, lo.rotate, lo.attention, lo.logprobs

    def off(first=None, **kw):
        return attention(first=None if first is None else np.asarray(first) + 1, **kw)

    def late(softcap=0.0, scale=1.0, **kw):
        return attention(softcap=softcap / scale if softcap else 0.0, scale=scale * 1.01, **kw)

    wrong = {"softmax_over_all": ("moe_route", lambda x, r, k, n: route(x, r, k, not n)),
             "half_turn": ("rotate", lambda x, c, s, a: rotate(x, c, s, not a)),
             "window_off_by_one": ("attention", off), "scale_after_cap": ("attention", late),
             "entropy_sign": ("logprobs", lambda *a: (logprobs(*a)[0], -logprobs(*a)[1], *logprobs(*a)[2:]))}[plant]
    monkeypatch.setattr(lo, *wrong)
    with pytest.raises(AssertionError):
        pins[plant]()
