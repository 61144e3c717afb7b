"""Python binding of the layer operators (include/qmm_layer.h): argument
marshalling over libqmm, in the manner of the products' binding.

* ``qmm_moe_route(x, router, top_k, renormalize=True)`` -> ``(ids, weights, logits)``
* ``qmm_moe(x, ids, weights, gate_up, down, bits, group_size, strips=False)`` -> y
* ``qmm_kv_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, adjacent=False)`` -> rotated q
* ``qmm_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts, max_q, max_kv, ...)`` -> out
* ``qmm_logprobs(logits, targets=None, top=0)`` -> ``(logprob, entropy, top_logprobs, top_ids)``

Work runs on the current stream of the tensors' device; results are new
tensors unless ``out`` arguments are given. The workspace is the decode
product's, one per device and stream (in a graph capture one of the graph's
own), unless one is passed; calls that share one must not overlap in time.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

import weight_only_group_amd as _qmm

QMM_BF16, QMM_STRIPS = 1, 2
QMM_RENORMALIZE, QMM_ADJACENT, QMM_FP32 = 4, 8, 16
MOE_MAX_TOKENS = 64

# Every symbol qmm_layer.h declares.
EXPORTS = (
    "qmm_moe_route_workspace_bytes", "qmm_moe_route", "qmm_moe_workspace_bytes", "qmm_moe", "qmm_kv_append",
    "qmm_attention_workspace_bytes", "qmm_attention", "qmm_logprobs_workspace_bytes", "qmm_logprobs",
)


class Experts(ctypes.Structure):
    """qmm_experts of the C ABI."""

    _fields_ = [("qweight", ctypes.c_void_p), ("qweight_lo", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


def declare(lib):
    P, I, L, SZ, U, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint, ctypes.c_float)
    E = ctypes.POINTER(Experts)
    for name, res, args in (
            ("qmm_moe_route_workspace_bytes", SZ, [I, I, I]),
            ("qmm_moe_route", I, [P, I, I, P, I, I, U, P, P, P, P, SZ, P]),
            ("qmm_moe_workspace_bytes", SZ, [I, I, I, I, I]),
            ("qmm_moe", I, [P, I, I, I, I, I, P, P, E, E, I, I, U, P, P, SZ, P]),
            ("qmm_kv_append", I, [P, L, P, L, P, L, I, I, I, I, P, P, I, I, P, P, P, P, P, I, I, U, P]),
            ("qmm_attention_workspace_bytes", SZ, [I, I, I, I, I, I, I]),
            ("qmm_attention", I, [P, L, I, I, I, I, P, P, I, I, P, I, P, P, I, I, I, P, P, F, F, P, U, P, P, SZ, P]),
            ("qmm_logprobs_workspace_bytes", SZ, [I, I, I]),
            ("qmm_logprobs", I, [P, L, I, I, P, I, U, P, P, P, P, P, SZ, P])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


def _array(t, name, dtype, shape, dev):
    """A contiguous tensor on `dev` of exactly this type and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.device == dev and t.is_contiguous():
            return t
    except AttributeError:  # no tensor: the checks below say so
        pass
    _qmm._gpu(t, name, dtype, ndim=len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev} (got {t.device})")
    return t


def _result(out, like, shape):
    """`out`, checked, or a new tensor of `like`'s type and device."""
    if out is None:
        return like.new_empty(shape)
    return _array(out, "out", like.dtype, shape, like.device)


@functools.lru_cache(maxsize=4096)
def _need(name, *shape):
    """A call's ..._workspace_bytes (a plan of the shape alone: asked once per shape and device)."""
    return getattr(_qmm.library(), name + "_workspace_bytes")(*shape[1:])


def _launch(name, dev, args, out=(), workspace=None, shape=None):
    """Calls the entry point on the device's current stream; with `shape`, a workspace goes before the stream."""
    here = torch._C._cuda_getDevice()
    if here != dev.index:
        with torch.cuda.device(dev):
            return _launch(name, dev, args, out, workspace, shape)
    stream = torch._C._cuda_getCurrentRawStream(here)
    if shape is not None:
        if workspace is not None:
            _qmm._given_workspace(workspace, dev)
        elif need := _need(name, here, *shape):
            if not torch.cuda.is_current_stream_capturing():
                workspace = _qmm._workspaces.get((here, stream))
            if workspace is None or workspace.numel() < need:
                workspace = _qmm.gemv_workspace(dev, need)
        if workspace is None:
            args += (None, 0, stream)
        else:
            args += (workspace.data_ptr(), workspace.numel() * workspace.element_size(), stream)
    else:
        args += (stream,)
    status = getattr(_qmm._lib or _qmm.library(), name)(*args)
    if status:
        _qmm._check(status, name)
    return out


def _sizes(**sizes):
    """Refuses sizes past 32 bits: they would reach the library cut to their low bits, as other sizes."""
    for name, n in sizes.items():
        if not -2**31 <= n < 2**31:
            raise ValueError(f"{name}={n} must be below 2^31")


def _p(t):
    return None if t is None else t.data_ptr()


def qmm_moe_route(x, router, top_k: int, renormalize: bool = True, workspace=None):
    """The experts of each token: ``ids`` (T, top_k) int32, largest logit first, their ``weights``
    (T, top_k) float32, and the ``logits`` (T, E) float32 = x @ router.T. ``router`` is (E, H)."""
    dt = _qmm._data_dtype(x, "x")
    _qmm._gpu(x, "x", dt)
    T, H = x.shape
    dev = x.device
    E = router.shape[0] if isinstance(router, torch.Tensor) and router.dim() else 0
    _array(router, "router", dt, (E, H), dev)
    k = max(0, top_k)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    logits = weights.new_empty((T, E))
    flags = (QMM_BF16 if dt == torch.bfloat16 else 0) | (QMM_RENORMALIZE if renormalize else 0)
    return _launch("qmm_moe_route", dev, (_p(x), T, H, _p(router), E, top_k, flags, _p(ids), _p(weights), _p(logits)),
                   (ids, weights, logits), workspace, (T, H, E))


def _experts(w, name, E, K, N, bits, group_size, dt, strips, dev):
    """(qweight, qweight_lo, zeros, scales) of E experts, checked, as the C structure."""
    qw, qlo, zeros, scales = w
    if bits in _qmm.BITS and (group_size == -1 or (group_size > 0 and K % group_size == 0)):
        shapes = _qmm.packed_shapes(K, N, bits)
        if strips:
            shapes = tuple(s and _qmm.strips_shape(s[0], N) for s in shapes)
        _array(qw, f"{name} qweight", torch.int32, (E, *shapes[0]), dev)
        if bits == 3:
            if qlo is None:
                raise ValueError(f"{name}: 3-bit weights need qweight_lo (the 1-bit plane)")
            _array(qlo, f"{name} qweight_lo", torch.int32, (E, *shapes[1]), dev)
        groups = 1 if group_size == -1 else K // group_size
        _array(zeros, f"{name} zeros", dt, (E, groups, N), dev)
        _array(scales, f"{name} scales", dt, (E, groups, N), dev)
    return Experts(*(None if t is None else t.data_ptr() for t in (qw, qlo if bits == 3 else None, zeros, scales)))


def qmm_moe(x, ids, weights, gate_up, down, bits: int, group_size: int, strips: bool = False, out=None, workspace=None):
    """y[t] = sum_j weights[t, j] * (silu(g) * u) @ dequantize(down[ids[t, j]]), (g, u) the halves of
    x[t] @ dequantize(gate_up[ids[t, j]]), for up to 64 tokens. ``gate_up`` and ``down`` are each
    ``(qweight, qweight_lo, zeros, scales)`` with a leading expert axis, the planes K-major or, with
    ``strips=True``, in the 16-column strips of qmm_to_strips."""
    dt = _qmm._data_dtype(x, "x")
    _qmm._gpu(x, "x", dt)
    T, H = x.shape
    dev = x.device
    k = ids.shape[1] if isinstance(ids, torch.Tensor) and ids.dim() == 2 else 0
    _array(ids, "ids", torch.int32, (T, k), dev)
    _array(weights, "weights", torch.float32, (T, k), dev)
    if down[2].dim() != 3 or gate_up[2].dim() != 3 or gate_up[2].shape[2] % 2:
        raise ValueError("zeros must be (E, G, 2 I) for gate_up and (E, G, H) for down")
    E, _, N = gate_up[2].shape
    I = N // 2
    gu = _experts(gate_up, "gate_up", E, H, N, bits, group_size, dt, strips, dev)
    dn = _experts(down, "down", E, I, H, bits, group_size, dt, strips, dev)
    y = _result(out, x, (T, H))
    return _launch("qmm_moe", dev, (_p(x), T, H, I, E, k, _p(ids), _p(weights), ctypes.byref(gu), ctypes.byref(dn), bits,
                                    group_size, _qmm._flags(dt, strips), _p(y)), y, workspace, (T, H, I, E, k))


def _heads(t, name, dt):
    """(T, heads, D) with dense heads; the token stride is free (a view of a product's rows).
    Returns T, heads, D and that stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (got {t.device})")
    if t.dtype is not dt:
        raise TypeError(f"{name} must be {dt} (got {t.dtype})")
    if t.dim() == 3:
        T, h, D = t.shape
        st, sh, sd = t.stride()
        if (sd == 1 and (h < 2 or sh == D)) or not T * h * D:
            return T, h, D, h * D if T < 2 else st  # one token's stride is never used; a view may report any
    raise ValueError(f"{name} must be (tokens, heads, D) with dense heads (got shape {tuple(t.shape)}, strides {t.stride()})")


def _cache(k_cache, v_cache, D, dt, dev):
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4 or k_cache.shape[3] != D:
        raise ValueError(f"k_cache must be a tensor (pages, Hkv, page_size, {D})")
    _array(k_cache, "k_cache", dt, k_cache.shape, dev)
    _array(v_cache, "v_cache", dt, k_cache.shape, dev)
    return k_cache.shape


def qmm_kv_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, adjacent: bool = False, out=None):
    """Rotates q (T, Hq, D) and k (T, Hkv, D) by the rows ``positions`` of cos and sin (P, R / 2), stores
    k and v at ``slots`` (int64; a token with a slot outside the cache is not stored) of the caches
    (pages, Hkv, page_size, D), and returns the rotated q. q, k and v may be views of one product's
    rows. ``adjacent``: pairs are (2i, 2i + 1), else (i, i + R / 2). cos None: no rotation."""
    dt = _qmm._data_dtype(q, "q")
    T, Hq, D, qs = _heads(q, "q", dt)
    Tk, Hkv, Dk, ks = _heads(k, "k", dt)
    Tv, Hv, Dv, vs = _heads(v, "v", dt)
    dev = q.device
    if not (T == Tk == Tv and Hkv == Hv and D == Dk == Dv):
        raise ValueError(f"k and v must be ({T}, Hkv, {D}) (got {tuple(k.shape)}, {tuple(v.shape)})")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be on {dev} (got {k.device}, {v.device})")
    pages, hkv, page_size, _ = _cache(k_cache, v_cache, D, dt, dev)
    if hkv != Hkv:
        raise ValueError(f"k_cache has {hkv} heads, k has {Hkv}")
    P = R = 0
    if cos is not None:
        P, half = cos.shape if isinstance(cos, torch.Tensor) and cos.dim() == 2 else (0, 0)
        _array(cos, "cos", torch.float32, (P, half), dev)
        _array(sin, "sin", torch.float32, (P, half), dev)
        _array(positions, "positions", torch.int32, (T,), dev)
        R = 2 * half
    _array(slots, "slots", torch.int64, (T,), dev)
    out = _result(out, q, (T, Hq, D))
    flags = (QMM_BF16 if dt == torch.bfloat16 else 0) | (QMM_ADJACENT if adjacent else 0)
    turn = (_p(cos), _p(sin), R, P, _p(positions)) if R else (None, None, 0, 0, None)
    return _launch("qmm_kv_append", dev, (_p(q), qs, _p(k), ks, _p(v), vs, T, Hq, Hkv, D, *turn, _p(slots), _p(out),
                                          _p(k_cache), _p(v_cache), pages, page_size, flags), out)


def qmm_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts, max_q: int, max_kv: int, scale=None,
                  softcap: float = 0.0, slopes=None, first=None, end=None, out=None, workspace=None):
    """Attention of the queries q (T, Hq, D) to the cached keys of their sequences. Sequence b has the
    rows q_starts[b] to q_starts[b + 1] and kv_lens[b] cached tokens, its new ones the last. A query at
    position p sees the keys from ``first`` (default 0) up to, without, ``end`` (default p + 1); one that
    sees none gets 0, and so does a token of no sequence. ``scale`` defaults to 1 / sqrt(D); ``softcap`` c > 0 takes c tanh(s / c) of the
    scores; ``slopes`` (Hq,) subtract slope * |p - key position|. max_q and max_kv bound the lengths."""
    dt = _qmm._data_dtype(q, "q")
    T, Hq, D, qs = _heads(q, "q", dt)
    dev = q.device
    pages, Hkv, page_size, _ = _cache(k_cache, v_cache, D, dt, dev)
    B, table_stride = page_table.shape if isinstance(page_table, torch.Tensor) and page_table.dim() == 2 else (0, 0)
    _array(page_table, "page_table", torch.int32, (B, table_stride), dev)
    _array(kv_lens, "kv_lens", torch.int32, (B,), dev)
    _array(q_starts, "q_starts", torch.int32, (B + 1,), dev)
    if not (0 <= max_q < 2**31 and 0 <= max_kv < 2**31 > table_stride):
        _sizes(max_q=max_q, max_kv=max_kv, table_stride=table_stride)
    if first is not None:
        _array(first, "first", torch.int32, (T,), dev)
    if end is not None:
        _array(end, "end", torch.int32, (T,), dev)
    if slopes is not None:
        _array(slopes, "slopes", torch.float32, (Hq,), dev)
    out = _result(out, q, (T, Hq, D))
    if B == 0 or max_q == 0:  # tokens of no sequence: the call writes nothing then
        out.zero_()
    args = (_p(q), qs, T, Hq, Hkv, D, _p(k_cache), _p(v_cache), pages, page_size, _p(page_table), table_stride,
            _p(kv_lens), _p(q_starts), B, max_q, max_kv, _p(first), _p(end), 1.0 / math.sqrt(D) if scale is None else scale,
            softcap, _p(slopes), QMM_BF16 if dt == torch.bfloat16 else 0, _p(out))
    return _launch("qmm_attention", dev, args, out, workspace, (B, T, Hq, Hkv, D, max_q, max_kv))


def qmm_logprobs(logits, targets=None, top: int = 0, workspace=None):
    """Per row of logits (M, V) (float16, bfloat16 or float32; rows may be strided): the log probability
    of ``targets`` (int64; None: not asked for), the entropy, and the ``top`` likeliest tokens' log
    probabilities and ids. All float32, ids int32. A negative target gives 0."""
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype not in (*_qmm.DTYPES, torch.float32):
        raise TypeError(f"logits must be float16, bfloat16 or float32 (got {logits.dtype})")
    if not logits.is_cuda:
        raise ValueError(f"logits must be on a GPU (got {logits.device})")
    if logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be (M, V) with dense rows (got shape {tuple(logits.shape)}, strides {logits.stride()})")
    M, V = logits.shape
    stride = V if M < 2 else logits.stride(0)
    dev = logits.device
    if targets is not None:
        _array(targets, "targets", torch.int64, (M,), dev)
    n = max(0, top)
    entropy = torch.empty(M, dtype=torch.float32, device=dev)
    logprob = None if targets is None else entropy.new_empty(M)
    top_logprobs = entropy.new_empty((M, n))
    top_ids = torch.empty((M, n), dtype=torch.int32, device=dev)
    flags = {torch.float16: 0, torch.bfloat16: QMM_BF16, torch.float32: QMM_FP32}[logits.dtype]
    return _launch("qmm_logprobs", dev, (_p(logits), stride, M, V, _p(targets), top, flags, _p(logprob), _p(entropy),
                                         _p(top_logprobs), _p(top_ids)),
                   (logprob, entropy, top_logprobs, top_ids), workspace, (M, V, top))
