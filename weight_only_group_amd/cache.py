"""Python binding of the 4-bit key/value cache and of the care of a cache's pages
(include/qmm_cache.h), in the manner of the layer operators' binding.

* ``kv4_page_bytes(page_size, D, group_size)``: bytes of one head of a page; a cache is uint8 (pages, Hkv, that)
* ``qmm_kv4_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, group_size, adjacent=False)`` -> rotated q
* ``qmm_kv4_gather(k_cache, v_cache, slots, D, group_size, dtype)`` -> ``(k, v)`` in 16 bits
* ``qmm_kv4_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts, max_q, max_kv, group_size, ...)`` -> out
* ``kv4_attention_plan_info(B, T, Hq, Hkv, D, max_q, max_kv, biased=False)`` -> the kernel and grid of such a call
* ``qmm_kv_copy_pages(caches, src, dst)``, ``qmm_kv_compact(caches, page_table, kv_lens, page_size)``: for
  caches of either kind, those of all layers at once

Streams, workspaces and results are as for the layer operators.
"""
from __future__ import annotations

import ctypes
import functools
import math

import torch

import weight_only_group_amd as _qmm

from .layer import QMM_ADJACENT, QMM_BF16, _array, _heads, _launch, _p, _result, _sizes

GROUPS = (32, 64, 128)
LARGEST = 16384  # keys and values are cut to this size
LARGEST_SCALE = 2728  # a group whose scale is beyond it stands for NaN

# Every symbol qmm_cache.h declares.
EXPORTS = (
    "qmm_kv4_page_bytes", "qmm_kv4_append", "qmm_kv4_gather", "qmm_kv4_attention_workspace_bytes", "qmm_kv4_attention",
    "qmm_kv4_attention_plan_info", "qmm_kv_copy_pages", "qmm_kv_compact_workspace_bytes", "qmm_kv_compact",
)


def declare(lib):
    P, I, L, SZ, U, F = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_uint, ctypes.c_float)
    for name, res, args in (
            ("qmm_kv4_page_bytes", SZ, [I, I, I]),
            ("qmm_kv4_append", I, [P, L, P, L, P, L, I, I, I, I, I, P, P, I, I, P, P, P, P, P, I, I, U, P]),
            ("qmm_kv4_gather", I, [P, P, I, I, I, I, I, P, I, U, P, P, P]),
            ("qmm_kv4_attention_workspace_bytes", SZ, [I, I, I, I, I, I, I]),
            ("qmm_kv4_attention", I, [P, L, I, I, I, I, I, P, P, I, I, P, I, P, P, I, I, I, P, P, F, F, P, U, P, P, SZ, P]),
            ("qmm_kv4_attention_plan_info", I, [I, I, I, I, I, I, I, I, P, I]),
            ("qmm_kv_copy_pages", I, [P, P, I, I, P, P, I, P]),
            ("qmm_kv_compact_workspace_bytes", SZ, [I]),
            ("qmm_kv_compact", I, [P, P, I, I, P, I, P, I, I, P, P, P, P, SZ, P])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


@functools.lru_cache(maxsize=256)
def kv4_page_bytes(page_size: int, D: int, group_size: int) -> int:
    """Bytes of one head of a page of a 4-bit cache, page_size (D / 2 + 4 D / group_size). ``page_size`` is a multiple
    of 8, D 64, 128 or 256, ``group_size`` (channels per scale) 32, 64 or 128 and at most D."""
    _sizes(page_size=page_size, D=D, group_size=group_size)
    n = _qmm.library().qmm_kv4_page_bytes(page_size, D, group_size)
    if not n:
        raise ValueError(f"page_size={page_size} must be a positive multiple of 8, D={D} 64, 128 or 256, "
                         f"group_size={group_size} 32, 64 or 128 and at most D")
    return n


def _kv4_cache(k_cache, v_cache, D, group_size, dev):
    """Pages, heads and page size of a 4-bit cache, checked."""
    block = kv4_page_bytes(8, D, group_size)
    shape = k_cache.shape if isinstance(k_cache, torch.Tensor) else ()
    if len(shape) != 3 or shape[2] % block or not shape[2]:
        raise ValueError(f"k_cache must be a tensor (pages, Hkv, kv4_page_bytes(page_size, {D}, {group_size}))")
    _array(k_cache, "k_cache", torch.uint8, shape, dev)
    _array(v_cache, "v_cache", torch.uint8, shape, dev)
    return shape[0], shape[1], shape[2] // block * 8


def qmm_kv4_append(q, k, v, cos, sin, positions, slots, k_cache, v_cache, group_size: int, adjacent: bool = False, out=None):
    """qmm_kv_append to a 4-bit cache: rotates q (T, Hq, D) and k (T, Hkv, D) by the rows ``positions`` of cos and sin
    (P, R / 2), quantises k and v per group of ``group_size`` channels into the ``slots`` (int64; a token with a slot
    outside the cache is not stored) of the caches (uint8, (pages, Hkv, kv4_page_bytes(...))), and returns the rotated q.
    Values are cut to +-16384. ``adjacent``: pairs are (2i, 2i + 1), else (i, i + R / 2). cos None: no rotation."""
    dt = _qmm._data_dtype(q, "q")
    T, Hq, D, qs = _heads(q, "q", dt)
    Tk, Hkv, Dk, ks = _heads(k, "k", dt)
    Tv, Hv, Dv, vs = _heads(v, "v", dt)
    dev = q.device
    if not (T == Tk == Tv and Hkv == Hv and D == Dk == Dv):
        raise ValueError(f"k and v must be ({T}, Hkv, {D}) (got {tuple(k.shape)}, {tuple(v.shape)})")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be on {dev} (got {k.device}, {v.device})")
    pages, hkv, page_size = _kv4_cache(k_cache, v_cache, D, group_size, dev)
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
    return _launch("qmm_kv4_append", dev, (_p(q), qs, _p(k), ks, _p(v), vs, T, Hq, Hkv, D, group_size, *turn, _p(slots),
                                           _p(out), _p(k_cache), _p(v_cache), pages, page_size, flags), out)


def qmm_kv4_gather(k_cache, v_cache, slots, D: int, group_size: int, dtype=torch.float16):
    """The keys and values (T, Hkv, D) of the ``slots`` (int64, (T,)) of a 4-bit cache in ``dtype`` (float16 or bfloat16).
    Slots may repeat; one outside the cache gives 0."""
    if dtype not in _qmm.DTYPES:
        raise TypeError(f"dtype must be float16 or bfloat16 (got {dtype})")
    _qmm._gpu(slots, "slots", torch.int64, ndim=1)
    dev, T = slots.device, slots.shape[0]
    pages, Hkv, page_size = _kv4_cache(k_cache, v_cache, D, group_size, dev)
    k = torch.empty((T, Hkv, D), dtype=dtype, device=dev)
    v = torch.empty_like(k)
    return _launch("qmm_kv4_gather", dev, (_p(k_cache), _p(v_cache), pages, Hkv, page_size, D, group_size, _p(slots), T,
                                           QMM_BF16 if dtype == torch.bfloat16 else 0, _p(k), _p(v)), (k, v))


def qmm_kv4_attention(q, k_cache, v_cache, page_table, kv_lens, q_starts, max_q: int, max_kv: int, group_size: int, scale=None,
                      softcap: float = 0.0, slopes=None, first=None, end=None, out=None, workspace=None):
    """qmm_attention to a 4-bit cache: attention of the queries q (T, Hq, D) to the cached keys of their sequences.
    Sequence b has the rows q_starts[b] to q_starts[b + 1] and kv_lens[b] cached tokens, its new ones the last. A query at
    position p sees the keys from ``first`` (default 0) up to, without, ``end`` (default p + 1); one that sees none gets
    0, and so does a token of no sequence. ``scale`` defaults to 1 / sqrt(D); ``softcap`` c > 0 takes c tanh(s / c) of
    the scores; ``slopes`` (Hq,) subtract slope * |p - key position|. max_q and max_kv bound the lengths."""
    dt = _qmm._data_dtype(q, "q")
    T, Hq, D, qs = _heads(q, "q", dt)
    dev = q.device
    pages, Hkv, page_size = _kv4_cache(k_cache, v_cache, D, group_size, dev)
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
    args = (_p(q), qs, T, Hq, Hkv, D, group_size, _p(k_cache), _p(v_cache), pages, page_size, _p(page_table), table_stride,
            _p(kv_lens), _p(q_starts), B, max_q, max_kv, _p(first), _p(end), 1.0 / math.sqrt(D) if scale is None else scale,
            softcap, _p(slopes), QMM_BF16 if dt == torch.bfloat16 else 0, _p(out))
    return _launch("qmm_kv4_attention", dev, args, out, workspace, (B, T, Hq, Hkv, D, max_q, max_kv))


KV4_KERNELS = ("tile", "pair", "parts", "blocks")
KV4_PLAN_FIELDS = ("kernel", "rows", "blocks", "resident", "parts", "cus")


def kv4_attention_plan_info(B: int, T: int, Hq: int, Hkv: int, D: int, max_q: int, max_kv: int, biased: bool = False) -> dict:
    """The launch qmm_kv4_attention makes for these sizes on the current device, with or without slopes (host only);
    ``kernel`` is one of KV4_KERNELS."""
    _sizes(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, max_q=max_q, max_kv=max_kv)
    info = (ctypes.c_int32 * len(KV4_PLAN_FIELDS))()
    _qmm._check(_qmm.library().qmm_kv4_attention_plan_info(B, T, Hq, Hkv, D, max_q, max_kv, biased, ctypes.addressof(info), len(info)),
                "qmm_kv4_attention_plan_info")
    return dict(zip(KV4_PLAN_FIELDS, (KV4_KERNELS[info[0]], *info[1:])))


def _pools(caches):
    """Pointers, bytes per page, count, pages and device of caches (each contiguous, pages first), checked."""
    if isinstance(caches, torch.Tensor) or not len(caches):
        raise ValueError("caches must be a sequence of tensors, one at least")
    try:  # of many caches the checks take longer than the copies: the fewest calls for those that are right
        first = caches[0]
        pages, index = first.size(0), first.get_device()
        bad = index < 0 or any([t.get_device() != index or t.dim() < 2 or t.size(0) != pages or not t.is_contiguous() for t in caches])
        sizes = [] if bad else [t.nbytes // pages for t in caches]
        bad = bad or 0 in sizes
    except (AttributeError, IndexError, ZeroDivisionError, RuntimeError):
        bad = True
    if bad:
        _refuse_pools(caches)
    n = len(sizes)
    _sizes(pages=pages)
    return (ctypes.c_void_p * n)(*[t.data_ptr() for t in caches]), (ctypes.c_int64 * n)(*sizes), n, pages, first.device


def _refuse_pools(caches):
    """The error of caches that _pools finds wrong."""
    for i, t in enumerate(caches):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"caches[{i}] must be a torch.Tensor")
        if not t.is_cuda:
            raise ValueError(f"caches[{i}] must be on a GPU (got {t.device})")
        if t.device != caches[0].device:
            raise ValueError(f"caches[{i}] must be on {caches[0].device} (got {t.device})")
        if t.dim() < 2 or t.shape[0] != caches[0].shape[0] or not t.numel():
            raise ValueError(f"caches[{i}] must have the first one's pages and more dimensions (got shape {tuple(t.shape)})")
        if not t.is_contiguous():
            raise ValueError(f"caches[{i}] must be contiguous")
    raise ValueError("caches must be tensors in memory of their own")


def qmm_kv_copy_pages(caches, src, dst):
    """Page dst[i] of every cache becomes its page src[i] (int32, (n,)). ``caches``: any number of them, (pages, ...)
    contiguous and of any type. A pair with an index outside the cache is left out. A page may be copied many times; none
    may be in ``dst`` twice, nor in ``dst`` and, of another pair, in ``src``.

    A fork of a sequence: its table's row is copied, and its last page, which both would go on to write, copied to a
    page of the new one's own."""
    pointers, sizes, n_caches, pages, dev = _pools(caches)
    n = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() == 1 else 0
    _array(src, "src", torch.int32, (n,), dev)
    _array(dst, "dst", torch.int32, (n,), dev)
    _sizes(n=n)
    _launch("qmm_kv_copy_pages", dev, (pointers, sizes, n_caches, pages, _p(src), _p(dst), n))


def qmm_kv_compact(caches, page_table, kv_lens, page_size: int, workspace=None):
    """Packs the pages in use (page_table[b, i], i < ceil(kv_lens[b] / page_size)) of all ``caches`` into the lowest ones.
    Returns the page table with them renamed, ``moved_to`` (pages,) int32, the place of each page now (-1: it was free),
    and ``live`` (1,) int32, their number: the pages from there on are free. Pages in use below ``live`` stay."""
    _sizes(page_size=page_size)
    pointers, sizes, n_caches, pages, dev = _pools(caches)
    B, table_stride = page_table.shape if isinstance(page_table, torch.Tensor) and page_table.dim() == 2 else (0, 0)
    _array(page_table, "page_table", torch.int32, (B, table_stride), dev)
    _array(kv_lens, "kv_lens", torch.int32, (B,), dev)
    table = torch.empty_like(page_table)
    moved_to = page_table.new_empty(pages)
    live = page_table.new_empty(1)
    return _launch("qmm_kv_compact", dev, (pointers, sizes, n_caches, pages, _p(page_table), table_stride, _p(kv_lens), B,
                                           page_size, _p(table), _p(moved_to), _p(live)), (table, moved_to, live), workspace,
                   (pages,))
