"""The C ABI's operators over a caller-owned cache, on torch tensors.

Argument marshalling only (shapes, types, strides and devices are read from the
tensors; everything else is checked by the library): ``include/lps.h`` states
what each operator computes. Every call is enqueued on the current stream of
its tensors' device and returns at once. Lengths, offsets and positions are
host integers (a list, a numpy array or a CPU tensor).
"""
from __future__ import annotations

import ctypes

import numpy as np

from . import _capi
from ._capi import check as _check

__all__ = ["attention_prompt_packed", "attention_tree_verify", "kv_rows_append", "kv_rows_accept"]

_I4, _I6, _I8 = (ctypes.c_int64 * n for n in (4, 6, 8))


def _host(x, n: int, what: str) -> np.ndarray:
    """`n` host integers as an int32 array."""
    a = np.asarray(x)
    if a.dtype != np.int32:
        if a.dtype.kind not in "iu" and a.size:
            raise ValueError(f"{what} must hold integers")
        if a.size and (a.min() < -2**31 or a.max() >= 2**31):
            raise ValueError(f"{what} must fit 32 bits")
        a = a.astype(np.int32)
    if a.shape != (n,):
        raise ValueError(f"{what} must hold {n} values, not an array of shape {a.shape}")
    return np.ascontiguousarray(a)


def _type(t) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return _capi.LPS_TYPE_BF16
    if t.dtype is torch.float16:
        return _capi.LPS_TYPE_FP16
    raise ValueError(f"tensors must be bfloat16 or float16, not {t.dtype}")


def _same(first, *others) -> None:
    import torch
    if not first.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    grad = torch.is_grad_enabled()
    if grad and first.requires_grad:
        raise ValueError("there is no backward pass: detach the tensors or call under torch.no_grad()")
    for t in others:
        if t.dtype is not first.dtype or t.device != first.device:
            raise ValueError("tensors must share one type and one device")
        if grad and t.requires_grad:
            raise ValueError("there is no backward pass: detach the tensors or call under torch.no_grad()")


def _strides(t, n_outer: int) -> list:
    """Element strides of the outer axes; an axis of one entry counts as dense."""
    st, shape = t.stride(), t.shape
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("the head dimension must be contiguous")
    dense, out = shape[-1], [0] * n_outer
    for i in range(n_outer - 1, -1, -1):
        out[i] = st[i] if shape[i] > 1 else dense
        dense *= shape[i]
    return out


def _cache(c, what: str) -> None:
    if not c.is_contiguous():
        raise ValueError(f"{what} must be contiguous [batch, kv heads, max_ctx, head_dim]")


def _int_rows(t, first, shape, what: str) -> None:
    import torch
    if t.dtype is not torch.int32 or t.device != first.device or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {shape} on the same device")


class _On:
    """The tensors' device as the current one, and its current stream."""

    def __init__(self, t):
        import torch
        self.index, self.torch = t.device.index, torch

    def __enter__(self):
        cuda = self.torch.cuda
        self.before = cuda.current_device()
        if self.before != self.index:
            cuda.set_device(self.index)
        return cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self.before != self.index:
            self.torch.cuda.set_device(self.before)


def attention_prompt_packed(q, k, v, offsets, out=None, scale: float = 0.0):
    """Causal attention of whole prompts packed one after another.

    ``q`` [tokens, q heads, head_dim], ``k`` and ``v`` [tokens, kv heads, head_dim] (column ranges of
    one fused projection are fine), ``offsets`` n + 1 host integers: sequence s holds the tokens
    ``offsets[s]:offsets[s + 1]``. Returns ``out`` like ``q`` (rows outside the offsets are not written).
    ``scale`` 0 means 1/sqrt(head_dim)."""
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    tokens, nq, hd = q.shape
    nkv = k.shape[1]
    if k.shape != (tokens, nkv, hd) or v.shape != k.shape:
        raise ValueError("k and v must be [tokens, kv heads, head_dim] of q's tokens and head_dim")
    kind = _type(q)
    if out is None:
        _same(q, k, v)
        out = q.new_empty((tokens, nq, hd))
    else:
        _same(q, k, v, out)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    n = len(offsets) - 1
    if n < 0:
        raise ValueError("offsets must hold n + 1 values")
    off = _host(offsets, n + 1, "offsets")
    if off[-1] > tokens:
        raise ValueError("offsets reach past the tokens")
    if n == 0 or tokens == 0:
        return out
    st = _I8(*_strides(q, 2), *_strides(k, 2), *_strides(v, 2), *_strides(out, 2))
    with _On(q) as stream:
        _check(_capi.load().attention_prompt_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), kind, n,
                                                    off.ctypes.data, nq, nkv, hd, st, scale, stream))
    return out


def attention_tree_verify(q, k_cache, v_cache, parents, pos, rows, out=None, scale: float = 0.0):
    """Attention of drafted trees over a cache; one drafted row is an ordinary decode step.

    ``q`` [batch, width, q heads, head_dim]; caches [batch, kv heads, max_ctx, head_dim], the drafts' own
    keys and values stored from row ``pos[b]`` on; ``parents`` int32 [batch, width] on the device (-1: the
    draft hangs from the last committed token); ``pos`` and ``rows`` host integers per sequence. Returns
    ``out`` like ``q``; its rows from ``rows[b]`` on are not written."""
    if q.dim() != 4 or k_cache.dim() != 4:
        raise ValueError("q must be [batch, width, q heads, head_dim], the caches [batch, kv heads, max_ctx, head_dim]")
    batch, width, nq, hd = q.shape
    _, nkv, max_ctx, _ = k_cache.shape
    if k_cache.shape != (batch, nkv, max_ctx, hd) or v_cache.shape != k_cache.shape:
        raise ValueError("the caches must be [batch, kv heads, max_ctx, head_dim] of q's batch and head_dim")
    kind = _type(q)
    if out is None:
        _same(q, k_cache, v_cache)
        out = q.new_empty((batch, width, nq, hd))
    else:
        _same(q, k_cache, v_cache, out)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    _cache(k_cache, "k_cache")
    _cache(v_cache, "v_cache")
    _int_rows(parents, q, (batch, width), "parents")
    p, r = _host(pos, batch, "pos"), _host(rows, batch, "rows")
    st = _I6(*_strides(q, 3), *_strides(out, 3))
    L = _capi.load()
    with _On(q) as stream:
        need = L.attention_tree_workspace_bytes(batch, width, p.ctypes.data, r.ctypes.data, nq, nkv, hd)
        ws = q.new_empty((need // q.element_size(),)) if need > 0 else None
        _check(L.attention_tree_verify(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(), kind,
                                       batch, width, p.ctypes.data, r.ctypes.data, parents.data_ptr(), nq, nkv, hd,
                                       max_ctx, st, scale, ws.data_ptr() if need > 0 else None, max(need, 0), stream))
    return out


def kv_rows_append(k, v, offsets, k_cache, v_cache, start) -> None:
    """Packed key and value rows [tokens, kv heads, head_dim] into the cache [sequences, kv heads, max_ctx,
    head_dim]: token i of sequence s (``offsets[s]:offsets[s + 1]``) goes to row ``start[s] + i``."""
    if k.dim() != 3 or k_cache.dim() != 4:
        raise ValueError("k and v must be [tokens, kv heads, head_dim], the caches [sequences, kv heads, max_ctx, head_dim]")
    tokens, nkv, hd = k.shape
    n, _, max_ctx, _ = k_cache.shape
    if v.shape != k.shape or k_cache.shape != (n, nkv, max_ctx, hd) or v_cache.shape != k_cache.shape:
        raise ValueError("k and v, and the two caches, must agree in shape, kv heads and head_dim")
    _type(k)
    _same(k, v, k_cache, v_cache)
    _cache(k_cache, "k_cache")
    _cache(v_cache, "v_cache")
    off, at = _host(offsets, n + 1, "offsets"), _host(start, n, "start")
    if off[-1] > tokens:
        raise ValueError("offsets reach past the tokens")
    if tokens == 0:
        return
    with _On(k) as stream:
        _check(_capi.load().kv_rows_append(k.data_ptr(), v.data_ptr(), n, off.ctypes.data, k_cache.data_ptr(),
                                           v_cache.data_ptr(), at.ctypes.data, nkv, hd, max_ctx,
                                           _I4(*_strides(k, 2), *_strides(v, 2)), stream))


def kv_rows_accept(k_cache, v_cache, pos, path, accepted) -> None:
    """The accepted path of drafted trees, moved in place: cache row ``pos[b] + path[b, i]`` to row
    ``pos[b] + i`` for i < ``accepted[b]``, in every layer. Caches [layers, batch, kv heads, max_ctx,
    head_dim] (or without the layer axis); ``path`` int32 [batch, width] ascending and ``accepted`` int32
    [batch] on the device, ``pos`` host integers. A sequence whose path breaks the rules is left as it was."""
    if k_cache.dim() not in (4, 5) or v_cache.shape != k_cache.shape:
        raise ValueError("the caches must be [layers, batch, kv heads, max_ctx, head_dim], both alike")
    batch, nkv, max_ctx, hd = k_cache.shape[-4:]
    layers = k_cache.shape[0] if k_cache.dim() == 5 else 1
    _type(k_cache)
    _same(k_cache, v_cache)
    _cache(k_cache, "k_cache")
    _cache(v_cache, "v_cache")
    if path.dim() != 2:
        raise ValueError("path must be [batch, width]")
    width = path.shape[1]
    _int_rows(path, k_cache, (batch, width), "path")
    _int_rows(accepted, k_cache, (batch,), "accepted")
    p = _host(pos, batch, "pos")
    with _On(k_cache) as stream:
        _check(_capi.load().kv_rows_accept(k_cache.data_ptr(), v_cache.data_ptr(), layers, batch, nkv, hd, max_ctx,
                                           p.ctypes.data, width, path.data_ptr(), accepted.data_ptr(), stream))
