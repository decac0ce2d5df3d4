"""The C ABI's operators over a caller-owned cache, on torch tensors.

Argument marshalling only (shapes, types, strides and devices are read from the
tensors; everything else is checked by the library): ``include/lps.h`` states
what each operator computes. Every call is enqueued on the current stream of
its tensors' device and returns at once. Lengths, offsets and positions are
host integers (a list, a numpy array or a CPU tensor).

A call's kernels take a few microseconds when the work is small, so the
marshalling is written for few Python operations: strides and host integers
are handed over as packed bytes, which ctypes passes as they are.
"""
from __future__ import annotations

import struct

import numpy as np

from . import _capi
from ._capi import check as _check

__all__ = ["attention_prompt_packed", "attention_tree_verify", "kv_rows_append", "kv_rows_accept"]

_S4, _S6, _S8 = (struct.Struct(f"{n}q").pack for n in (4, 6, 8))
_int32 = np.dtype(np.int32)
_torch = _types = _stream_of = _current = None


def _need_torch() -> None:
    """The parts of torch the calls use, looked up once (the package itself does not need torch)."""
    global _torch, _types, _stream_of, _current
    import torch
    _types = {torch.bfloat16: _capi.LPS_TYPE_BF16, torch.float16: _capi.LPS_TYPE_FP16}
    _stream_of, _current = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
    _torch = torch


def _host(x, n: int, what: str) -> bytes:
    """`n` host integers as packed int32."""
    a = x if type(x) is np.ndarray else np.asarray(x)
    if a.shape != (n,):
        raise ValueError(f"{what} must hold {n} values, not an array of shape {a.shape}")
    if a.dtype is not _int32 and a.dtype != _int32:
        if a.dtype.kind not in "iu" and n:
            raise ValueError(f"{what} must hold integers")
        if n and (a.min() < -2**31 or a.max() >= 2**31):
            raise ValueError(f"{what} must fit 32 bits")
        a = a.astype(np.int32)
    return a.tobytes()


def _alike(tensors) -> tuple:
    """(library type, device index) that all the tensors share."""
    if _torch is None:
        _need_torch()
    first = tensors[0]
    dtype, dev = first.dtype, first.get_device()
    kind = _types.get(dtype)
    if kind is None:
        raise ValueError(f"tensors must be bfloat16 or float16, not {dtype}")
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    grad = False
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != dev:
            raise ValueError("tensors must share one type and one device")
        grad = grad or t.requires_grad
    if grad and _torch.is_grad_enabled():
        raise ValueError("there is no backward pass: detach the tensors or call under torch.no_grad()")
    return kind, dev


def _strides3(t, n: int, heads: int, hd: int) -> tuple:
    """Token and head stride of a [n, heads, hd] tensor; an axis of one entry counts as dense."""
    a, b, c = t.stride()
    if c != 1:
        raise ValueError("the head dimension must be contiguous")
    if heads == 1:
        b = hd
    return (a if n > 1 else heads * hd), b


def _cache(c, what: str) -> None:
    if not c.is_contiguous():
        raise ValueError(f"{what} must be contiguous [batch, kv heads, max_ctx, head_dim]")


def _int_rows(t, dev: int, shape, what: str) -> None:
    if t.dtype is not _torch.int32 or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)} on the same device")


def _call(fn, dev: int, *args) -> None:
    """fn(*args, stream) with the tensors' device current, on its current stream."""
    here = _current()
    if here == dev:
        rc = fn(*args, _stream_of(dev))
    else:
        _torch.cuda.set_device(dev)
        try:
            rc = fn(*args, _stream_of(dev))
        finally:
            _torch.cuda.set_device(here)
    if rc < 0:
        _check(rc)


def attention_prompt_packed(q, k, v, offsets, out=None, scale: float = 0.0):
    """Causal attention of whole prompts packed one after another.

    ``q`` [tokens, q heads, head_dim], ``k`` and ``v`` [tokens, kv heads, head_dim] (column ranges of
    one fused projection are fine), ``offsets`` n + 1 host integers: sequence s holds the tokens
    ``offsets[s]:offsets[s + 1]``. Returns ``out`` like ``q`` (rows outside the offsets are not written).
    ``scale`` 0 means 1/sqrt(head_dim)."""
    shape, kshape = q.shape, k.shape
    if len(shape) != 3 or len(kshape) != 3:
        raise ValueError("q, k and v must be [tokens, heads, head_dim]")
    tokens, nq, hd = shape
    nkv = kshape[1]
    if kshape[0] != tokens or kshape[2] != hd or v.shape != kshape:
        raise ValueError("k and v must be [tokens, kv heads, head_dim] of q's tokens and head_dim")
    if out is None:
        kind, dev = _alike((q, k, v))
        out = _torch.empty(shape, dtype=q.dtype, device=q.device)
    else:
        kind, dev = _alike((q, k, v, out))
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    n = len(offsets) - 1
    if n < 0:
        raise ValueError("offsets must hold n + 1 values")
    off = _host(offsets, n + 1, "offsets")
    if offsets[n] > tokens:
        raise ValueError("offsets reach past the tokens")
    if n == 0 or tokens == 0:
        return out
    st = _S8(*_strides3(q, tokens, nq, hd), *_strides3(k, tokens, nkv, hd), *_strides3(v, tokens, nkv, hd),
             *_strides3(out, tokens, nq, hd))
    _call(_capi.load().attention_prompt_packed, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), kind, n,
          off, nq, nkv, hd, st, scale)
    return out


def attention_tree_verify(q, k_cache, v_cache, parents, pos, rows, out=None, scale: float = 0.0):
    """Attention of drafted trees over a cache; one drafted row is an ordinary decode step.

    ``q`` [batch, width, q heads, head_dim]; caches [batch, kv heads, max_ctx, head_dim], the drafts' own
    keys and values stored from row ``pos[b]`` on; ``parents`` int32 [batch, width] on the device (-1: the
    draft hangs from the last committed token); ``pos`` and ``rows`` host integers per sequence. Returns
    ``out`` like ``q``; its rows from ``rows[b]`` on are not written."""
    shape, cshape = q.shape, k_cache.shape
    if len(shape) != 4 or len(cshape) != 4:
        raise ValueError("q must be [batch, width, q heads, head_dim], the caches [batch, kv heads, max_ctx, head_dim]")
    batch, width, nq, hd = shape
    nkv, max_ctx = cshape[1], cshape[2]
    if cshape[0] != batch or cshape[3] != hd or v_cache.shape != cshape:
        raise ValueError("the caches must be [batch, kv heads, max_ctx, head_dim] of q's batch and head_dim")
    if out is None:
        kind, dev = _alike((q, k_cache, v_cache))
        out = _torch.empty(shape, dtype=q.dtype, device=q.device)
    else:
        kind, dev = _alike((q, k_cache, v_cache, out))
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    _cache(k_cache, "k_cache")
    _cache(v_cache, "v_cache")
    _int_rows(parents, dev, (batch, width), "parents")
    p, r = _host(pos, batch, "pos"), _host(rows, batch, "rows")
    st = []
    for t in (q, out):
        a, b, c, d = t.stride()
        if d != 1:
            raise ValueError("the head dimension must be contiguous")
        st += (a if batch > 1 else width * nq * hd), (b if width > 1 else nq * hd), (c if nq > 1 else hd)
    _call(_capi.load().attention_tree_verify, dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
          kind, batch, width, p, r, parents.data_ptr(), nq, nkv, hd, max_ctx, _S6(*st), scale)
    return out


def kv_rows_append(k, v, offsets, k_cache, v_cache, start) -> None:
    """Packed key and value rows [tokens, kv heads, head_dim] into the cache [sequences, kv heads, max_ctx,
    head_dim]: token i of sequence s (``offsets[s]:offsets[s + 1]``) goes to row ``start[s] + i``."""
    shape, cshape = k.shape, k_cache.shape
    if len(shape) != 3 or len(cshape) != 4:
        raise ValueError("k and v must be [tokens, kv heads, head_dim], the caches [sequences, kv heads, max_ctx, head_dim]")
    tokens, nkv, hd = shape
    n, max_ctx = cshape[0], cshape[2]
    if v.shape != shape or cshape[1] != nkv or cshape[3] != hd or v_cache.shape != cshape:
        raise ValueError("k and v, and the two caches, must agree in shape, kv heads and head_dim")
    _, dev = _alike((k, v, k_cache, v_cache))
    _cache(k_cache, "k_cache")
    _cache(v_cache, "v_cache")
    off, at = _host(offsets, n + 1, "offsets"), _host(start, n, "start")
    if offsets[n] > tokens:
        raise ValueError("offsets reach past the tokens")
    if tokens == 0:
        return
    st = _S4(*_strides3(k, tokens, nkv, hd), *_strides3(v, tokens, nkv, hd))
    _call(_capi.load().kv_rows_append, dev, k.data_ptr(), v.data_ptr(), n, off, k_cache.data_ptr(), v_cache.data_ptr(),
          at, nkv, hd, max_ctx, st)


def kv_rows_accept(k_cache, v_cache, pos, path, accepted) -> None:
    """The accepted path of drafted trees, moved in place: cache row ``pos[b] + path[b, i]`` to row
    ``pos[b] + i`` for i < ``accepted[b]``, in every layer. Caches [layers, batch, kv heads, max_ctx,
    head_dim] (or without the layer axis); ``path`` int32 [batch, width] ascending and ``accepted`` int32
    [batch] on the device, ``pos`` host integers. A sequence whose path breaks the rules is left as it was."""
    cshape = k_cache.shape
    if len(cshape) not in (4, 5) or v_cache.shape != cshape:
        raise ValueError("the caches must be [layers, batch, kv heads, max_ctx, head_dim], both alike")
    batch, nkv, max_ctx, hd = cshape[-4:]
    layers = cshape[0] if len(cshape) == 5 else 1
    _, dev = _alike((k_cache, v_cache))
    _cache(k_cache, "k_cache")
    _cache(v_cache, "v_cache")
    if len(path.shape) != 2:
        raise ValueError("path must be [batch, width]")
    width = path.shape[1]
    _int_rows(path, dev, (batch, width), "path")
    _int_rows(accepted, dev, (batch,), "accepted")
    _call(_capi.load().kv_rows_accept, dev, k_cache.data_ptr(), v_cache.data_ptr(), layers, batch, nkv, hd, max_ctx,
          _host(pos, batch, "pos"), width, path.data_ptr(), accepted.data_ptr())
