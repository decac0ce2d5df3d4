"""The C ABI's operators over a caller-owned cache, on torch tensors.

Argument marshalling only, in ``csrc/marshal.c`` (shapes, types, strides and devices are read from the
tensors; everything else is checked by the library): ``include/lps.h`` states what each operator
computes. Every call is enqueued on the current stream of its tensors' device and returns at once.
Lengths, offsets and positions are host integers (a list, a numpy array or a CPU tensor). A tensor that
does not fit is a ValueError, a refusal of the library an LpsError. The attention kernels bound every wait; one that
gives up leaves an invalid ``out``, which ``cache_ops_status`` says.
"""
from __future__ import annotations

from . import _capi

__all__ = ["attention_prompt_packed", "attention_tree_verify", "kv_rows_append", "kv_rows_accept", "cache_ops_status"]

_m = None


def _ready():
    """The marshalling module, with the library loaded and torch known to it (the package itself needs no torch)."""
    global _m
    _capi.load()
    import torch

    try:
        from . import _marshal
    except ImportError as e:
        raise RuntimeError("the torch wrappers' marshalling is missing for this Python: build it first "
                           "(python -m layer_pipeline_staged_gb300.build, which needs Python.h)") from e
    _marshal.init(_capi.LpsError, torch)
    _m = _marshal
    return _m


def attention_prompt_packed(q, k, v, offsets, out=None, scale=0.0):
    """Causal attention of whole prompts packed one after another.

    ``q`` [tokens, q heads, head_dim], ``k`` and ``v`` [tokens, kv heads, head_dim] (column ranges of
    one fused projection are fine), ``offsets`` n + 1 host integers: sequence s holds the tokens
    ``offsets[s]:offsets[s + 1]``. Returns ``out`` like ``q`` (rows outside the offsets are not written).
    ``scale`` 0 means 1/sqrt(head_dim). ``cache_ops_status`` reports a kernel that gave up."""
    return (_m or _ready()).prompt(q, k, v, offsets, out, scale)


def attention_tree_verify(q, k_cache, v_cache, parents, pos, rows, out=None, scale=0.0):
    """Attention of drafted trees over a cache; one drafted row is an ordinary decode step.

    ``q`` [batch, width, q heads, head_dim]; caches [batch, kv heads, max_ctx, head_dim], the drafts' own
    keys and values stored from row ``pos[b]`` on; ``parents`` int32 [batch, width] on the device (-1: the
    draft hangs from the last committed token); ``pos`` and ``rows`` host integers per sequence. Returns
    ``out`` like ``q``; its rows from ``rows[b]`` on are not written. ``cache_ops_status`` reports a kernel
    that gave up."""
    return (_m or _ready()).tree(q, k_cache, v_cache, parents, pos, rows, out, scale)


def kv_rows_append(k, v, offsets, k_cache, v_cache, start) -> None:
    """Packed key and value rows [tokens, kv heads, head_dim] into the cache [sequences, kv heads, max_ctx,
    head_dim]: token i of sequence s (``offsets[s]:offsets[s + 1]``) goes to row ``start[s] + i``."""
    (_m or _ready()).append(k, v, offsets, k_cache, v_cache, start)


def kv_rows_accept(k_cache, v_cache, pos, path, accepted) -> None:
    """The accepted path of drafted trees, moved in place: cache row ``pos[b] + path[b, i]`` to row
    ``pos[b] + i`` for i < ``accepted[b]``, in every layer. Caches [layers, batch, kv heads, max_ctx,
    head_dim] (or without the layer axis); ``path`` int32 [batch, width] ascending and ``accepted`` int32
    [batch] on the device, ``pos`` host integers. A sequence whose path breaks the rules is left as it was."""
    (_m or _ready()).accept(k_cache, v_cache, pos, path, accepted)


def cache_ops_status(stream=None) -> None:
    """Wait for ``stream`` (a ``torch.cuda.Stream``; None: the current one) and raise LpsError when a wait inside
    an attention kernel has given up on its device since the last check: at least one call's ``out`` is then
    invalid. Calls on every stream of the device share the report, which the check clears."""
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _capi.check(_capi.load().cache_ops_status(s.cuda_stream))
