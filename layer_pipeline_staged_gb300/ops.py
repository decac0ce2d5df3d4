"""The C ABI's operators over a caller-owned cache, contiguous or in pages, on torch tensors.

Argument marshalling only, in ``csrc/marshal.c`` (shapes, types, strides and devices are read from the
tensors; everything else is checked by the library): ``include/lps.h`` states what each operator
computes. Every call is enqueued on the current stream of its tensors' device and returns at once.
Lengths, offsets and positions are host integers (a list, a numpy array or a CPU tensor) for the contiguous cache, and
int32 tensors on the device for the pages, so that a captured call replays with what they hold then. A tensor that
does not fit is a ValueError, a refusal of the library an LpsError. The attention kernels bound every wait; one that
gives up leaves an invalid ``out`` (and ``key_weights``, for the rows that the call saw), which ``cache_ops_status`` says.
"""
from __future__ import annotations

import math

from . import _capi

__all__ = ["attention_prompt_packed", "attention_tree_verify", "kv_rows_append", "kv_rows_accept", "cache_ops_status",
           "rotary_frequencies", "rotary_rows", "rotary_append_paged", "attention_paged_decode", "kv_pages_evict",
           "logits_adjust"]

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
    _marshal.init(_capi.LpsError, torch, _tensors(torch))
    _m = _marshal
    return _m


def _tensors(torch):
    """The tensors' facts by torch's C++ interface, if they have been built for this torch; None: by its Python one."""
    try:
        from . import _tensors as t
    except ImportError:
        return None
    return t.api if torch.__version__.split("+")[0] == t.torch_version.split("+")[0] else None


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
    invalid (and the ``key_weights`` of what it saw). Calls on every stream of the device share the report, which the check clears."""
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.device(s.device):
        _capi.check(_capi.load().cache_ops_status(s.cuda_stream))


def rotary_frequencies(rot_dim, theta=10000.0, scaling=None, factor=1.0, original=None, slow=1.0, fast=4.0):
    """Radians a position of each of ``rot_dim / 2`` pairs, ``theta ** (-2 i / rot_dim)``: float64 on the CPU.

    ``scaling`` stretches them by ``factor`` >= 1 for longer contexts: "linear" divides all of them; "ntk" raises
    ``theta`` so that the last pair is divided and the first stays; "parts" divides the pairs that turn less than
    ``slow`` times over the ``original`` context, leaves those that turn more than ``fast`` times, and blends the
    others linearly in their turns (interpolation by parts; the attention's softening that goes with it is the
    ``magnitude`` of the calls, commonly ``0.1 * log(factor) + 1``)."""
    import torch

    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and at least 2")
    if not (theta > 0 and math.isfinite(theta) and factor >= 1 and math.isfinite(factor)):
        raise ValueError("theta must be positive and factor at least 1, both finite")
    if scaling == "ntk":
        if rot_dim < 4:
            raise ValueError("ntk scaling needs two pairs or more")
        theta = theta * factor ** (rot_dim / (rot_dim - 2))
    f = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    if scaling in (None, "ntk"):
        return f
    if scaling == "linear":
        return f / factor
    if scaling != "parts":
        raise ValueError('scaling must be None, "linear", "ntk" or "parts"')
    if original is None or not (original > 0 and fast > slow >= 0):
        raise ValueError("scaling by parts needs the original context, and fast > slow >= 0")
    keep = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0.0, 1.0)
    return f * (keep + (1.0 - keep) / factor)


def rotary_rows(q, k, positions, freqs, interleaved=False, magnitude=1.0, out=None):
    """Rotary positions on ``q`` [tokens, q heads, head_dim] and ``k`` [tokens, kv heads, head_dim].

    ``positions`` int32 [tokens]; ``freqs`` float64 [rot_dim / 2] on the device (``rotary_frequencies``; None: nothing
    turns): the first ``rot_dim`` elements of a head turn, as pairs (i, i + rot_dim / 2) or ``interleaved`` (2 i,
    2 i + 1), the others are copied; rot_dim is a multiple of 16. The negative positions turn back, which is also the
    gradient's way. Returns two new tensors, or ``out``, a pair of them, which may be (q, k) themselves."""
    q_out, k_out = (None, None) if out is None else out
    return (_m or _ready()).rows(q, k, positions, freqs, interleaved, magnitude, q_out, k_out)


def rotary_append_paged(q, k, v, offsets, lengths, table, k_pages, v_pages, freqs, positions=None, interleaved=False,
                        magnitude=1.0, key_weights=None, q_out=None):
    """``rotary_rows``, with the turned keys and the values ``v`` written to the cache's pages; returns the turned q.

    Pages [pages, kv heads, page rows, head_dim], page rows a multiple of 8; ``table`` int32 [sequences, pages of each].
    Sequence s has the tokens ``offsets[s]:offsets[s + 1]`` (int32 on the device; None: one token a sequence), the last
    of which goes to row ``lengths[s] - 1``: ``lengths`` count the rows after the call. ``positions`` None means the row.
    ``key_weights`` float32 [pages, kv heads, page rows] gets zeros for the new rows. A row outside the table or on a
    page that does not exist is not stored. Tokens outside the offsets are not used, and their rows of the result
    are not written. ``q_out`` may be q itself."""
    return (_m or _ready()).append_paged(q, k, v, offsets, lengths, table, k_pages, v_pages, freqs, positions, interleaved,
                                         magnitude, key_weights, q_out)


def attention_paged_decode(q, k_pages, v_pages, table, lengths, key_weights=None, decay=1.0, out=None, scale=0.0):
    """Attention of one token a sequence over its rows ``[0, lengths[b])`` in pages.

    ``q`` [batch, q heads, head_dim], pages and ``table`` as for ``rotary_append_paged``, ``lengths`` int32 [batch] with the
    new token's own row counted. A sequence of no rows (or of a length that its table has no room for) gives zeros, and
    rows on a page that does not exist are not seen. With ``key_weights`` float32 [pages, kv heads, page rows] every row's
    weight, summed over the kv head's query heads, is added to ``decay`` times what is there (0: replaces it); the weights of
    a page that two of the call's sequences share are undefined after it, and the call's workspace takes 4 bytes a query head
    and row that the table has room for.
    ``scale`` 0 means 1/sqrt(head_dim). ``cache_ops_status`` reports a kernel that gave up. ``out`` is not q."""
    return (_m or _ready()).decode_paged(q, k_pages, v_pages, table, lengths, out, scale, key_weights, decay)


def kv_pages_evict(k_pages, v_pages, key_weights, table, lengths, new_table, budget, recent=0):
    """Of every sequence the last ``recent`` rows and the heaviest others by ``key_weights``, ``budget`` in all and for
    each kv head its own, copied in order with their weights to rows 0, 1, .. of ``new_table``'s pages.

    Returns the new lengths, int32 [batch]: ``min(length, budget)``, or -1 for a sequence whose length or pages break the
    rules, of which nothing is copied. The old pages are only read and may be shared (whose weights
    ``attention_paged_decode`` does not keep apart); the new ones must be none of them. Equal weights: the lowest row stays. Positions were turned into the keys before: the next token keeps its own."""
    return (_m or _ready()).evict_paged(k_pages, v_pages, key_weights, table, lengths, new_table, budget, recent)


def logits_adjust(logits, tokens=None, lengths=None, prompt_lengths=None, repetition=None, frequency=None, presence=None,
                  bias_ids=None, bias=None, allowed=None, out=None):
    """Penalties, biases and a grammar's mask on ``logits`` [batch, vocabulary] (float32, bfloat16 or float16), in this order.

    ``tokens`` int32 [batch, history] with ``lengths`` int32 [batch]: a row's history, its output from ``prompt_lengths`` on
    (None: all of it). ``repetition``, ``frequency``, ``presence`` float32 [batch]: positive logits of tokens in the history
    are divided by the first and others multiplied by it; the second times the token's count in the output, and the third
    once, are subtracted. ``bias_ids`` int32 and ``bias`` float32 [batch, entries] are added (entries outside the vocabulary
    are not). ``allowed`` int32 [batch, (vocabulary + 31) / 32]: tokens whose bit is not set become -inf. Returns a new
    tensor, or ``out``, which may be ``logits``."""
    return (_m or _ready()).adjust(logits, tokens, lengths, prompt_lengths, repetition, frequency, presence, bias_ids, bias,
                                   allowed, out)
