"""Cases for measuring the operators of a decode step over a paged key/value cache.

Pages ``[pages][kv heads][page rows][head_dim]``; a sequence's table names its pages in order, and row j of the
sequence is row ``j % page rows`` of page ``table[j // page rows]``. Lengths, tables and positions lie on the device,
so that one captured step serves every later one. Four operators that follow each other:

- ``rotary``: rotary positions on queries and keys (half or interleaved pairs, all or the first part of the head,
  frequencies stretched for long contexts), and ``append``, the same with the rotated keys and the values written to
  their pages;
- ``attend``: attention of one new token a sequence over its pages, with the weight that each cached key got where the
  cache is to be thinned out;
- ``evict``: the most attended rows and the latest ones copied together to new pages;
- ``logits``: penalties for repeated tokens, biases and a grammar's mask on the logits.

With ``own`` false ``run`` computes them in elementary torch operations, in 32 bits (angles in 64), rounded once at the
end; with ``own`` true it calls this package.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEVICE = "cuda"


# ---- cases ----------------------------------------------------------------------------------------

def _rotary(name, tokens, first, nq, nkv, hd, rot, interleaved, stretch, dtype="bf16"):
    return {"name": name, "op": "rotary", "tokens": tokens, "first": first, "nq": nq, "nkv": nkv, "hd": hd, "rot": rot,
            "interleaved": interleaved, "stretch": stretch, "dtype": dtype}


def _append(name, counts, lens, page, nq, nkv, hd, rot, interleaved, stretch, dtype="bf16"):
    return {"name": name, "op": "append", "counts": counts, "lens": lens, "page": page, "nq": nq, "nkv": nkv, "hd": hd,
            "rot": rot, "interleaved": interleaved, "stretch": stretch, "dtype": dtype}


def _attend(name, lens, page, nq, nkv, hd, weights=False, dtype="bf16"):
    return {"name": name, "op": "attend", "lens": lens, "page": page, "nq": nq, "nkv": nkv, "hd": hd,
            "weights": weights, "dtype": dtype}


def _evict(name, lens, budget, recent, page, nkv, hd, dtype="bf16"):
    return {"name": name, "op": "evict", "lens": lens, "budget": budget, "recent": recent, "page": page, "nkv": nkv,
            "hd": hd, "dtype": dtype}


def _logits(name, batch, vocab, history, biases, mask, dtype="fp32"):
    return {"name": name, "op": "logits", "batch": batch, "vocab": vocab, "history": history, "biases": biases,
            "mask": mask, "dtype": dtype}


# a serving batch of 32: an empty slot, short chats and long ones
_B32 = "0,1,17,64,65,8192,4000,777,2500,8100,129,1024,5000,6001,333,16,7000,3999,48,2222,900,128,512,7777,1,4500,640,95,6400,2047,1500,8000"


def listed():
    return [
        # one decode step's token of the 1B decoder, rotated and stored: launch latency
        _append("append_one", "1", "1000", 16, 32, 8, 64, 64, False, 1.0),
        # two long prompts of the 8B decoder, stretched to four times its context, stored in pages
        _append("append_prompts", "8184,4001", "8184,4513", 16, 32, 8, 128, 128, False, 4.0),
        # a packed prompt's queries and keys, interleaved pairs in the first half of each head, in fp16
        _rotary("rotary_part", 4096, 100000, 48, 12, 128, 64, True, 1.0, "fp16"),
        # one sequence of the 1B decoder near its context: latency, and the split over a short length
        _attend("attend_one", "1000", 16, 32, 8, 64),
        # a serving batch of the 8B decoder, lengths of every kind
        _attend("attend_b32", _B32, 16, 32, 8, 128),
        # the same with each key's weight written down for a later eviction, in fp16 and larger pages
        _attend("attend_weights", "8192,4000,777,8100,1,6001,3333,5000", 64, 32, 8, 128, True, "fp16"),
        # 24 long contexts of the zero-padded decoder's heads: the largest
        _attend("attend_long", "32700,131,20011,32001,9,26000,30500,12345,32768,1000,27000,31999,"
                               "15000,32000,8000,30001,25555,32700,4097,22222,29000,31000,18000,32500", 32, 48, 12, 128),
        # one short cache halved
        _evict("evict_one", "1000", 512, 64, 16, 8, 64),
        # eight caches of very different lengths brought to 4096 rows
        _evict("evict_b8", "8192,4096,8100,6001,777,4097,7000,8191", 4096, 256, 16, 8, 128),
        # one row of the 1B decoder's logits, a short history: latency
        _logits("logits_one", 1, 32000, 200, 8, True),
        # 64 rows of the 8B decoder's logits with long histories
        _logits("logits_b64", 64, 128256, 8192, 64, True),
        # odd vocabulary in bf16, no grammar, many rows
        _logits("logits_odd", 100, 65537, 1000, 0, False, "bf16"),
    ]


_HEADS = ((4, 2, 64), (32, 8, 64), (32, 8, 128), (48, 12, 128), (32, 32, 64), (8, 1, 128), (12, 4, 128), (28, 4, 128),
          (16, 1, 64))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(values):
    return ",".join(map(str, values))


def draw(rng):
    op = rng.choice(("append", "append", "rotary", "attend", "attend", "attend", "evict", "logits", "logits"))
    nq, nkv, hd = rng.choice(_HEADS)
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    page = rng.choice((8, 16, 16, 24, 32, 64, 128))
    rot = rng.choice((hd, hd, hd // 2, hd // 4))
    inter, stretch = rng.choice((False, True)), rng.choice((1.0, 1.0, 2.0, 4.0, 8.0))
    if op == "rotary":
        c = _rotary("", _log(rng, 1, 8000), _log(rng, 1, 120000), nq, nkv, hd, rot, inter, stretch, dtype)
    elif op == "append":
        n = rng.choice((1, rng.randint(1, 16), rng.randint(1, 64)))
        if rng.random() < 0.5:
            counts = [1] * n
        else:
            longest = _log(rng, 1, max(1, 8000 // n))
            counts = [longest] + [rng.randint(0, longest) for _ in range(n - 1)]
        lens = [c + rng.choice((0, _log(rng, 1, 4000))) for c in counts]
        c = _append("", _text(counts), _text(lens), page, nq, nkv, hd, rot, inter, stretch, dtype)
    elif op == "attend":
        n = rng.choice((1, rng.randint(1, 8), rng.randint(1, 24), rng.randint(1, 64)))
        longest = _log(rng, 1, max(1, 24 * 32000 * 12 // (max(nkv, 12) * max(n, 24))))
        lens = [longest] + [rng.choice((0, 1, rng.randint(0, longest), rng.randint(0, longest), longest)) for _ in range(n - 1)]
        rng.shuffle(lens)
        c = _attend("", _text(lens), page, nq, nkv, hd, rng.random() < 0.4, dtype)
    elif op == "evict":
        n = rng.choice((1, rng.randint(1, 8)))
        longest = _log(rng, 1, 8192)
        lens = [longest] + [rng.randint(0, longest) for _ in range(n - 1)]
        budget = rng.randint(1, min(longest, 4096))
        c = _evict("", _text(lens), budget, rng.randint(0, budget), page, min(nkv, 8), hd, dtype)
    else:
        vocab, history, biases = _log(rng, 500, 128256), rng.choice((0, _log(rng, 1, 8192))), rng.choice((0, rng.randint(1, 100)))
        c = _logits("", _log(rng, 1, min(128, 64 * 128256 // vocab)), vocab, history, biases,
                    rng.random() < 0.6 or not history + biases, rng.choice(("fp32", "fp32", "bf16", "fp16")))
    del c["name"]
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def work(case):
    op, size = case["op"], 4 if case["dtype"] == "fp32" else 2
    if op == "rotary":
        n = case["tokens"]
        return {"bytes": 2 * n * (case["nq"] + case["nkv"]) * case["hd"] * size + 4 * n,
                "flops": 3 * n * (case["nq"] + case["nkv"]) * case["rot"]}
    if op == "append":
        n = sum(_ints(case["counts"]))
        return {"bytes": 2 * n * (case["nq"] + 2 * case["nkv"]) * case["hd"] * size + 4 * n,
                "flops": 3 * n * (case["nq"] + case["nkv"]) * case["rot"]}
    if op == "attend":
        lens, nq, nkv, hd = _ints(case["lens"]), case["nq"], case["nkv"], case["hd"]
        tables = 4 * sum(-(-n // case["page"]) for n in lens)
        return {"bytes": sum(lens) * nkv * (2 * hd * size + 4 * case["weights"]) + 2 * len(lens) * nq * hd * size + tables,
                "flops": 4 * hd * nq * sum(lens)}
    if op == "evict":
        lens, row = _ints(case["lens"]), 2 * case["hd"] * size + 4
        kept = sum(min(n, case["budget"]) for n in lens)
        return {"bytes": case["nkv"] * (4 * sum(lens) + (2 * row - 4) * kept), "flops": 0}
    n = case["batch"] * case["vocab"]
    return {"bytes": 2 * n * size + case["mask"] * n // 8 + case["batch"] * (4 * case["history"] + 8 * case["biases"]),
            "flops": 4 * n}


# ---- inputs ---------------------------------------------------------------------------------------

THETA, ORIGINAL, SLOW, FAST = 500000.0, 8192, 1.0, 4.0  # the frequencies' base; the context they were learnt on


def _frequencies(rot, stretch):
    """Radians a position of each pair. Stretched by parts: pairs that turn less than SLOW times over the learnt
    context turn `stretch` times slower, those that turn more than FAST times stay, the others lie between."""
    f = THETA ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    keep = np.clip((ORIGINAL * f / (2 * math.pi) - SLOW) / (FAST - SLOW), 0.0, 1.0)
    return f * (keep + (1.0 - keep) / stretch)


def _magnitude(stretch):
    return 1.0 if stretch <= 1.0 else 0.1 * math.log(stretch) + 1.0


def _table(host, lens, page, extra=0):
    """(table, pages): each sequence's pages at places of their own, in no order; -1 where it has none."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + extra + 1
    table = np.full((len(lens), max(max(need), 1)), -1, np.int32)
    free, at = host.permutation(pages).astype(np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = free[at:at + n]
        at += n
    return table, pages, free[at:]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    host = np.random.default_rng(int(seed))
    op, dt = case["op"], _DTYPES[case["dtype"]]
    s = {"op": op}

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=dtype)

    def put(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(DEVICE)

    if op in ("rotary", "append"):
        # q, k and v are column ranges of one fused projection
        nq, nkv, hd = case["nq"], case["nkv"], case["hd"]
        counts = [case["tokens"]] if op == "rotary" else _ints(case["counts"])
        n = sum(counts)
        fused = normal(n, (nq + 2 * nkv) * hd)
        s["q"] = fused[:, : nq * hd].view(n, nq, hd)
        s["k"] = fused[:, nq * hd: (nq + nkv) * hd].view(n, nkv, hd)
        s["v"] = fused[:, (nq + nkv) * hd:].view(n, nkv, hd)
        s.update(freqs=put(_frequencies(case["rot"], case["stretch"])), interleaved=case["interleaved"],
                 magnitude=_magnitude(case["stretch"]))
    if op == "rotary":
        s["positions"] = put(np.arange(case["first"], case["first"] + case["tokens"], dtype=np.int32))
    elif op == "append":
        # rows evicted earlier leave positions ahead of the cache's rows
        lens = np.array(_ints(case["lens"]), np.int32)
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        ahead = host.integers(0, 50000, size=len(lens))
        positions = np.concatenate([np.arange(c, dtype=np.int64) + int(l) - c + a for c, l, a in zip(counts, lens, ahead)])
        table, pages, _ = _table(host, lens.tolist(), case["page"])
        s.update(positions=put(positions.astype(np.int32)), offsets=put(offsets), lengths=put(lens), table=put(table))
        s["kp"], s["vp"] = (normal(pages, nkv, case["page"], hd) for _ in range(2))
    elif op in ("attend", "evict"):
        lens, hd, nkv, page = _ints(case["lens"]), case["hd"], case["nkv"], case["page"]
        new = [min(n, case["budget"]) for n in lens] if op == "evict" else []
        table, pages, free = _table(host, lens, page, sum(-(-n // page) for n in new))
        s.update(table=put(table), lengths=put(np.array(lens, np.int32)))
        s["kp"], s["vp"] = (normal(pages, nkv, page, hd) for _ in range(2))
        if op == "attend":
            s["q"] = normal(len(lens), case["nq"], hd)
            if case["weights"]:
                s["weights"] = torch.zeros(pages, nkv, page, device=DEVICE)
        else:
            # accumulated weights: a few rows hold most, many none at all
            heavy = normal(pages, nkv, page, dtype=torch.float32)
            s["weights"] = torch.where(heavy > -0.5, (2.5 * heavy).exp(), torch.zeros_like(heavy))
            fresh = np.full((len(lens), -(-case["budget"] // page)), -1, np.int32)
            at = 0
            for b, n in enumerate(new):
                m = -(-n // page)
                fresh[b, :m] = free[at:at + m]
                at += m
            s.update(fresh=put(fresh), budget=case["budget"], recent=case["recent"])
    else:
        batch, vocab, width = case["batch"], case["vocab"], case["history"]
        s["logits"] = (3.0 * normal(batch, vocab, dtype=torch.float32)).to(dt)
        if width:
            # a text's tokens: a few come again and again
            tokens = np.minimum(host.zipf(1.3, size=(batch, width)), vocab) - 1
            lengths = host.integers(width // 2, width + 1, size=batch)
            s["tokens"] = put(((tokens * 7919) % vocab).astype(np.int32))
            s["lengths"] = put(lengths.astype(np.int32))
            s["prompts"] = put((lengths * host.uniform(0, 1, size=batch)).astype(np.int32))
            for name, lo, hi in (("repetition", 1.0, 1.5), ("frequency", 0.0, 0.5), ("presence", -0.5, 1.0)):
                s[name] = put(host.uniform(lo, hi, size=batch).astype(np.float32))
        if case["biases"]:
            ids = np.stack([host.choice(vocab, size=case["biases"], replace=False) for _ in range(batch)])
            s["bias_ids"] = put(ids.astype(np.int32))
            s["bias"] = put(host.normal(0, 4, size=ids.shape).astype(np.float32))
        if case["mask"]:
            s["allowed"] = put(host.integers(-2 ** 31, 2 ** 31, size=(batch, -(-vocab // 32)), dtype=np.int64).astype(np.int32))
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    if own:
        import layer_pipeline_staged_gb300 as lps

        if s["op"] == "rotary":
            return lps.rotary_rows(s["q"], s["k"], s["positions"], s["freqs"], interleaved=s["interleaved"],
                                   magnitude=s["magnitude"])
        if s["op"] == "append":
            q = lps.rotary_append_paged(s["q"], s["k"], s["v"], s["offsets"], s["lengths"], s["table"], s["kp"], s["vp"],
                                        s["freqs"], positions=s["positions"], interleaved=s["interleaved"],
                                        magnitude=s["magnitude"])
            return q, s["kp"], s["vp"]
        if s["op"] == "attend":
            if "weights" in s:
                # the weights of this step alone
                return lps.attention_paged_decode(s["q"], s["kp"], s["vp"], s["table"], s["lengths"],
                                                  key_weights=s["weights"], decay=0.0), s["weights"]
            return lps.attention_paged_decode(s["q"], s["kp"], s["vp"], s["table"], s["lengths"])
        if s["op"] == "evict":
            lengths = lps.kv_pages_evict(s["kp"], s["vp"], s["weights"], s["table"], s["lengths"], s["fresh"], s["budget"],
                                         s["recent"])
            return s["kp"], s["vp"], s["weights"], lengths
        return lps.logits_adjust(s["logits"], tokens=s.get("tokens"), lengths=s.get("lengths"),
                                 prompt_lengths=s.get("prompts"), repetition=s.get("repetition"),
                                 frequency=s.get("frequency"), presence=s.get("presence"), bias_ids=s.get("bias_ids"),
                                 bias=s.get("bias"), allowed=s.get("allowed"))
    return {"rotary": _plain_rotary, "append": _plain_append, "attend": _plain_attend, "evict": _plain_evict,
            "logits": _plain_logits}[s["op"]](s)


def _rotate(x, s):
    f = s["freqs"]
    rot = 2 * f.numel()
    angle = s["positions"].double()[:, None] * f
    cos, sin = ((t * s["magnitude"]).float()[:, None, :] for t in (angle.cos(), angle.sin()))
    head, rest = x[..., :rot].float(), x[..., rot:]
    a, b = (head[..., 0::2], head[..., 1::2]) if s["interleaved"] else (head[..., : rot // 2], head[..., rot // 2:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((ra, rb), -1).flatten(-2) if s["interleaved"] else torch.cat((ra, rb), -1)
    return torch.cat((turned.to(x.dtype), rest), -1)


def _plain_rotary(s):
    return _rotate(s["q"], s), _rotate(s["k"], s)


def _plain_append(s):
    off, page = s["offsets"].long(), s["kp"].shape[2]
    token = torch.arange(s["k"].shape[0], device=off.device)
    b = torch.searchsorted(off[1:], token, right=True)
    row = s["lengths"].long()[b] - (off[b + 1] - token)
    at = s["table"][b, row // page].long()
    s["kp"][at, :, row % page] = _rotate(s["k"], s)
    s["vp"][at, :, row % page] = s["v"]
    return _rotate(s["q"], s), s["kp"], s["vp"]


def _plain_attend(s):
    q, table, lengths = s["q"], s["table"].long(), s["lengths"].long()
    batch, nq, hd = q.shape
    _, nkv, page, _ = s["kp"].shape
    rows = table.shape[1] * page
    seen = torch.arange(rows, device=q.device) < lengths[:, None]  # [B, rows]
    at = table.clamp_min(0)
    k, v = (p[at].permute(0, 2, 1, 3, 4).reshape(batch, nkv, rows, hd).float() for p in (s["kp"], s["vp"]))
    scores = torch.matmul(q.float().view(batch, nkv, nq // nkv, hd), k.transpose(-1, -2)).mul_(hd ** -0.5)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    w = scores.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    w = w.div_(w.sum(-1, keepdim=True).clamp_min(1e-30))
    o = torch.matmul(w, v).view(batch, nq, hd).to(q.dtype)
    if "weights" not in s:
        return o
    of_key = w.sum(2).view(batch, nkv, -1, page).permute(0, 2, 1, 3)  # [B, pages of it, nkv, page]
    kept = torch.where(seen.view(batch, -1, 1, page), of_key, s["weights"][at])
    s["weights"][at[table >= 0]] = kept[table >= 0]
    return o, s["weights"]


def _plain_evict(s):
    table, lengths, fresh = s["table"].long(), s["lengths"].long(), s["fresh"].long()
    budget, recent = s["budget"], s["recent"]
    batch = table.shape[0]
    _, nkv, page, hd = s["kp"].shape
    rows = table.shape[1] * page
    row = torch.arange(rows, device=table.device)
    at = table.clamp_min(0)
    w = s["weights"][at].permute(0, 2, 1, 3).reshape(batch, nkv, rows)
    key = torch.where((row >= lengths[:, None] - recent)[:, None], math.inf, w)
    key = torch.where((row < lengths[:, None])[:, None], key, -math.inf)
    first = key.sort(dim=-1, descending=True, stable=True).indices[..., :budget]  # ties: the lowest row first
    new = lengths.clamp_max(budget)
    taken = torch.arange(first.shape[-1], device=table.device) < new[:, None]
    src = torch.where(taken[:, None], first, rows).sort(-1).values  # [B, nkv, budget], what is not taken last
    b, g, i = torch.nonzero(taken[:, None].expand(-1, nkv, -1), as_tuple=True)
    r = src[b, g, i]
    old, into = at[b, r // page], fresh[b, i // page]
    for x in (s["kp"], s["vp"], s["weights"]):
        x[into, g, i % page] = x[old, g, r % page]
    return s["kp"], s["vp"], s["weights"], new.int()


def _plain_logits(s):
    x = s["logits"].float()
    batch, vocab = x.shape
    if "tokens" in s:
        tokens, at = s["tokens"].long(), torch.arange(s["tokens"].shape[1], device=x.device)
        real = at < s["lengths"][:, None]
        made = (real & (at >= s["prompts"][:, None])).float()
        anywhere = torch.zeros_like(x).scatter_add_(1, tokens, real.float()) > 0
        count = torch.zeros_like(x).scatter_add_(1, tokens, made)
        r = s["repetition"][:, None]
        x = torch.where(anywhere, torch.where(x > 0, x / r, x * r), x)
        x = x - s["frequency"][:, None] * count - s["presence"][:, None] * (count > 0)
    if "bias" in s:
        x = x.scatter_add(1, s["bias_ids"].long(), s["bias"])
    if "allowed" in s:
        at = torch.arange(vocab, device=x.device)
        x = x.masked_fill((s["allowed"][:, at // 32] >> (at % 32)) & 1 == 0, -math.inf)
    return x.to(s["logits"].dtype)


# ---- the definition, in 64 bits --------------------------------------------------------------------

def _turn64(x, positions, case):
    """Each pair as a complex number, turned by its position's angle."""
    rot = case["rot"]
    f = torch.from_numpy(_frequencies(rot, case["stretch"])).to(x.device)
    turn = torch.polar(torch.full_like(f, _magnitude(case["stretch"])).expand(len(positions), -1),
                       positions.double()[:, None] * f)[:, None, :]
    y = x.double().clone()
    pairs = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(y[..., pairs[0]], y[..., pairs[1]]) * turn
    y[..., pairs[0]], y[..., pairs[1]] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _turn64(s["q"], s["positions"], case), _turn64(s["k"], s["positions"], case)
    if case["op"] == "append":
        kp, vp, k = s["kp"].double(), s["vp"].double(), _turn64(s["k"], s["positions"], case)
        off, table = s["offsets"].tolist(), s["table"]
        for b, n in enumerate(s["lengths"].tolist()):
            lo, hi = off[b], off[b + 1]
            rows = torch.arange(n - (hi - lo), n, device=table.device)
            at = table[b].long()[rows // case["page"]]
            kp[at, :, rows % case["page"]] = k[lo:hi]
            vp[at, :, rows % case["page"]] = s["v"][lo:hi].double()
        return _turn64(s["q"], s["positions"], case), kp, vp
    if case["op"] == "attend":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
        weights = s["weights"].double() if case["weights"] else None
        group, page = case["nq"] // case["nkv"], case["page"]
        for b, n in enumerate(s["lengths"].tolist()):
            if n == 0:
                continue
            rows = torch.arange(n, device=DEVICE)
            at, j = s["table"][b].long()[rows // page], rows % page
            k, v = s["kp"][at, :, j].double(), s["vp"][at, :, j].double()  # [n, nkv, hd]
            q = s["q"][b].double().view(case["nkv"], group, case["hd"])
            z = torch.einsum("ghd,ngd->ghn", q, k) / math.sqrt(case["hd"])
            p = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
            o[b] = torch.einsum("ghn,ngd->ghd", p, v).reshape(case["nq"], case["hd"])
            if weights is not None:
                weights[at, :, j] = p.sum(1).T
        return (o, weights) if weights is not None else o
    if case["op"] == "evict":
        kp, vp, weights = s["kp"].clone(), s["vp"].clone(), s["weights"].clone()
        table, fresh, held = s["table"].cpu().numpy(), s["fresh"].cpu().numpy(), s["weights"].cpu().numpy()
        page, budget, recent = case["page"], case["budget"], case["recent"]
        for b, n in enumerate(s["lengths"].tolist()):
            rows = np.arange(n)
            for h in range(case["nkv"]):
                kept = rows
                if n > budget:
                    w = held[table[b, rows // page], h, rows % page][: n - recent]
                    best = np.lexsort((np.arange(n - recent), -w))[: budget - recent]
                    kept = np.concatenate([np.sort(best), rows[n - recent:]])
                to = np.arange(len(kept))
                old, into = (torch.from_numpy(t).to(DEVICE).long() for t in (table[b, kept // page], fresh[b, to // page]))
                j, i = (torch.from_numpy(t % page).to(DEVICE) for t in (kept, to))
                for x, y in ((kp, s["kp"]), (vp, s["vp"]), (weights, s["weights"])):
                    x[into, h, i] = y[old, h, j]
        return kp.double(), vp.double(), weights.double(), None
    x = s["logits"].double()
    for b in range(case["batch"]):
        if "tokens" in s:
            n, prompt = int(s["lengths"][b]), int(s["prompts"][b])
            count = torch.bincount(s["tokens"][b, prompt:n].long(), minlength=case["vocab"]).double()
            ids = torch.unique(s["tokens"][b, :n].long())
            r, old = s["repetition"][b].double(), x[b, ids]
            x[b, ids] = torch.where(old > 0, old / r, old * r)
            x[b] -= s["frequency"][b].double() * count + s["presence"][b].double() * (count > 0)
        if "bias" in s:
            x[b, s["bias_ids"][b].long()] += s["bias"][b].double()
        if "allowed" in s:
            bits = np.unpackbits(s["allowed"][b].cpu().numpy().view(np.uint8), bitorder="little")[: case["vocab"]]
            x[b, torch.from_numpy(bits == 0).to(DEVICE)] = -math.inf
    return x
