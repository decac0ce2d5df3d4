"""Cases for measuring the operators over packed prompts, drafted trees and the key/value cache.

Four operators that work together on one cache ``[batch][kv heads][max_ctx][head_dim]``:

- ``prompt``: causal attention of whole prompts of different lengths, packed one after another;
- ``append``: the packed prompts' (or drafts') key and value rows written to their cache rows;
- ``tree``: attention of a tree of drafted tokens over the cache (one drafted token is plain decoding);
- ``accept``: the accepted path's rows moved together behind the committed ones, in every layer.

With ``own`` false ``run`` computes them in elementary torch operations, in 32 bits, rounded once at the end;
with ``own`` true it calls this package.
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
DEVICE = "cuda"


# ---- cases ----------------------------------------------------------------------------------------

def _prompt(name, lens, nq, nkv, hd, dtype="bf16"):
    return {"name": name, "op": "prompt", "lens": lens, "nq": nq, "nkv": nkv, "hd": hd, "dtype": dtype}


def _append(name, lens, starts, max_ctx, nkv, hd, dtype="bf16"):
    return {"name": name, "op": "append", "lens": lens, "starts": starts, "max_ctx": max_ctx, "nkv": nkv, "hd": hd,
            "dtype": dtype}


def _tree(name, pos, rows, width, max_ctx, nq, nkv, hd, dtype="bf16"):
    return {"name": name, "op": "tree", "pos": pos, "rows": rows, "width": width, "max_ctx": max_ctx, "nq": nq,
            "nkv": nkv, "hd": hd, "dtype": dtype}


def _accept(name, pos, rows, width, max_ctx, layers, nkv, hd, dtype="bf16"):
    return {"name": name, "op": "accept", "pos": pos, "rows": rows, "width": width, "max_ctx": max_ctx,
            "layers": layers, "nkv": nkv, "hd": hd, "dtype": dtype}


def listed():
    return [
        # three short questions of the smallest decoder at once: launch latency
        _prompt("prompt_short", "5,1,12", 4, 2, 64),
        # a serving batch of mixed requests, one of them empty: ragged ends everywhere
        _prompt("prompt_ragged", "517,1,130,1024,77,0,333", 32, 8, 128),
        # four chats of the 1B decoder near its context length, in fp16
        _prompt("prompt_1b_fp16", "1000,1024,999,512", 32, 8, 64, "fp16"),
        # the 8B decoder's whole context as one prompt: the tensor cores' rate
        _prompt("prompt_8b", "8184", 32, 8, 128),
        # the zero-padded decoder's heads, a batch of four long prompts: the largest
        _prompt("prompt_padded_b4", "4033,4096,2500,3999", 48, 12, 128),
        # drafts of eight sequences stored before they are verified
        _append("append_drafts", "26,26,1,13,26,7,26,20", "8100,17,4000,0,777,2048,6500,8000", 8192, 8, 128),
        # a long prompt's rows stored behind nothing, and a second one's behind a shared prefix
        _append("append_prompts", "8184,4001", "0,512", 8192, 8, 128),
        # one token over the 1B decoder's context: plain decoding, latency
        _tree("tree_one_token", "1000", "1", 1, 1024, 32, 8, 64),
        # a tree of 26 drafts over the 8B decoder's context: every cache row read once
        _tree("tree_8b", "8150", "26", 26, 8192, 32, 8, 128),
        # eight sequences of very different lengths, up to 64 drafts each, over a long cache
        _tree("tree_long_b8", "32700,131,20011,32001,9,26000,30500,12345", "64,64,33,64,1,64,50,64", 64, 32768, 32, 8,
              128),
        # one sequence's accepted path in the 8B decoder's 32 layers
        _accept("accept_8b", "1000", "5", 26, 1088, 32, 8, 128),
        # eight sequences, paths of up to 16 of 26 drafts
        _accept("accept_b8", "900,0,77,512,640,1,333,998", "16,3,0,9,1,16,12,7", 26, 1024, 16, 8, 64),
    ]


_HEADS = ((4, 2, 64), (32, 8, 64), (32, 8, 128), (48, 12, 128), (32, 32, 64), (8, 1, 128), (12, 4, 128), (28, 4, 128))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "tree", "tree", "append", "accept"))
    nq, nkv, hd = rng.choice(_HEADS)
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op == "prompt":
        n = rng.randint(1, 12)
        longest = _log(rng, 1, int(math.sqrt(8184.0 * 8184 * 32 / (nq * n))))
        lens = [longest] + [rng.choice((0, 1, rng.randint(0, longest), rng.randint(0, longest), longest))
                            for _ in range(n - 1)]
        rng.shuffle(lens)
        c = _prompt("", ",".join(map(str, lens)), nq, nkv, hd, dtype)
    elif op == "append":
        n = rng.randint(1, 8)
        longest = _log(rng, 1, 4000)
        lens = [longest] + [rng.randint(0, longest) for _ in range(n - 1)]
        starts = [_log(rng, 1, 4000) - 1 for _ in range(n)]
        c = _append("", ",".join(map(str, lens)), ",".join(map(str, starts)), 8192, nkv, hd, dtype)
    elif op == "tree":
        n, width = rng.randint(1, 8), rng.choice((1, 4, 8, 17, 26, 48, 64))
        longest = _log(rng, 1, 32000 if nkv <= 8 else 12000)
        pos = [longest] + [rng.choice((0, rng.randint(0, longest), rng.randint(0, longest))) for _ in range(n - 1)]
        rows = [rng.randint(1, width) for _ in range(n)]
        c = _tree("", ",".join(map(str, pos)), ",".join(map(str, rows)), width, longest + width + rng.randint(0, 99),
                  nq, nkv, hd, dtype)
    else:
        n, width, layers = rng.randint(1, 8), rng.choice((4, 8, 17, 26, 64)), rng.randint(1, 16)
        pos = [rng.randint(0, 900) for _ in range(n)]
        rows = [rng.randint(0, width) for _ in range(n)]
        c = _accept("", ",".join(map(str, pos)), ",".join(map(str, rows)), width, 1024, layers, min(nkv, 12), hd, dtype)
    del c["name"]
    return c


def _ints(text):
    return [int(x) for x in text.split(",")]


def work(case):
    hd, nkv = case["hd"], case["nkv"]
    if case["op"] == "prompt":
        lens, nq = _ints(case["lens"]), case["nq"]
        pairs = sum(n * (n + 1) // 2 for n in lens)  # (query, key) pairs the causal mask leaves
        return {"bytes": 2 * sum(lens) * hd * 2 * (nq + nkv), "flops": 4 * hd * nq * pairs}
    if case["op"] == "append":
        return {"bytes": 2 * 2 * sum(_ints(case["lens"])) * nkv * hd * 2, "flops": 0}
    if case["op"] == "tree":
        pos, rows, nq = _ints(case["pos"]), _ints(case["rows"]), case["nq"]
        kv = sum(p + r for p, r in zip(pos, rows)) * nkv * hd * 2 * 2
        return {"bytes": kv + 2 * sum(rows) * nq * hd * 2 + 4 * sum(rows),
                "flops": 4 * hd * nq * sum((p + 1) * r for p, r in zip(pos, rows))}
    return {"bytes": 2 * 2 * sum(_ints(case["rows"])) * case["layers"] * nkv * hd * 2, "flops": 0}


# ---- inputs ---------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    host = np.random.default_rng(int(seed))
    dt, hd, nkv = _DTYPES[case["dtype"]], case["hd"], case["nkv"]
    s = {"op": case["op"]}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=dt)

    if case["op"] in ("prompt", "append"):
        lens = _ints(case["lens"])
        offsets = np.zeros(len(lens) + 1, np.int32)
        offsets[1:] = np.cumsum(lens)
        s["offsets"], s["offsets_dev"] = offsets, torch.from_numpy(offsets).to(DEVICE)
        s["longest"], n = max(lens), int(offsets[-1])
    if case["op"] == "prompt":
        # rows of one fused projection: q, k and v are column ranges of it
        nq = case["nq"]
        fused = normal(n, (nq + 2 * nkv) * hd)
        s["q"] = fused[:, : nq * hd].view(n, nq, hd)
        s["k"] = fused[:, nq * hd: (nq + nkv) * hd].view(n, nkv, hd)
        s["v"] = fused[:, (nq + nkv) * hd:].view(n, nkv, hd)
    elif case["op"] == "append":
        fused = normal(n, 2 * nkv * hd)
        s["k"], s["v"] = fused[:, : nkv * hd].view(n, nkv, hd), fused[:, nkv * hd:].view(n, nkv, hd)
        s["starts"] = np.array(_ints(case["starts"]), np.int32)
        s["starts_dev"] = torch.from_numpy(s["starts"]).to(DEVICE)
        s["kc"], s["vc"] = (normal(len(lens), nkv, case["max_ctx"], hd) for _ in range(2))
    elif case["op"] == "tree":
        nq, width = case["nq"], case["width"]
        pos, rows = np.array(_ints(case["pos"]), np.int32), np.array(_ints(case["rows"]), np.int32)
        # each draft hangs from one of the eight before it, or from the last committed token
        parents = np.empty((len(pos), width), np.int32)
        for t in range(width):
            parents[:, t] = host.integers(max(-1, t - 8), t, size=len(pos))
        s.update(pos=pos, rows=rows, pos_dev=torch.from_numpy(pos).to(DEVICE), rows_dev=torch.from_numpy(rows).to(DEVICE),
                 parents=torch.from_numpy(parents).to(DEVICE), reach=int((pos + rows).max()),
                 q=normal(len(pos), width, nq, hd), out=torch.zeros(len(pos), width, nq, hd, device=DEVICE, dtype=dt),
                 kc=normal(len(pos), nkv, case["max_ctx"], hd), vc=normal(len(pos), nkv, case["max_ctx"], hd))
    else:
        width, pos, rows = case["width"], np.array(_ints(case["pos"]), np.int32), np.array(_ints(case["rows"]), np.int32)
        path = np.full((len(pos), width), -1, np.int32)
        for b, r in enumerate(rows):
            path[b, :r] = np.sort(host.choice(width, size=int(r), replace=False))
        s.update(pos=pos, pos_dev=torch.from_numpy(pos).to(DEVICE), path=torch.from_numpy(path).to(DEVICE),
                 accepted=torch.from_numpy(rows).to(DEVICE))
        s["kc"], s["vc"] = (normal(case["layers"], len(pos), nkv, case["max_ctx"], hd) for _ in range(2))
    return s


# ---- one pass -------------------------------------------------------------------------------------

def run(s):
    if own:
        import layer_pipeline_staged_gb300 as lps

        if s["op"] == "prompt":
            return lps.attention_prompt_packed(s["q"], s["k"], s["v"], s["offsets"])
        if s["op"] == "append":
            lps.kv_rows_append(s["k"], s["v"], s["offsets"], s["kc"], s["vc"], s["starts"])
            return s["kc"], s["vc"]
        if s["op"] == "tree":
            return lps.attention_tree_verify(s["q"], s["kc"], s["vc"], s["parents"], s["pos"], s["rows"], out=s["out"])
        lps.kv_rows_accept(s["kc"], s["vc"], s["pos"], s["path"], s["accepted"])
        return s["kc"], s["vc"]
    return {"prompt": _plain_prompt, "append": _plain_append, "tree": _plain_tree, "accept": _plain_accept}[s["op"]](s)


def _softmax_rows(scores):
    """Weights of each row over the last axis, and nothing where a row has no finite score."""
    top = scores.amax(-1, keepdim=True)
    w = scores.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    return w.div_(w.sum(-1, keepdim=True).clamp_min(1e-30))


def _plain_prompt(s):
    q, k, v, off, longest = s["q"], s["k"], s["v"], s["offsets_dev"].long(), s["longest"]
    n, nq, hd = q.shape
    nkv = k.shape[1]
    lens = off[1:] - off[:-1]
    at = torch.arange(longest, device=q.device)
    rows = (off[:-1, None] + at).clamp_max(n - 1)  # [B, longest]: each sequence's tokens, padded to the longest
    batch = rows.shape[0]
    qp = q.float()[rows].view(batch, longest, nkv, nq // nkv, hd).permute(0, 2, 3, 1, 4).reshape(batch, nkv, -1, hd)
    kp, vp = k.float()[rows].permute(0, 2, 1, 3), v.float()[rows].permute(0, 2, 1, 3)
    scores = torch.matmul(qp, kp.transpose(-1, -2)).mul_(hd ** -0.5).view(batch, nkv, nq // nkv, longest, longest)
    scores.masked_fill_(at[None, :] > at[:, None], -math.inf)
    scores.masked_fill_((at >= lens[:, None])[:, None, None, None, :], -math.inf)
    o = torch.matmul(_softmax_rows(scores).view(batch, nkv, -1, longest), vp)
    o = o.view(batch, nq, longest, hd).permute(0, 2, 1, 3)
    return o[at < lens[:, None]].to(q.dtype)  # the tokens that exist, packed again


def _plain_append(s):
    off, start = s["offsets_dev"].long(), s["starts_dev"].long()
    token = torch.arange(s["k"].shape[0], device=off.device)
    b = torch.searchsorted(off[1:], token, right=True)
    row = start[b] + token - off[b]
    s["kc"][b, :, row] = s["k"]
    s["vc"][b, :, row] = s["v"]
    return s["kc"], s["vc"]


def _plain_tree(s):
    q, pos, rows, parents, reach = s["q"], s["pos_dev"].long(), s["rows_dev"].long(), s["parents"].long(), s["reach"]
    batch, width, nq, hd = q.shape
    nkv = s["kc"].shape[1]
    draft = torch.arange(width, device=q.device)
    step = (parents[:, :, None] == draft).double() + torch.eye(width, device=q.device, dtype=torch.float64)
    above = torch.linalg.matrix_power(step, width) > 0  # [B, t, a]: a is t or one of its ancestors
    key = torch.arange(reach, device=q.device)
    ahead = key - pos[:, None]  # [B, reach]: the draft that a cache row holds
    of_draft = torch.gather(above, 2, ahead.clamp(0, width - 1)[:, None, :].expand(-1, width, -1))
    seen = (ahead < 0)[:, None, :] | (of_draft & ((ahead >= 0) & (ahead < rows[:, None]))[:, None, :])
    kf, vf = s["kc"][:, :, :reach].float(), s["vc"][:, :, :reach].float()
    qf = q.float().view(batch, width, nkv, nq // nkv, hd).permute(0, 2, 3, 1, 4).reshape(batch, nkv, -1, hd)
    scores = torch.matmul(qf, kf.transpose(-1, -2)).mul_(hd ** -0.5).view(batch, nkv, nq // nkv, width, reach)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    o = torch.matmul(_softmax_rows(scores).view(batch, nkv, -1, reach), vf)
    o = o.view(batch, nq, width, hd).permute(0, 2, 1, 3).to(q.dtype)
    s["out"].copy_(torch.where((draft < rows[:, None])[:, :, None, None], o, s["out"]))
    return s["out"]


def _plain_accept(s):
    pos, path, accepted = s["pos_dev"].long(), s["path"].long(), s["accepted"].long()
    i = torch.arange(path.shape[1], device=path.device)
    taken = i < accepted[:, None]
    b = torch.arange(path.shape[0], device=path.device)[:, None].expand_as(path)[taken]
    src, dst = (pos[:, None] + path)[taken], (pos[:, None] + i)[taken]
    s["kc"][:, b, :, dst] = s["kc"][:, b, :, src]
    s["vc"][:, b, :, dst] = s["vc"][:, b, :, src]
    return s["kc"], s["vc"]


# ---- the definition, in 64 bits --------------------------------------------------------------------

def _attend64(q, k, v, allowed):
    """One kv head's rows by log-sum-exp: q [G, t, hd], k and v [n, hd], allowed [t, n]."""
    z = torch.einsum("gtd,nd->gtn", q.double(), k.double()) / math.sqrt(q.shape[-1])
    z = z.masked_fill(~allowed, -math.inf)
    return torch.einsum("gtn,nd->gtd", torch.exp(z - torch.logsumexp(z, -1, keepdim=True)), v.double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prompt":
        q, k, v, off = s["q"], s["k"], s["v"], s["offsets"]
        group = case["nq"] // case["nkv"]
        o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
        for lo, hi in zip(off[:-1], off[1:]):
            for t0 in range(int(lo), int(hi), 2048):
                t1 = min(t0 + 2048, int(hi))
                allowed = torch.ones(t1 - t0, t1 - int(lo), dtype=torch.bool, device=q.device).tril(t0 - int(lo))
                for h in range(case["nkv"]):
                    heads = slice(h * group, (h + 1) * group)
                    o[t0:t1, heads] = _attend64(q[t0:t1, heads].transpose(0, 1), k[lo:t1, h], v[lo:t1, h],
                                                allowed).transpose(0, 1)
        return o
    if case["op"] == "append":
        kc, vc = s["kc"].clone(), s["vc"].clone()
        for b, start in enumerate(s["starts"]):
            lo, hi = int(s["offsets"][b]), int(s["offsets"][b + 1])
            kc[b, :, start:start + hi - lo] = s["k"][lo:hi].transpose(0, 1)
            vc[b, :, start:start + hi - lo] = s["v"][lo:hi].transpose(0, 1)
        return kc.double(), vc.double()
    if case["op"] == "tree":
        o = s["out"].double()
        group = case["nq"] // case["nkv"]
        parents = s["parents"].cpu().numpy()
        for b, (pos, rows) in enumerate(zip(s["pos"].tolist(), s["rows"].tolist())):
            allowed = torch.zeros(rows, pos + rows, dtype=torch.bool)
            allowed[:, :pos] = True
            for t in range(rows):
                a = t
                while a >= 0:
                    allowed[t, pos + a] = True
                    a = int(parents[b, a])
            allowed = allowed.to(o.device)
            for h in range(case["nkv"]):
                heads = slice(h * group, (h + 1) * group)
                o[b, :rows, heads] = _attend64(s["q"][b, :rows, heads].transpose(0, 1), s["kc"][b, h, :pos + rows],
                                               s["vc"][b, h, :pos + rows], allowed).transpose(0, 1)
        return o
    path, taken = s["path"].cpu().numpy(), s["accepted"].cpu().numpy()
    kc, vc = s["kc"].clone(), s["vc"].clone()
    for b, pos in enumerate(s["pos"].tolist()):
        for i in range(int(taken[b])):
            kc[:, b, :, pos + i] = s["kc"][:, b, :, pos + int(path[b, i])]
            vc[:, b, :, pos + i] = s["vc"][:, b, :, pos + int(path[b, i])]
    return kc.double(), vc.double()
