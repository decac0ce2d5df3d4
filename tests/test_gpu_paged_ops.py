"""Rotary positions, the append to pages, eviction and the logits' adjustment on the GPU, against their definitions in
64 bits, and a captured decode step of all of them.

Tolerance of a turned element x cos a - y sin a, with u = eps / 2 of the element type: the result is rounded once, u |o|;
the angle's fraction of half a turn is rounded to fp32, off by 2^-25 half turns, 1.6 2^-24 radians; sincospi by 2 ulp, 2
2^-24; the factor by the magnitude, the product and the sum by half an ulp each, 1.5 2^-24 in all: (1 + u) 6 2^-24 magnitude
(|x| + |y|). A frequency is held to 2^-52 relative, counted where positions are large.
Logits: at most 8 roundings to fp32 of sums of the terms' magnitudes, and the result's own.
"""
import math
from fractions import Fraction

import numpy as np
import pytest

import layer_pipeline_staged_gb300 as lps

torch = pytest.importorskip("torch")
from paged import DT, Paged, gen, i32, randn  # noqa: E402
from test_gpu_paged_attention import attend64, close  # noqa: E402

pytestmark = pytest.mark.gpu


def turn64(x, positions, f, interleaved, mag):
    """(turned x [tokens, heads, hd] in 64 bits, bound)."""
    rot, u = 2 * len(f), torch.finfo(x.dtype).eps / 2
    y = x.double().clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    angle = (positions.double()[:, None] * f.to(x.device))[:, None]
    p, q = x[..., a].double(), x[..., b].double()
    y[..., a], y[..., b] = mag * (p * angle.cos() - q * angle.sin()), mag * (q * angle.cos() + p * angle.sin())
    tol = torch.zeros_like(y)
    far = 2.0 ** -50 * angle.abs()  # the frequency's rounding, here and in the kernel
    tol[..., a] = tol[..., b] = (1 + u) * (6 * 2.0 ** -24 + far) * mag * (p.abs() + q.abs())
    tol[..., :rot] += u * y[..., :rot].abs() + (2.0 ** -25 if x.dtype == torch.float16 else 0.0)
    return y, tol


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("hd,rot", [(64, 64), (128, 128), (128, 64), (128, 32), (64, 16), (64, 48), (128, 112)])
@pytest.mark.parametrize("tokens", [1, 5, 257, 1023])
def test_rotary_rows(tokens, hd, rot, dtype, interleaved):
    g = gen(tokens)
    fused = randn(g, tokens, 7, hd, dtype=DT[dtype])
    q, k = fused[:, :4], fused[:, 4:6]
    pos = torch.randint(0, 131072, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    f = lps.rotary_frequencies(rot, 500000.0)
    mag = 1.0 if rot == hd else 1.2
    qo, ko = lps.rotary_rows(q, k, pos, f.cuda(), interleaved=interleaved, magnitude=mag)
    for x, y in ((q, qo), (k, ko)):
        ref, tol = turn64(x, pos, f, interleaved, mag)
        close(y, ref, tol)
        assert torch.equal(y[..., rot:], x[..., rot:])
    a, b = q.contiguous(), k.contiguous()
    same = lps.rotary_rows(a, b, pos, f.cuda(), interleaved=interleaved, magnitude=mag, out=(a, b))  # in place
    assert same[0] is a and same[1] is b and torch.equal(a, qo) and torch.equal(b, ko)


@pytest.mark.parametrize("interleaved", [False, True])
def test_negative_positions_turn_back_and_are_the_gradient(interleaved):
    """The turn is linear, and orthogonal at magnitude 1: its transpose is the turn by the negative positions. Checked
    against autograd through the 64-bit formula, and against differences."""
    g, f = gen(3), lps.rotary_frequencies(32, 10000.0)
    q, k = randn(g, 6, 2, 64, dtype=torch.bfloat16), randn(g, 6, 1, 64, dtype=torch.bfloat16)
    pos = i32([0, 1, 17, 1000, 65536, 131071])
    there = lps.rotary_rows(q, k, pos, f.cuda(), interleaved=interleaved)
    back = lps.rotary_rows(*there, -pos, f.cuda(), interleaved=interleaved)
    for x, y in ((q, back[0]), (k, back[1])):
        ref, tol = turn64(there[0] if x is q else there[1], -pos, f, interleaved, 1.0)
        close(y, ref, tol)
    grad = randn(g, 6, 2, 64, dtype=torch.bfloat16)
    leaf = q.double().requires_grad_()
    angle = (pos.double()[:, None] * f.cuda())[:, None]
    a, b = (leaf[..., 0:32:2], leaf[..., 1:32:2]) if interleaved else (leaf[..., :16], leaf[..., 16:32])
    ra, rb = a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()
    turned = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    (torch.cat((turned, leaf[..., 32:]), -1) * grad.double()).sum().backward()
    got = lps.rotary_rows(grad, k, -pos, f.cuda(), interleaved=interleaved)[0]
    _, tol = turn64(grad, -pos, f, interleaved, 1.0)
    close(got, leaf.grad, tol, "gradient")
    step = torch.zeros_like(q)
    step[:, :, 3] = 1.0  # the function is linear: a difference of any size is exact but for the roundings
    moved = turn64(q.double() + step.double(), pos, f, interleaved, 1.0)[0] - turn64(q.double(), pos, f, interleaved, 1.0)[0]
    close(got[:, :, 3], (moved * grad.double()).sum(-1), tol[:, :, 3] + 1e-12, "difference")


def test_positions_at_the_ends_of_32_bits():
    """Whole turns drop out exactly: against the angle's fraction of a turn in rational arithmetic."""
    pi = Fraction("3.14159265358979323846264338327950288419716939937510")
    f = lps.rotary_frequencies(64, 10000.0)
    pos = [2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, -(10 ** 9)]
    q = torch.zeros(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    q[..., :32] = 1.0
    out = lps.rotary_rows(q, q.clone(), i32(pos), f.cuda())[0].double().cpu()
    for t, p in enumerate(pos):
        for i in range(32):
            turns = Fraction(float(f[i])) * p / (2 * pi)
            a = 2 * math.pi * float(turns - math.floor(turns))
            off = 2.0 ** -8 + 6 * 2.0 ** -24 + 2 * math.pi * abs(float(turns)) * 2.0 ** -51
            assert abs(out[t, 0, i] - math.cos(a)) <= off and abs(out[t, 0, 32 + i] - math.sin(a)) <= off


@pytest.mark.parametrize("scaling,kw", [(None, {}), ("linear", {"factor": 4.0}), ("ntk", {"factor": 4.0}),
                                        ("parts", {"factor": 8.0, "original": 8192})])
def test_frequencies_turn_the_calls(scaling, kw):
    f = lps.rotary_frequencies(128, 500000.0, scaling, **kw)
    q, k = randn(gen(1), 40, 2, 128, dtype=torch.bfloat16), randn(gen(2), 40, 2, 128, dtype=torch.bfloat16)
    pos = torch.arange(100000, 100040, device="cuda", dtype=torch.int32)
    out, _ = lps.rotary_rows(q, k, pos, f.cuda())
    close(out, *turn64(q, pos, f, False, 1.0))


def check_append(counts, lens, nq, nkv, hd, page, dtype, rot, first=0, behind=0, positions=None, interleaved=False):
    g = gen(sum(counts) + 1)
    off = np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)
    n = int(off[-1]) + behind
    c = Paged(lens, nkv, hd, page, dtype)
    fused = randn(g, n, nq + 2 * nkv, hd, dtype=dtype)
    q, k, v = fused[:, :nq], fused[:, nq:nq + nkv], fused[:, nq + nkv:]
    f = lps.rotary_frequencies(rot, 10000.0) if rot else None
    kw = torch.full((c.pages, nkv, page), 3.0, device="cuda")
    row_of = np.zeros(n, np.int32)
    for s, m in enumerate(counts):
        row_of[off[s]:off[s + 1]] = np.arange(lens[s] - m, lens[s])
    pos = i32(row_of) if positions is None else positions(n)
    kp, vp, q_out = c.kp.clone(), c.vp.clone(), torch.full_like(q, 9.0)
    decode = first == behind == 0 and list(counts) == [1] * len(counts)
    for offsets in ([i32(off), None] if decode else [i32(off)]):
        got = lps.rotary_append_paged(q, k, v, offsets, c.lengths, c.table, kp, vp, None if f is None else f.cuda(),
                                      positions=None if positions is None else pos, interleaved=interleaved, key_weights=kw,
                                      q_out=q_out)
        assert got is q_out
    live = slice(int(off[0]), int(off[-1]))
    if rot:
        qr, qt = turn64(q, pos, f, interleaved, 1.0)
        kr, kt = turn64(k, pos, f, interleaved, 1.0)
    else:
        qr, qt, kr, kt = q.double(), torch.zeros_like(q, dtype=torch.float64), k.double(), torch.zeros_like(k, dtype=torch.float64)
    close(q_out[live], qr[live], qt[live], "q")
    assert (q_out[: live.start] == 9.0).all() and (q_out[live.stop:] == 9.0).all()
    kr_got, new = kp.clone(), torch.zeros(c.pages, page, dtype=torch.bool, device="cuda")
    for s, m in enumerate(counts):
        if not m:
            continue
        rows = torch.arange(lens[s] - m, lens[s], device="cuda")
        at, j = c.table[s].long()[rows // page], rows % page
        close(kp[at, :, j], kr[off[s]:off[s + 1]], kt[off[s]:off[s + 1]], f"keys of {s}")
        assert torch.equal(vp[at, :, j], v[off[s]:off[s + 1]])
        assert (kw[at, :, j] == 0).all()
        new[at, j] = True
    old = (~new)[:, None, :].expand(-1, nkv, -1)
    assert torch.equal(kr_got[old].nan_to_num(), c.kp[old].nan_to_num()) and torch.equal(vp[old].nan_to_num(), c.vp[old].nan_to_num())
    assert (kw[old] == 3.0).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("counts,lens", [([1], [1]), ([1, 1, 1], [17, 1, 64]), ([0, 40, 0, 1, 300, 0], [0, 40, 9, 65, 301, 16]),
                                         ([1] * 300, list(range(1, 301)))])
@pytest.mark.parametrize("nq,nkv,hd,page,rot", [(4, 2, 64, 16, 64), (32, 8, 128, 8, 32), (3, 1, 128, 24, 0), (5, 5, 64, 128, 48)])
def test_append(counts, lens, nq, nkv, hd, page, rot, dtype):
    check_append(counts, lens, nq, nkv, hd, page, DT[dtype], rot)


def test_append_beside_unused_tokens_and_with_positions_of_its_own():
    check_append([7, 0, 30], [20, 5, 30], 4, 2, 64, 16, torch.bfloat16, 64, first=3, behind=11)
    check_append([7, 0, 30], [20, 5, 30], 4, 2, 64, 16, torch.bfloat16, 64, positions=lambda n: i32(np.arange(n) * 1000 + 5),
                 interleaved=True)


def test_append_stores_nothing_outside_the_table():
    nkv, hd, page = 2, 64, 16
    c = Paged([16, 16, 16, 16, 16], nkv, hd, page, torch.bfloat16)
    q, k, v = (randn(gen(1), 5, h, hd, dtype=torch.bfloat16) for h in (4, nkv, nkv))
    f, pos = lps.rotary_frequencies(64).cuda(), i32([4, 5, 6, 7, 8])
    kp, vp = c.kp.clone(), c.vp.clone()
    table = c.table.clone()
    table[3], table[4] = -1, c.pages
    out = lps.rotary_append_paged(q, k, v, None, i32([0, 17, -2 ** 31, 3, 3]), table, kp, vp, f, positions=pos)
    assert torch.equal(kp.nan_to_num(), c.kp.nan_to_num()) and torch.equal(vp.nan_to_num(), c.vp.nan_to_num())
    close(out, *turn64(q, pos, f.cpu(), False, 1.0))
    # offsets that make no sense: rows may go to any row that the table names, and nothing outside it is touched
    guard = torch.full((3, c.pages, nkv, page, hd), 7.0, device="cuda", dtype=torch.bfloat16)
    lps.rotary_append_paged(q, k, v, i32([0, 2 ** 30, -5, 3, 2, 5]), c.lengths, c.table, guard[1], guard[1].clone(), f, positions=pos)
    assert (guard[0] == 7.0).all() and (guard[2] == 7.0).all()


# ---- eviction -----------------------------------------------------------------------------------------

def evicted(w, n, budget, recent):
    """The rows that stay of n with weights w (numpy), in order."""
    if n <= budget:
        return np.arange(n)
    w = np.where(np.isnan(w[: n - recent]), -np.inf, w[: n - recent])
    nan = np.isnan(w)
    best = np.lexsort((np.arange(n - recent), nan, -w))[: budget - recent]
    return np.concatenate([np.sort(best), np.arange(n - recent, n)])


def check_evict(lens, nkv, hd, page, budget, recent, weights, width=None):
    need = sum(-(-min(n, budget) // page) for n in lens)
    c = Paged(lens, nkv, hd, page, torch.bfloat16, spare=need + 2)
    kw = torch.full((c.pages, nkv, page), 77.0, device="cuda")
    for b, n in enumerate(lens):
        at, j = c.at(b)
        kw[at, :, j] = weights(b, nkv, n).T
    fresh = np.full((len(lens), -(-budget // page) if width is None else width), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-min(n, budget) // page)
        fresh[b, :m] = c.free[at:at + m]
        at += m
    kp, vp, w = c.kp.clone(), c.vp.clone(), kw.clone()
    new = lps.kv_pages_evict(kp, vp, w, c.table, c.lengths, i32(fresh), budget, recent)
    assert new.tolist() == [min(n, budget) for n in lens] and new.dtype == torch.int32
    ek, ev, ew = c.kp.clone(), c.vp.clone(), kw.clone()
    for b, n in enumerate(lens):
        for h in range(nkv):
            at, j = c.at(b)
            rows = evicted(kw[at, h, j].cpu().numpy(), n, budget, recent)
            src = torch.from_numpy(rows).cuda()
            dst = torch.arange(len(rows), device="cuda")
            to, i = i32(fresh)[b].long()[dst // page], dst % page
            for pool, was in ((ek, c.kp), (ev, c.vp), (ew, kw)):
                pool[to, h, i] = was[at[src], h, j[src]]
    for got, want in ((kp, ek), (vp, ev), (w, ew)):
        assert torch.equal(torch.nan_to_num(got, nan=-123.0), torch.nan_to_num(want, nan=-123.0))


def _spread(seed):
    return lambda b, nkv, n: torch.rand(nkv, n, generator=gen(seed + b), device="cuda") ** 8


@pytest.mark.parametrize("lens,budget,recent", [([100], 50, 10), ([100], 100, 3), ([101], 100, 0), ([5, 0, 1, 300, 64], 64, 64),
                                                ([2000, 1, 1024, 1025], 1023, 1), ([9000, 33], 4000, 100), ([40], 1, 0), ([40], 1, 1)])
@pytest.mark.parametrize("nkv,hd,page", [(2, 64, 16), (1, 128, 24), (3, 128, 8)])
def test_evict(nkv, hd, page, lens, budget, recent):
    check_evict(lens, nkv, hd, page, budget, recent, _spread(1))


@pytest.mark.parametrize("kind", ["equal", "few", "zeros", "negative", "nan", "inf"])
def test_evict_orders_weights_and_breaks_ties_by_the_lowest_row(kind):
    def weights(b, nkv, n):
        x = torch.rand(nkv, n, generator=gen(9 + b), device="cuda")
        if kind == "equal":
            return torch.ones_like(x)
        if kind == "few":
            return (x * 4).floor()
        if kind == "zeros":
            return torch.where(x > 0.5, torch.zeros_like(x), -torch.zeros_like(x))
        if kind == "negative":
            return x - 0.5
        x[:, ::3] = float("nan") if kind == "nan" else float("inf")
        if kind == "inf":
            x[:, 1::3] = -float("inf")
        return x
    check_evict([1500, 70], 2, 64, 16, 600, 20, weights)


def test_evict_leaves_sequences_that_break_the_rules():
    c = Paged([100, 100, 100, 100, 100], 2, 64, 16, torch.bfloat16, spare=30)
    kw = torch.rand(c.pages, 2, 16, generator=gen(1), device="cuda")
    table, fresh = c.table.clone(), i32(c.free[:20].reshape(5, 4))
    table[1, 2] = -1
    table[2, 0] = c.pages
    fresh[3, 3] = 2 ** 31 - 1
    lengths = i32([100, 100, 100, 100, 113])
    kp, vp, w = c.kp.clone(), c.vp.clone(), kw.clone()
    new = lps.kv_pages_evict(kp, vp, w, table, lengths, fresh, 64, 5)
    assert new.tolist() == [64, -1, -1, -1, -1]
    touched = torch.zeros(c.pages, dtype=torch.bool, device="cuda")
    touched[fresh[0].long()] = True
    for got, was in ((kp, c.kp), (vp, c.vp), (w, kw)):
        assert torch.equal(got[~touched].nan_to_num(), was[~touched].nan_to_num())
    other = torch.full((5, 7), -1, device="cuda", dtype=torch.int32)
    other[4, 0] = int(c.free[20])
    assert lps.kv_pages_evict(kp, vp, w, c.table, i32([-1, 0, 2 ** 31 - 1, -2 ** 31, 5]), other, 112, 0).tolist() == [-1, 0, -1, -1, 5]


# ---- logits -------------------------------------------------------------------------------------------

def adjust64(x, tokens, lengths, prompts, rep, freq, pres, ids, bias, allowed):
    """(result, bound) on the CPU in 64 bits."""
    u = torch.finfo(x.dtype).eps / 2
    y = x.double().cpu().clone()
    mag = y.abs()
    batch, vocab = y.shape
    for b in range(batch):
        if tokens is not None:
            hist = tokens[b, : int(lengths[b].clamp(0, tokens.shape[1]))].cpu().long()
            made = hist[max(0, int(prompts[b])):] if prompts is not None else hist
            hist, made = (t[(t >= 0) & (t < vocab)] for t in (hist, made))
            c = torch.bincount(made, minlength=vocab).double()
            some = torch.unique(hist)
            r = 1.0 if rep is None else float(rep[b])
            y[b, some] = torch.where(y[b, some] > 0, y[b, some] / r, y[b, some] * r)
            fr, pr = (0.0 if t is None else float(t[b]) for t in (freq, pres))
            mag[b] = torch.maximum(mag[b], y[b].abs()) + abs(fr) * c + abs(pr) * (c > 0)
            y[b] -= fr * c + pr * (c > 0)
        if ids is not None:
            for i, v in zip(ids[b].tolist(), bias[b].double().tolist()):
                if 0 <= i < vocab:
                    y[b, i] += v
                    mag[b, i] += abs(v)
        if allowed is not None:
            bits = np.unpackbits(allowed[b].cpu().numpy().view(np.uint8), bitorder="little")[:vocab]
            y[b, torch.from_numpy(bits == 0)] = -math.inf
    tol = u * torch.where(torch.isfinite(y), y.abs(), torch.zeros_like(y)) + (1 + u) * 8 * 2.0 ** -24 * mag + (2.0 ** -25 if x.dtype == torch.float16 else 0)
    return y, tol


def same_logits(got, ref, tol):
    got = got.double().cpu()
    fin = torch.isfinite(ref)
    assert torch.equal(got[~fin], ref[~fin])
    assert torch.isfinite(got[fin]).all() and ((got - ref)[fin].abs() <= tol[fin]).all()


def logits_inputs(batch, vocab, width, entries, dtype, seed=1):
    g, host = gen(seed), np.random.default_rng(seed)
    x = 4 * randn(g, batch, vocab, dtype=torch.float32)
    d = {"tokens": None, "lengths": None, "prompt_lengths": None, "repetition": None, "frequency": None, "presence": None,
         "bias_ids": None, "bias": None}
    if width:
        d["tokens"] = i32(host.integers(-2, vocab + 3, size=(batch, width)) % max(2, vocab + 5 if seed % 2 else vocab // 3 + 1))
        d["tokens"][:, ::11] = -1
        d["lengths"] = i32(host.integers(-1, width + 2, size=batch))
        d["lengths"][0] = width
        d["prompt_lengths"] = i32(host.integers(-1, width + 2, size=batch))
        for name in ("repetition", "frequency", "presence"):
            d[name] = torch.rand(batch, generator=g, device="cuda") + (0.7 if name == "repetition" else -0.3)
    if entries:
        d["bias_ids"] = i32(host.integers(-1, vocab + 1, size=(batch, entries)))
        d["bias"] = randn(g, batch, entries, dtype=torch.float32)
    d["allowed"] = i32(host.integers(-2 ** 31, 2 ** 31, size=(batch, -(-vocab // 32))))
    return x.to(dtype), d


ORDER = ("tokens", "lengths", "prompt_lengths", "repetition", "frequency", "presence", "bias_ids", "bias", "allowed")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("batch,vocab,width,entries", [(1, 1, 1, 1), (3, 33, 40, 9), (2, 8191, 100, 0), (2, 8192, 0, 30), (5, 8193, 3000, 300),
                                                       (1, 32000, 8000, 8), (4, 50257, 77, 2), (2, 131073, 500, 1000)])
def test_logits(batch, vocab, width, entries, dtype):
    for seed in (1, 2):
        x, d = logits_inputs(batch, vocab, width, entries, dtype, seed)
        for drop in ((), ("allowed",), ("prompt_lengths", "presence"), ("bias_ids", "bias"), ("repetition",), ("frequency", "allowed")):
            kw = {k: v for k, v in d.items() if k not in drop and v is not None}
            ref = adjust64(x, *(kw.get(k) for k in ORDER))
            got = lps.logits_adjust(x, **kw)
            assert got.dtype == dtype
            same_logits(got, *ref)


def test_logits_in_place_strided_and_with_nothing_allowed():
    x, d = logits_inputs(3, 1001, 50, 5, torch.float32)
    want = lps.logits_adjust(x, **d)
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.full((3, 1010), 5.0, device="cuda", dtype=dtype)
        wide[:, 3:1004] = x
        view = wide[:, 3:1004]
        ref = lps.logits_adjust(view.contiguous(), **d)
        assert torch.equal(lps.logits_adjust(view, **d), ref)
        assert lps.logits_adjust(view, **d, out=view) is view and torch.equal(view, ref)
        assert (wide[:, :3] == 5.0).all() and (wide[:, 1004:] == 5.0).all()
    assert torch.equal(want, lps.logits_adjust(x, **d))
    none = torch.zeros(3, 32, device="cuda", dtype=torch.int32)
    assert (lps.logits_adjust(x, allowed=none) == -math.inf).all()
    odd = x.clone()
    odd[0, :3] = torch.tensor([float("nan"), float("inf"), -float("inf")])
    assert (lps.logits_adjust(odd, allowed=none) == -math.inf).all()
    got = lps.logits_adjust(odd, allowed=torch.full_like(none, -1))
    assert torch.equal(got.nan_to_num(nan=1e30), odd.nan_to_num(nan=1e30))


def test_logits_of_one_token_many_times():
    """One token is the whole history, and all the biases' entries."""
    x = torch.zeros(2, 20000, device="cuda")
    tokens, n = torch.full((2, 8000), 12345, device="cuda", dtype=torch.int32), i32([8000, 1])
    ones = torch.ones(2, device="cuda")
    out = lps.logits_adjust(x, tokens=tokens, lengths=n, frequency=0.25 * ones, presence=2 * ones,
                            bias_ids=torch.full((2, 500), 12345, device="cuda", dtype=torch.int32), bias=torch.full((2, 500), 0.5, device="cuda"))
    assert out[:, 12345].tolist() == [-2000.0 - 2.0 + 250.0, -0.25 - 2.0 + 250.0]
    out[:, 12345] = 0
    assert (out == 0).all()


# ---- a run of them ------------------------------------------------------------------------------------

def test_a_captured_decode_step_and_an_eviction():
    """Two prompts stored, then steps that one graph replays: rotate and append, attend, adjust the logits, choose; then an
    eviction, after which the graph goes on in the new pages. Every step against the formulas on the rows kept so far."""
    nq, nkv, hd, page, vocab, width = 8, 2, 64, 16, 500, 12
    g, dt, scale = gen(5), torch.bfloat16, hd ** -0.5
    prompts, room = [37, 100], 40
    f = lps.rotary_frequencies(hd, 10000.0, "parts", factor=2.0, original=64)
    fd = f.cuda()
    kp, vp = (torch.full((room, nkv, page, hd), float("nan"), device="cuda", dtype=dt) for _ in range(2))
    weights = torch.zeros(room, nkv, page, device="cuda")
    order = torch.randperm(room, generator=torch.Generator().manual_seed(1))
    table, fresh = order[:24].view(2, width).int().cuda(), order[24:40].view(2, 8).int().cuda()
    embed, head = randn(g, vocab, (nq + 2 * nkv) * hd, dtype=dt), randn(g, vocab, nq * hd, dtype=dt) * 0.3
    # the prompts: turned, attended (contiguous), stored
    off = [0, 37, 137]
    rows = randn(g, 137, nq + 2 * nkv, hd, dtype=dt)
    pos = torch.cat([torch.arange(n) for n in prompts]).int().cuda()
    q, k, v = rows[:, :nq], rows[:, nq:nq + nkv], rows[:, nq + nkv:]
    lengths = i32(prompts)
    q = lps.rotary_append_paged(q, k, v, i32(off), lengths, table, kp, vp, fd, key_weights=weights)
    kr = lps.rotary_rows(rows[:, :nq], k, pos, fd)[1]
    lps.attention_prompt_packed(q, kr, v, off)
    kept = [[kr[a:b].transpose(0, 1), v[a:b].transpose(0, 1)] for a, b in zip(off, off[1:])]

    tokens, positions = i32([3, 7]), i32(prompts)
    history, hist_len = torch.zeros(2, 64, device="cuda", dtype=torch.int32), torch.zeros(2, device="cuda", dtype=torch.int32)
    rep = torch.full((2,), 1.3, device="cuda")
    state = {}

    def step():
        lengths.add_(1)
        rows = embed[tokens.long()].view(2, nq + 2 * nkv, hd)
        q = lps.rotary_append_paged(rows[:, :nq], rows[:, nq:nq + nkv], rows[:, nq + nkv:], None, lengths, table, kp, vp, fd,
                                    positions=positions, key_weights=weights)
        o = lps.attention_paged_decode(q, kp, vp, table, lengths, key_weights=weights)
        logits = torch.matmul(o.view(2, -1).float(), head.float().T)
        history.scatter_(1, hist_len[:, None].long(), tokens[:, None])
        hist_len.add_(1)
        adjusted = lps.logits_adjust(logits, tokens=history, lengths=hist_len, repetition=rep)
        state.update(rows=rows, q=q, o=o, logits=logits, adjusted=adjusted)
        tokens.copy_(adjusted.argmax(-1).int())
        positions.add_(1)

    def check():
        was, n = state["was"], hist_len.tolist()[0]
        rows = embed[was.long()].view(2, nq + 2 * nkv, hd)
        at = positions - 1
        qr, qt = turn64(rows[:, :nq], at, f, False, 1.0)
        close(state["q"], qr, qt, "q")
        k = lps.rotary_rows(rows[:, :nq], rows[:, nq:nq + nkv], at, fd)[1]
        for b in range(2):
            kept[b][0] = torch.cat((kept[b][0], k[b][:, None]), 1)
            kept[b][1] = torch.cat((kept[b][1], rows[b, nq + nkv:][:, None]), 1)
            o, tol, _, _ = attend64(state["q"][b], kept[b][0], kept[b][1], scale)
            close(state["o"][b], o, tol, f"step {n}, sequence {b}")
        ref = adjust64(state["logits"], history, hist_len, None, rep, None, None, None, None, None)
        same_logits(state["adjusted"], *ref)
        assert torch.equal(tokens, state["adjusted"].argmax(-1).int())

    state["was"] = tokens.clone()
    step()
    check()
    saved = [x.clone() for x in (lengths, tokens, positions, history, hist_len, kp, vp, weights)]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    for x, y in zip((lengths, tokens, positions, history, hist_len, kp, vp, weights), saved):
        x.copy_(y)
    for _ in range(12):
        state["was"] = tokens.clone()
        graph.replay()
        check()
    # each step gave every head a weight of 1 in all, 13 steps and 4 heads a kv head
    for b in range(2):
        n = int(lengths[b])
        at, j = table[b].long()[torch.arange(n, device="cuda") // page], torch.arange(n, device="cuda") % page
        assert torch.allclose(weights[at, :, j].sum(0), torch.full((nkv,), 52.0, device="cuda"), rtol=1e-3)
    was_w = weights.clone()
    old = table.clone()
    new = lps.kv_pages_evict(kp, vp, weights, table, lengths, fresh, 48, 16)
    for b in range(2):
        n = int(lengths[b])
        rows_b = torch.arange(n, device="cuda")
        at, j = old[b].long()[rows_b // page], rows_b % page
        stay = [evicted(was_w[at, h, j].cpu().numpy(), n, 48, 16) for h in range(nkv)]
        kept[b] = [torch.stack([x[h, torch.from_numpy(stay[h]).cuda()] for h in range(nkv)]) for x in kept[b]]
        assert int(new[b]) == min(n, 48)
    table.fill_(-1)
    table[:, :8] = fresh
    lengths.copy_(new)
    for _ in range(10):
        state["was"] = tokens.clone()
        graph.replay()
        check()
    lps.cache_ops_status()
