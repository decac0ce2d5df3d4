"""The operators over a caller-owned cache on the GPU: packed-prompt attention, drafted-tree attention
and the cache's row moves, against the formula in 64 bits.

Tolerance of an attention output, per element, with u = eps / 2 of the element type, A = sum_j p_j |v_j|
and n keys:
  - the result is rounded once:                                             u |o|
  - each softmax weight is rounded to the element type before P.V:          u A
  - fp32: a score is a sum of head_dim products, off by at most head_dim 2^-24 S with S = scale sum |q k|,
    which moves p by that much relative, numerator and denominator: 2 head_dim 2^-24 S; the exponent's
    argument x = (s - m) log2 e is rounded twice, |x| <= 4 S: 8 S 2^-24; the hardware exp2 is off by
    2^-22; sums over n keys: 2 n 2^-24. Together c A.
  - fp16 only: weights below 2^-14 are off by 2^-25 each, with a denominator of at least 1: n 2^-25 max|v|.
The row moves copy bits: they are compared exactly.
"""
import math
import os

import numpy as np
import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def attend64(q, k, v, allowed, scale=None):
    """(o, bound on |error|): rows q [t, nq, hd] against keys k, v [n, nkv, hd] where allowed [t, n]; a row
    that sees nothing gives zeros. Values that no row of `allowed` sees take no part, whatever they hold."""
    t, nq, hd = q.shape
    n, nkv = k.shape[:2]
    u = torch.finfo(q.dtype).eps / 2
    scale = hd ** -0.5 if scale is None else scale
    qd = q.double().reshape(t, nkv, nq // nkv, hd)
    kd, vd = k.double(), v.double()
    used = allowed.any(0)
    kd = torch.where(used[:, None, None], kd, torch.zeros_like(kd))
    vd = torch.where(used[:, None, None], vd, torch.zeros_like(vd))
    s = torch.einsum("tghd,ngd->tghn", qd, kd) * scale
    mag = torch.einsum("tghd,ngd->tghn", qd.abs(), kd.abs()).amax(-1, keepdim=True) * scale if n else s.new_zeros(t, nkv, nq // nkv, 1)
    s = s.masked_fill(~allowed[:, None, None, :], -math.inf)
    top = s.amax(-1, keepdim=True) if n else s.new_full((t, nkv, nq // nkv, 1), -math.inf)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    o = torch.einsum("tghn,ngd->tghd", p, vd)
    a = torch.einsum("tghn,ngd->tghd", p, vd.abs())
    c = u + 2.0 ** -22 + (2 * hd + 8) * mag * 2.0 ** -24 + 2 * n * 2.0 ** -24
    tol = u * o.abs() + c * a
    if q.dtype == torch.float16:
        tol = tol + n * 2.0 ** -25 * (vd.abs().amax() if n else 0.0) + 2.0 ** -25
    return o.reshape(t, nq, hd), tol.reshape(t, nq, hd)


def check(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - ref).abs() - tol).max().item() if got.numel() else 0.0
    worst = ((got - ref).abs() / tol.clamp_min(1e-300)).max().item() if got.numel() else 0.0
    assert over <= 0, f"{what}: error is {worst:.3f} of its bound at worst"


def causal(n):
    return torch.ones(n, n, dtype=torch.bool, device="cuda").tril()


def offsets_of(lens, first=0):
    return np.concatenate([[first], first + np.cumsum(lens)]).astype(np.int32)


def check_prompt(q, k, v, off, out, scale=None):
    for s in range(len(off) - 1):
        lo, hi = int(off[s]), int(off[s + 1])
        if hi > lo:
            ref, tol = attend64(q[lo:hi], k[lo:hi], v[lo:hi], causal(hi - lo), scale)
            check(out[lo:hi], ref, tol, f"sequence {s} of {hi - lo} tokens")


# ---- packed prompts ------------------------------------------------------------------------------

LENS = {"one": [1], "ends": [127, 128, 129], "tiny": [2, 0, 1, 3, 0], "wide": [255, 257, 1, 300], "long": [1021, 5]}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (8, 2, 128), (3, 1, 128), (7, 1, 64), (4, 4, 128), (16, 1, 64)])
def test_prompt_matches_formula(nq, nkv, hd, dtype, lens):
    off = offsets_of(LENS[lens])
    n, g = int(off[-1]), _gen(11)
    q, k, v = (_randn(g, n, h, hd, dtype=DT[dtype]) for h in (nq, nkv, nkv))
    out = lps.attention_prompt_packed(q, k, v, off)
    check_prompt(q, k, v, off, out)
    again = lps.attention_prompt_packed(q, k, v, off.tolist())
    assert torch.equal(out, again)


@pytest.mark.parametrize("hd", [64, 128])
def test_prompt_strided_tensors(hd):
    """Column ranges of a fused projection, head-major tensors and a strided out: the dense call's bits."""
    nq, nkv, off, g = 8, 2, offsets_of([130, 7, 300]), _gen(5)
    n = int(off[-1])
    fused = _randn(g, n, (nq + 2 * nkv) * hd, dtype=torch.bfloat16)
    q = fused[:, : nq * hd].view(n, nq, hd)
    k = fused[:, nq * hd: (nq + nkv) * hd].view(n, nkv, hd)
    v = fused[:, (nq + nkv) * hd:].view(n, nkv, hd)
    ref = lps.attention_prompt_packed(q.contiguous(), k.contiguous(), v.contiguous(), off)
    check_prompt(q, k, v, off, ref)
    assert torch.equal(lps.attention_prompt_packed(q, k, v, off), ref)
    hm = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v)]
    out = torch.full((n, 2 * nq, hd), 7.0, device="cuda", dtype=torch.bfloat16)
    lps.attention_prompt_packed(*hm, off, out=out[:, ::2])
    assert torch.equal(out[:, ::2], ref) and (out[:, 1::2] == 7.0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("nq", [2, 8])
def test_prompt_unseen_values_change_nothing(bad, nq):
    """Tokens outside the offsets, other sequences and later tokens of the same sequence hold NaN or inf."""
    nkv, hd, g = 2, 128, _gen(3)
    off = np.array([3, 150, 150, 291], np.int32)
    q, k, v = (_randn(g, 300, h, hd, dtype=torch.bfloat16) for h in (nq, nkv, nkv))
    clean = lps.attention_prompt_packed(q, k, v, off, out=torch.full_like(q, 9.0))
    assert (clean[:3] == 9.0).all() and (clean[291:] == 9.0).all()
    check_prompt(q, k, v, off, clean)
    for at, lo, hi in [(slice(0, 3), 3, 291), (slice(291, 300), 3, 291), (slice(150, 291), 3, 150), (slice(100, 150), 3, 100),
                       (slice(100, 150), 150, 291), (slice(200, 201), 150, 200), (slice(149, 150), 3, 149)]:
        for which in (1, 2, 3):
            k2, v2 = k.clone(), v.clone()
            if which & 1:
                k2[at] = bad
            if which & 2:
                v2[at, :, 5:70:3] = bad
            got = lps.attention_prompt_packed(q, k2, v2, off, out=torch.full_like(q, 9.0))
            assert torch.equal(got[lo:hi], clean[lo:hi]), (at, which)
    # and a value that is seen arrives
    v2 = v.clone()
    v2[200, :, 7] = bad
    got = lps.attention_prompt_packed(q, k, v2, off)
    assert not torch.isfinite(got[200:291, :, 7]).any()
    if math.isinf(bad):
        assert (got[200:291, :, 7] == bad).all()
    others = [d for d in range(hd) if d != 7]
    assert torch.equal(got[150:291][:, :, others], clean[150:291][:, :, others])


@pytest.mark.parametrize("dtype", DT)
def test_prompt_extreme_scores(dtype):
    """Scores that grow along the keys, fall along them, are all equal, or reach the exponent's ends."""
    nq, nkv, hd, n = 4, 2, 64, 700
    for kind in ("rising", "falling", "equal", "sharp"):
        g = _gen(9)
        q, k, v = (_randn(g, n, h, hd, dtype=DT[dtype]) for h in (nq, nkv, nkv))
        if kind in ("rising", "falling"):
            q = q.abs()
            ramp = torch.linspace(0.0, 30.0, n, device="cuda")
            ramp = ramp if kind == "rising" else ramp.flip(0)
            k = (ramp[:, None, None].expand(n, nkv, hd) / 4).to(DT[dtype]).contiguous()
        elif kind == "equal":
            k = torch.zeros_like(k)
        else:
            q = (q.float() * 20).to(DT[dtype])
        off = offsets_of([n])
        check_prompt(q, k, v, off, lps.attention_prompt_packed(q, k, v, off))
    for scale in (1.0, 1e-4, 0.37):
        check_prompt(q, k, v, off, lps.attention_prompt_packed(q, k, v, off, scale=scale), scale)


def test_prompt_more_items_than_sms():
    """Enough tiles that every CTA takes over others, long and short ones, of one tile and of two."""
    off, g = offsets_of([1500, 33, 0, 700, 129, 64, 65, 1, 1000, 200]), _gen(17)
    n, nq, nkv, hd = int(off[-1]), 32, 8, 128
    q, k, v = (_randn(g, n, h, hd, dtype=torch.bfloat16) for h in (nq, nkv, nkv))
    out = lps.attention_prompt_packed(q, k, v, off)
    check_prompt(q, k, v, off, out)
    for _ in range(3):
        assert torch.equal(lps.attention_prompt_packed(q, k, v, off), out)
    # repaired values in one item leave the items around it as they were
    v2 = v.clone()
    v2[1400, 3, 40] = float("inf")
    got = lps.attention_prompt_packed(q, k, v2, off)
    assert (got[1400:1500, 12:16, 40] == float("inf")).all()
    got[1400:1500, 12:16, 40] = out[1400:1500, 12:16, 40]
    assert torch.equal(got, out)


@pytest.mark.parametrize("shift", [8, 16])
def test_prompt_output_alignment(shift):
    """Output rows on 16 and on 32 bytes: the same bits, and nothing between them touched."""
    off, g, nq, nkv, hd = offsets_of([70, 130]), _gen(19), 4, 2, 64
    n = int(off[-1])
    q, k, v = (_randn(g, n, h, hd, dtype=torch.float16) for h in (nq, nkv, nkv))
    ref = lps.attention_prompt_packed(q, k, v, off)
    buf = torch.full((n, nq * (hd + shift) + shift), 3.0, device="cuda", dtype=torch.float16)
    out = buf[:, shift:].view(n, nq, hd + shift)[:, :, :hd]
    lps.attention_prompt_packed(q, k, v, off, out=out)
    assert torch.equal(out, ref)
    out.fill_(3.0)
    assert (buf == 3.0).all()


def test_prompt_many_sequences():
    """More sequences than one launch carries."""
    rng = np.random.default_rng(1)
    off, g = offsets_of(rng.integers(0, 9, 700)), _gen(2)
    n = int(off[-1])
    q, k, v = (_randn(g, n, h, 64, dtype=torch.float16) for h in (4, 2, 2))
    check_prompt(q, k, v, off, lps.attention_prompt_packed(q, k, v, off))


# ---- drafted trees -------------------------------------------------------------------------------

def allowed_of(parents, pos, rows):
    m = torch.zeros(rows, pos + rows, dtype=torch.bool)
    m[:, :pos] = True
    for t in range(rows):
        a, seen = t, []
        while a >= 0:
            seen.append(pos + a)
            up = int(parents[a])
            if up < -1 or up >= a:
                seen = None
                break
            a = up
        if seen is None:
            m[t, :] = False
        else:
            m[t, seen] = True
    return m.cuda()


def random_parents(seed, batch, width):
    rng = np.random.default_rng(seed)
    p = np.empty((batch, width), np.int32)
    for t in range(width):
        p[:, t] = rng.integers(max(-1, t - 6), t, size=batch)
    return p


def check_tree(q, kc, vc, parents, pos, rows, out, before=None):
    for b in range(len(pos)):
        n = int(pos[b] + rows[b])
        ref, tol = attend64(q[b, :rows[b]], kc[b, :, :n].transpose(0, 1), vc[b, :, :n].transpose(0, 1),
                            allowed_of(parents[b], int(pos[b]), int(rows[b])))
        check(out[b, :rows[b]], ref, tol, f"sequence {b} (pos {pos[b]}, {rows[b]} rows)")
        if before is not None:
            assert torch.equal(out[b, rows[b]:], before[b, rows[b]:])


def tree_case(seed, pos, rows, width, nq, nkv, hd, dtype, extra=3):
    g = _gen(seed)
    pos, rows = np.array(pos, np.int32), np.array(rows, np.int32)
    ctx = int((pos + rows).max()) + extra
    q = _randn(g, len(pos), width, nq, hd, dtype=dtype)
    kc, vc = (_randn(g, len(pos), nkv, ctx, hd, dtype=dtype) for _ in range(2))
    return q, kc, vc, random_parents(seed, len(pos), width), pos, rows


TREES = {
    "decode": ([0, 1, 127, 128, 1000], [1, 1, 1, 1, 1], 1),
    "ragged": ([0, 100, 5, 640, 127], [17, 0, 1, 26, 2], 26),
    "full": ([0, 70, 1500], [64, 63, 64], 64),
    "edges": ([64, 128, 120, 255], [64, 64, 8, 1], 64),
    "longer": ([5000, 3], [31, 31], 31),
}


@pytest.mark.parametrize("tree", TREES)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("nq,nkv,hd", [(4, 2, 64), (8, 2, 128), (3, 1, 128), (14, 2, 64), (4, 4, 128), (16, 1, 128)])
def test_tree_matches_formula(nq, nkv, hd, dtype, tree):
    pos, rows, width = TREES[tree]
    q, kc, vc, parents, pos, rows = tree_case(21, pos, rows, width, nq, nkv, hd, DT[dtype])
    pd = torch.from_numpy(parents).cuda()
    for extra in (kc, vc):  # rows behind the drafts hold NaN
        for b in range(len(pos)):
            extra[b, :, pos[b] + rows[b]:] = float("nan")
    before = torch.full_like(q, 5.0)
    out = lps.attention_tree_verify(q, kc, vc, pd, pos, rows, out=before.clone())
    check_tree(q, kc, vc, parents, pos, rows, out, before)
    again = lps.attention_tree_verify(q, kc, vc, pd, pos.tolist(), rows.tolist(), out=before.clone())
    assert torch.equal(out, again)


def test_tree_of_one_chain_is_the_prompt():
    """A chain of drafts over an empty cache sees what the tokens of a prompt see."""
    nq, nkv, hd, n, g = 8, 2, 128, 50, _gen(4)
    q, k, v = (_randn(g, n, h, hd, dtype=torch.bfloat16) for h in (nq, nkv, nkv))
    off = offsets_of([n])
    kc, vc = (torch.full((1, nkv, n, hd), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lps.kv_rows_append(k, v, off, kc, vc, [0])
    chain = torch.arange(-1, n - 1, device="cuda", dtype=torch.int32)[None]
    out = lps.attention_tree_verify(q[None], kc, vc, chain, [0], [n])
    check_prompt(q, k, v, off, out[0])
    check_prompt(q, k, v, off, lps.attention_prompt_packed(q, k, v, off))


@pytest.mark.parametrize("pos", [0, 90, 700])
def test_tree_unseen_drafts_change_nothing(pos):
    """A draft that another one does not descend from may hold NaN or inf: nothing of it arrives."""
    q, kc, vc, _, p, r = tree_case(8, [pos], [6], 6, 8, 2, 128, torch.bfloat16)
    parents = np.array([[-1, -1, 0, 1, 2, -1]], np.int32)  # 0-2-4 and 1-3, and 5 alone
    pd = torch.from_numpy(parents).cuda()
    clean = lps.attention_tree_verify(q, kc, vc, pd, p, r)
    check_tree(q, kc, vc, parents, p, r, clean)
    for bad in (float("nan"), float("inf")):
        k2, v2 = kc.clone(), vc.clone()
        k2[:, :, pos + 1] = bad
        v2[:, :, pos + 1] = bad
        v2[:, :, pos + 3, 11] = -bad
        got = lps.attention_tree_verify(q, k2, v2, pd, p, r)
        assert torch.equal(got[:, [0, 2, 4, 5]], clean[:, [0, 2, 4, 5]])
        assert not torch.isfinite(got[:, [1, 3]]).any()


@pytest.mark.parametrize("hd", [64, 128])
def test_far_larger_scores_of_other_rows_change_no_bit(hd):
    """Later tokens of a prompt and another branch's drafts with finite keys whose scores are far above a row's
    own: the row has the bits that it has without them, rows that see them beside it in its tile or not."""
    nq, nkv, n, g = 8, 2, 400, _gen(12)
    q, k, v = (_randn(g, n, h, hd, dtype=torch.bfloat16) for h in (nq, nkv, nkv))
    clean = lps.attention_prompt_packed(q, k, v, [0, n])
    for at in (135, 150, 259, 300):
        k2 = k.clone()
        k2[at:] *= 40
        got = lps.attention_prompt_packed(q, k2, v, [0, n])
        assert torch.equal(got[:at], clean[:at]) and not torch.equal(got[at:], clean[at:])
        check_prompt(q, k2, v, np.array([0, n], np.int32), got)
    parents = np.array([[-1, -1, 0, 1, 2, -1]], np.int32)  # 0-2-4 and 1-3, and 5 alone
    pd = torch.from_numpy(parents).cuda()
    for pos in (5, 300, 2000):
        tq, kc, vc, _, p, r = tree_case(9, [pos], [6], 6, nq, nkv, hd, torch.bfloat16)
        kc[:, :, :pos] *= 0.05
        clean = lps.attention_tree_verify(tq, kc, vc, pd, p, r)
        kc[:, :, pos + 1] *= 40
        got = lps.attention_tree_verify(tq, kc, vc, pd, p, r)
        assert torch.equal(got[:, [0, 2, 4, 5]], clean[:, [0, 2, 4, 5]]) and not torch.equal(got[:, [1, 3]], clean[:, [1, 3]])
        check_tree(tq, kc, vc, parents, p, r, got)


def test_tree_bad_parents_give_zeros():
    q, kc, vc, _, p, r = tree_case(8, [200, 3], [8, 8], 8, 4, 2, 64, torch.float16)
    parents = np.array([[-1, 0, 5, 2, 1, -2, 6, 3], [-1, 99, 1, 0, -2147483648, 2147483647, 3, 0]], np.int32)
    out = lps.attention_tree_verify(q, kc, vc, torch.from_numpy(parents).cuda(), p, r)
    check_tree(q, kc, vc, parents, p, r, out)
    assert (out[0, [2, 3, 5, 6, 7]] == 0).all() and (out[1, [1, 2, 4, 5]] == 0).all()
    assert (out[0, [0, 1, 4]] != 0).any() and (out[1, [0, 3, 6, 7]] != 0).any()


def test_tree_strided_q_and_out():
    q, kc, vc, parents, p, r = tree_case(6, [300, 10], [9, 4], 9, 8, 2, 64, torch.bfloat16)
    pd = torch.from_numpy(parents).cuda()
    ref = lps.attention_tree_verify(q, kc, vc, pd, p, r, out=torch.zeros_like(q))
    wide = torch.zeros(2, 9, 8 * 64 + 64, device="cuda", dtype=torch.bfloat16)
    wide[:, :, : 8 * 64] = q.view(2, 9, 512)
    out = torch.zeros(9, 8, 2, 64, device="cuda", dtype=torch.bfloat16).permute(2, 0, 1, 3)
    lps.attention_tree_verify(wide[:, :, :512].view(2, 9, 8, 64), kc, vc, pd, p, r, out=out)
    assert torch.equal(out, ref)


@pytest.mark.parametrize("nq,nkv,width", [(8, 2, 16), (16, 4, 64), (5, 1, 33)])
def test_tree_of_many_sequences(nq, nkv, width):
    """More clusters than run at once, of very different lengths, and sequences without drafts among them."""
    rng = np.random.default_rng(6)
    batch = 256 if nq == 8 else 90
    pos = np.concatenate([[3000, 2900], rng.integers(0, 500, batch - 2)]).astype(np.int32)
    rows = rng.integers(0, width + 1, batch).astype(np.int32)
    q, kc, vc, parents, pos, rows = tree_case(23, pos, rows, width, nq, nkv, 64, torch.bfloat16)
    out = lps.attention_tree_verify(q, kc, vc, torch.from_numpy(parents).cuda(), pos, rows, out=torch.full_like(q, 2.0))
    check_tree(q, kc, vc, parents, pos, rows, out, torch.full_like(q, 2.0))


def test_tree_scores_far_apart():
    """One key far above all others, in the first, a middle and the last part of the cache: every part but
    one has weights next to nothing in the join."""
    for at in (0, 2000, 4090):
        q, kc, vc, parents, pos, rows = tree_case(25, [4095], [3], 3, 4, 2, 128, torch.bfloat16)
        kc[:, :, at] = (q[:, 0, :, :].view(1, 2, 2, 128).float().mean(2) * 8).to(torch.bfloat16)
        out = lps.attention_tree_verify(q, kc, vc, torch.from_numpy(parents).cuda(), pos, rows)
        check_tree(q, kc, vc, parents, pos, rows, out)


def test_tree_cache_past_32_bits():
    """A cache of more than 2^32 bytes and 2^31 elements, read at its last head and sequence."""
    batch, nkv, ctx, hd = 2, 8, 1 << 20, 128
    kc, vc = (torch.empty(batch, nkv, ctx, hd, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pos, rows = np.array([3, ctx - 5], np.int32), np.array([2, 5], np.int32)
    g = _gen(1)
    q = _randn(g, batch, 5, nkv, hd, dtype=torch.bfloat16)
    for c in (kc, vc):
        c[1].normal_(generator=g)
        c[0, :, :64].normal_(generator=g)
    parents = random_parents(3, batch, 5)
    out = lps.attention_tree_verify(q, kc, vc, torch.from_numpy(parents).cuda(), pos, rows, out=torch.zeros_like(q))
    for h in (0, nkv - 1):  # head by head: the reference's doubles are large
        heads = slice(h, h + 1)
        check_tree(q[:, :, heads], kc[:, heads], vc[:, heads], parents, pos, rows, out[:, :, heads])


def test_tree_streams_and_graphs():
    """On a stream of its own, captured and replayed with other values in the same buffers, and two captured
    graphs replayed on two streams at once: the eager call's bits."""
    cases = [tree_case(30 + i, [2000 + i, 77], [13, 26], 26, 32, 8, 128, torch.bfloat16) for i in range(2)]
    side = torch.cuda.Stream()
    refs, graphs, outs, ins = [], [], [], []
    for q, kc, vc, parents, p, r in cases:
        pd = torch.from_numpy(parents).cuda()
        ref = lps.attention_tree_verify(q, kc, vc, pd, p, r, out=torch.zeros_like(q))
        check_tree(q, kc, vc, parents, p, r, ref)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = lps.attention_tree_verify(q, kc, vc, pd, p, r, out=torch.zeros_like(q))
        torch.cuda.synchronize()
        assert torch.equal(other, ref)
        out, qb = torch.zeros_like(q), torch.zeros_like(q)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lps.attention_tree_verify(qb, kc, vc, pd, p, r, out=out)
        qb.copy_(q)
        refs.append(ref), graphs.append(graph), outs.append(out), ins.append((qb, pd, kc, vc))
    torch.cuda.synchronize()
    for _ in range(5):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], refs[0]) and torch.equal(outs[1], refs[1])


def test_prompt_and_moves_in_a_graph():
    """The other operators captured and replayed on new values: the eager calls' bits."""
    nq, nkv, hd, off, ctx = 8, 2, 64, offsets_of([100, 40, 257]), 300
    n = int(off[-1])
    q, k, v = (torch.zeros(n, h, hd, device="cuda", dtype=torch.bfloat16) for h in (nq, nkv, nkv))
    kc, vc = (torch.zeros(2, 3, nkv, ctx, hd, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    path = torch.zeros(3, 4, device="cuda", dtype=torch.int32)
    taken = torch.zeros(3, device="cuda", dtype=torch.int32)

    def step(out):
        lps.attention_prompt_packed(q, k, v, off, out=out)
        lps.kv_rows_append(k, v, off, kc[1], vc[1], [0, 10, 43])
        lps.kv_rows_accept(kc, vc, [100, 50, 296], path, taken)
        return out

    out, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    step(out)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(out)
    for seed in (1, 2):
        g = _gen(seed)
        for t in (q, k, v, kc, vc):
            t.normal_(generator=g)
        path.copy_(torch.tensor([[0, 2, 3, 0], [1, 3, 0, 0], [3, 0, 0, 0]], dtype=torch.int32))
        taken.copy_(torch.tensor([3, 2, 1], dtype=torch.int32))
        before = kc.clone(), vc.clone()
        want = step(torch.zeros_like(q)).clone(), kc.clone(), vc.clone()
        kc.copy_(before[0]), vc.copy_(before[1]), out.zero_()
        graph.replay()
        for got, w in zip((out, kc, vc), want):
            assert torch.equal(got, w)


def test_calls_from_two_threads():
    """Two host threads, each on a stream of its own: each call's own result, and messages that stay apart."""
    import threading
    cases, got, errors = [tree_case(50 + i, [900 + 300 * i, 20], [9, 26], 26, 8, 2, 128, torch.bfloat16) for i in range(2)], {}, []
    refs = [lps.attention_tree_verify(*c[:3], torch.from_numpy(c[3]).cuda(), c[4], c[5], out=torch.zeros_like(c[0])) for c in cases]
    pds = [torch.from_numpy(c[3]).cuda() for c in cases]
    torch.cuda.synchronize()

    def work(i):
        try:
            q, kc, vc, _, p, r = cases[i]
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(50):
                    got[i] = lps.attention_tree_verify(q, kc, vc, pds[i], p, r, out=torch.zeros_like(q))
                try:
                    lps.attention_tree_verify(q, kc, vc, pds[i], [-1 - i, 0], r)
                    errors.append("not refused")
                except lps.LpsError as e:
                    assert e.code == lps.LPS_EINVAL
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported by the main thread
            errors.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for i in range(2):
        assert torch.equal(got[i], refs[i])


# ---- row moves -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("nkv,hd", [(1, 64), (3, 128), (8, 64)])
def test_append_writes_its_rows_and_no_others(nkv, hd, dtype):
    lens, start, ctx = [5, 0, 1, 200, 37], [0, 300, 299, 100, 263], 300
    off, g = offsets_of(lens, first=2), _gen(7)
    fused = _randn(g, int(off[-1]) + 4, 2 * nkv * hd, dtype=DT[dtype])
    fused[9, :40] = float("nan")  # bits are moved, whatever they mean
    k, v = fused[:, : nkv * hd].view(-1, nkv, hd), fused[:, nkv * hd:].view(-1, nkv, hd)
    kc, vc = (_randn(g, len(lens), nkv, ctx, hd, dtype=DT[dtype]) for _ in range(2))
    want = [kc.clone(), vc.clone()]
    for s, n in enumerate(lens):
        for w, t in zip(want, (k, v)):
            w[s, :, start[s]:start[s] + n] = t[off[s]:off[s + 1]].transpose(0, 1)
    lps.kv_rows_append(k, v, off, kc, vc, start)
    for got, w in zip((kc, vc), want):
        assert torch.equal(got.view(torch.int16), w.view(torch.int16))
    hm = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in (k, v)]
    kc2, vc2 = want[0].clone().zero_(), want[1].clone().zero_()
    lps.kv_rows_append(*hm, off, kc2, vc2, start)
    for s, n in enumerate(lens):
        assert torch.equal(kc2[s, :, start[s]:start[s] + n].view(torch.int16), kc[s, :, start[s]:start[s] + n].view(torch.int16))


def test_append_many_sequences():
    rng, g = np.random.default_rng(4), _gen(4)
    lens = rng.integers(0, 5, 600)
    off, start = offsets_of(lens), rng.integers(0, 4, 600).astype(np.int32)
    k, v = (_randn(g, int(off[-1]), 2, 64, dtype=torch.float16) for _ in range(2))
    kc, vc = (torch.zeros(600, 2, 8, 64, device="cuda", dtype=torch.float16) for _ in range(2))
    lps.kv_rows_append(k, v, off, kc, vc, start)
    want = torch.zeros_like(kc)
    for s in range(600):
        want[s, :, start[s]:start[s] + lens[s]] = k[off[s]:off[s + 1]].transpose(0, 1)
    assert torch.equal(kc, want)


@pytest.mark.parametrize("layers,nkv,hd", [(1, 8, 128), (3, 1, 64), (2, 5, 64)])
def test_accept_moves_paths_in_place(layers, nkv, hd):
    """Paths of every kind: none, one row, the identity, the last rows, a full one; and paths that break the
    rules (too long, descending, repeated, negative, past the width or the cache): those change nothing."""
    width, ctx, g = 64, 120, _gen(13)
    paths = [[], [0], [63], list(range(64)), list(range(8, 64)), [1, 2, 5, 6, 40], [0, 2, 1], [3, 3], [-1, 0], [2, 64],
             [5, 30], list(range(1, 64, 2)), [4]]
    count = [len(p) for p in paths]
    count[-1] = 65  # more than the width
    pos = np.array([0, 5, 50, 56, 1, 20, 9, 9, 9, 9, 100, 3, 7], np.int32)  # [10]: row 130 of 120
    good = [True] * 6 + [False] * 5 + [True, False]
    batch = len(paths)
    path = torch.full((batch, width), 7, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    kc, vc = (_randn(g, layers, batch, nkv, ctx, hd, dtype=torch.bfloat16) for _ in range(2))
    want = [kc.clone(), vc.clone()]
    for w, c in zip(want, (kc, vc)):
        for b, p in enumerate(paths):
            for i, x in enumerate(p if good[b] else []):
                w[:, b, :, pos[b] + i] = c[:, b, :, pos[b] + x]
    lps.kv_rows_accept(kc, vc, pos, path.cuda(), torch.tensor(count, dtype=torch.int32, device="cuda"))
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])


# ---- together ------------------------------------------------------------------------------------

def test_prompt_append_verify_accept_decode():
    """A speculative step as a server makes it: prompts attended and stored, a tree of drafts stored and
    verified, the accepted path kept, and the next token decoded over the cache by the framework's decode
    attention and by the tree of one row."""
    nq, nkv, hd, ctx, width, g = 8, 2, 128, 512, 12, _gen(40)
    lens = [300, 1, 129]
    off = offsets_of(lens)
    bf = torch.bfloat16
    q, k, v = (_randn(g, int(off[-1]), h, hd, dtype=bf) for h in (nq, nkv, nkv))
    kc, vc = (torch.full((3, nkv, ctx, hd), float("nan"), device="cuda", dtype=bf) for _ in range(2))
    check_prompt(q, k, v, off, lps.attention_prompt_packed(q, k, v, off))
    lps.kv_rows_append(k, v, off, kc, vc, [0, 0, 0])

    rows, parents = np.array([12, 7, 9], np.int32), random_parents(2, 3, width)
    doff = offsets_of(rows)
    dk, dv = (_randn(g, int(doff[-1]), nkv, hd, dtype=bf) for _ in range(2))
    lps.kv_rows_append(dk, dv, doff, kc, vc, lens)
    dq = _randn(g, 3, width, nq, hd, dtype=bf)
    pd = torch.from_numpy(parents).cuda()
    out = lps.attention_tree_verify(dq, kc, vc, pd, lens, rows)
    check_tree(dq, kc, vc, parents, np.array(lens), rows, out)

    path = torch.zeros(3, width, dtype=torch.int32)
    taken = []
    for b in range(3):  # the chain that ends in the last draft
        a, chain = int(rows[b]) - 1, []
        while a >= 0:
            chain.insert(0, a)
            a = int(parents[b, a])
        path[b, :len(chain)] = torch.tensor(chain, dtype=torch.int32)
        taken.append(len(chain))
    kept = [torch.cat([kc[b, :, :lens[b]], kc[b, :, lens[b] + path[b, :taken[b]].long().cuda()]], 1) for b in range(3)]
    lps.kv_rows_accept(kc, vc, lens, path.cuda(), torch.tensor(taken, dtype=torch.int32, device="cuda"))
    pos = [n + t for n, t in zip(lens, taken)]
    for b in range(3):
        assert torch.equal(kc[b, :, :pos[b]], kept[b])

    # the next token: its own row appended, then one row over the cache
    one = offsets_of([1, 1, 1])
    nk, nv = (_randn(g, 3, nkv, hd, dtype=bf) for _ in range(2))
    lps.kv_rows_append(nk, nv, one, kc, vc, pos)
    nqr = _randn(g, 3, 1, nq, hd, dtype=bf)
    root = np.full((3, 1), -1, np.int32)
    got = lps.attention_tree_verify(nqr, kc, vc, torch.from_numpy(root).cuda(), pos, [1, 1, 1])
    check_tree(nqr, kc, vc, root, np.array(pos), np.array([1, 1, 1]), got)
    L, f32 = _capi.load(), nqr.float().view(3, nq * hd).contiguous()
    ref = torch.empty_like(f32)
    cpos = np.array(pos, np.int32)
    stream = torch.cuda.current_stream().cuda_stream
    assert L.attention_decode_noalloc(f32.data_ptr(), kc.data_ptr(), vc.data_ptr(), ref.data_ptr(), 3, nq, nkv, hd, ctx,
                                      cpos.ctypes.data, stream) == 0
    assert L.attention_decode_noalloc_status(stream) == 0
    tol = attend64(nqr[0], kc[0, :, :pos[0] + 1].transpose(0, 1), vc[0, :, :pos[0] + 1].transpose(0, 1),
                   torch.ones(1, pos[0] + 1, dtype=torch.bool, device="cuda"))[1]
    assert ((got[0].double().view(-1) - ref[0].double()).abs() <= 2 * tol.view(-1)).all()


def test_host_integers_of_every_kind():
    """Offsets as a list, a tuple, arrays of several types and strides, and CPU tensors: the same bits; what is
    not a row of integers that fit 32 bits is refused."""
    g, nq, nkv, hd = _gen(3), 4, 2, 64
    q, k, v = (_randn(g, 50, h, hd, dtype=torch.bfloat16) for h in (nq, nkv, nkv))
    ref = lps.attention_prompt_packed(q, k, v, [0, 20, 50])
    wide = np.array([0, 7, 20, 7, 50, 7], np.int32)
    for off in ((0, 20, 50), np.array([0, 20, 50]), np.array([0, 20, 50], np.int32), np.array([0, 20, 50], np.uint8), wide[::2],
                np.array([50, 20, 0])[::-1], torch.tensor([0, 20, 50]), torch.tensor([0, 20, 50], dtype=torch.int32),
                [np.int64(0), 20, np.int16(50)], range(0, 51, 10)):
        got = lps.attention_prompt_packed(q, k, v, off)
        assert torch.equal(got, ref) or isinstance(off, range)
    many = [0] * 300 + [50]
    assert torch.equal(lps.attention_prompt_packed(q, k, v, many), lps.attention_prompt_packed(q, k, v, [0, 50]))
    for off in ([0.0, 50.0], np.array([0.0, 50.0]), np.array([False, True]), np.array([[0, 50]]), [0, 2**31], np.array([0, 2**40]),
                [], torch.tensor([0, 50]).cuda(), ["0", "50"], np.array(50)):
        with pytest.raises(ValueError):
            lps.attention_prompt_packed(q, k, v, off)
    with pytest.raises(TypeError):
        lps.attention_prompt_packed(q, k, v, None)
    with pytest.raises(TypeError):
        lps.attention_prompt_packed(q, k, v, [0, 50], scale="1")
    with torch.no_grad():
        assert torch.equal(lps.attention_prompt_packed(q.clone().requires_grad_(), k, v, [0, 20, 50]), ref)
    empty = lps.attention_prompt_packed(q[:0], k[:0], v[:0], [0, 0])
    assert empty.shape == (0, nq, hd)
    assert lps.attention_prompt_packed(q, k, v, [0]).shape == q.shape


class _Emptying:
    """An integer whose __index__ empties the list that holds it."""

    def __init__(self, values):
        self.values = values

    def __index__(self):
        self.values.clear()
        return 0


def test_host_integers_that_change_while_they_are_read():
    q = torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    values = [0] * 40
    values[0] = _Emptying(values)
    with pytest.raises(ValueError, match="changed"):
        lps.attention_prompt_packed(q, q, q, values)


_FIRST_CALL = """
import torch, layer_pipeline_staged_gb300 as lps
def t(*shape): return torch.randn(*shape, device="cuda", generator=gen).to(torch.bfloat16)
gen = torch.Generator("cuda").manual_seed(5)
q, k, v, kc, vc, tq = t(70, 8, 128), t(70, 2, 128), t(70, 2, 128), t(1, 2, 400, 128), t(1, 2, 400, 128), t(1, 3, 8, 128)
par = torch.tensor([[-1, 0, -1]], dtype=torch.int32, device="cuda")
path, taken = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
po, to = torch.zeros_like(q), torch.zeros_like(tq)
def step():
    lps.attention_prompt_packed(q, k, v, [0, 30, 70], out=po)
    lps.kv_rows_append(k, v, [0, 70], kc, vc, [200])
    lps.attention_tree_verify(tq, kc, vc, par, [300], [3], out=to)
    lps.kv_rows_accept(kc, vc, [300], path, taken)
first = kc.clone(), vc.clone()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
assert not po.any() and torch.equal(kc, first[0])
graph.replay()
got = po.clone(), to.clone(), kc.clone(), vc.clone()
kc.copy_(first[0]), vc.copy_(first[1]), po.zero_(), to.zero_()
step()
assert all(torch.equal(a, b) for a, b in zip(got, (po, to, kc, vc))) and po.any() and to.any()
print("same")
"""


def test_first_calls_are_captured():
    """A process whose first calls are made during a capture: what the library sets up once does not break it."""
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    run = subprocess.run([sys.executable, "-c", _FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=240)
    assert run.returncode == 0 and run.stdout.strip() == "same", run.stderr[-2000:]


# ---- refusals with real buffers --------------------------------------------------------------------

def test_refusals_of_tensors():
    q, k = torch.zeros(4, 4, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(4, 2, 64, device="cuda", dtype=torch.bfloat16)
    for bad in (lambda: lps.attention_prompt_packed(q.float(), k.float(), k.float(), [0, 4]),
                lambda: lps.attention_prompt_packed(q, k, k.half(), [0, 4]),
                lambda: lps.attention_prompt_packed(q, k, k[:3], [0, 4]),
                lambda: lps.attention_prompt_packed(q, k, k, [0, 5]),
                lambda: lps.attention_prompt_packed(q, k, k, [0.0, 4.0]),
                lambda: lps.attention_prompt_packed(q, k, k.cpu(), [0, 4]),
                lambda: lps.attention_prompt_packed(q.requires_grad_(), k, k, [0, 4]),
                lambda: lps.attention_prompt_packed(q.detach().transpose(1, 2).contiguous().transpose(1, 2), k, k, [0, 4])):
        with pytest.raises(ValueError):
            bad()
    q = q.detach()
    for bad in (lambda: lps.attention_prompt_packed(q, k, k, [0, 3, 2]), lambda: lps.attention_prompt_packed(q, k, k, [-1, 3]),
                lambda: lps.attention_prompt_packed(q[:, :3], k, k, [0, 4]),
                lambda: lps.attention_prompt_packed(q, k[:, :1].expand(4, 2, 64), k, [0, 4]),
                lambda: lps.attention_prompt_packed(q, k, k, [0, 4], scale=-1.0)):
        with pytest.raises(lps.LpsError) as e:
            bad()
        assert e.value.code == lps.LPS_EINVAL
    tq, kc = torch.zeros(2, 3, 4, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(2, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    par = torch.full((2, 3), -1, device="cuda", dtype=torch.int32)
    for bad in (lambda: lps.attention_tree_verify(tq, kc, kc, par.long(), [1, 1], [1, 1]),
                lambda: lps.attention_tree_verify(tq, kc, kc, par[:, :2], [1, 1], [1, 1]),
                lambda: lps.attention_tree_verify(tq, kc, kc, par, [1], [1, 1]),
                lambda: lps.attention_tree_verify(tq, kc.transpose(1, 2), kc, par, [1, 1], [1, 1]),
                lambda: lps.attention_tree_verify(tq, kc, kc, par, [1, 2**40], [1, 1])):
        with pytest.raises(ValueError):
            bad()
    for pos, rows in (([1, 14], [1, 3]), ([-1, 0], [1, 1]), ([0, 0], [4, 1])):
        with pytest.raises(lps.LpsError):
            lps.attention_tree_verify(tq, kc, kc, par, pos, rows)
    for vc, start in ((kc.clone(), [0, 15]), (kc, [0, 0])):
        with pytest.raises(lps.LpsError):
            lps.kv_rows_append(k, k, [0, 2, 4], kc, vc, start)
    assert _capi.load().cache_ops_status(torch.cuda.current_stream().cuda_stream) == lps.LPS_OK
