"""Attention of one token a sequence over a paged cache, on the GPU, against the formula in 64 bits.

Tolerance of an output, per element, with u = eps / 2 of the element type, A = sum_j p_j |v_j| and n keys:
  - the result is rounded once:                                                    u |o|
  - a weight enters P.V as hi + lo: hi is cut to 8 bits (fp16: 11), lo rounded to as many: off by 2^-7 2^-9 = 2^-16 of
    the weight (fp16: 2^-10 2^-11 = 2^-21), and 2^-24 for the part that keeps lo from being 0; fp16 weights, 2^7
    times larger (and the base at most the maximum), end at 2^-25: n 2^-32 max|v|
  - fp32, as the tensor core sums it (an addition may cut at 2^-23 instead of rounding at 2^-24, and aligned products
    once more: 4 times 2^-24): a score is a sum of hd products, off by 4 hd 2^-24 S with S = scale sum |q k|, which
    moves p by that much, in the numerator and the denominator: 8 hd 2^-24 S; the exponent's argument is rounded three
    times at up to 4 S (fp16: at up to 14 more): 3 (8 S + 14) 2^-24; exp2 2^-22 twice; sums over n keys: 8 n 2^-24. Together c A.
A key's weight is a sum over the group's heads of p: off by (c + group 2^-24) of it.
"""
import math

import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi

torch = pytest.importorskip("torch")
from paged import DT, Paged, gen, i32, randn  # noqa: E402

pytestmark = pytest.mark.gpu


def attend64(q, k, v, scale=None):
    """(o, bound, weights of the keys, their bound) of q [nq, hd] against k, v [nkv, n, hd]."""
    nq, hd = q.shape
    nkv, n, _ = k.shape
    group = nq // nkv
    if n == 0:
        return torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64), None, None
    scale = hd ** -0.5 if scale is None else scale
    qd, kd, vd = q.double().view(nkv, group, hd), k.double(), v.double()
    s = torch.einsum("ghd,gnd->ghn", qd, kd) * scale
    mag = torch.einsum("ghd,gnd->ghn", qd.abs(), kd.abs()).amax(-1, keepdim=True) * scale
    p = torch.softmax(s, -1)
    o, a = torch.einsum("ghn,gnd->ghd", p, vd), torch.einsum("ghn,gnd->ghd", p, vd.abs())
    u, half = torch.finfo(q.dtype).eps / 2, q.dtype == torch.float16
    c32 = 2 * 2.0 ** -22 + (8 * hd * mag + 3 * (8 * mag + 14) + 8 * n) * 2.0 ** -24
    tol = u * o.abs() + (1 + u) * ((2.0 ** -21 if half else 2.0 ** -16) + 2.0 ** -24 + c32) * a
    if half:
        tol = tol + n * 2.0 ** -32 * vd.abs().amax() + 2.0 ** -25  # and the result's own subnormals
    w = p.sum(1)
    return o.view(nq, hd), tol.view(nq, hd), w, ((c32 + group * 2.0 ** -24) * p).sum(1)


def close(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if got.numel():
        worst = ((got - ref).abs() / tol.clamp_min(1e-300)).max().item()
        assert ((got - ref).abs() <= tol).all(), f"{what}: error is {worst:.3f} of its bound at worst"


def check(c, q, out, weights=None, old=None, decay=1.0, scale=None):
    for b, n in enumerate(c.lens):
        o, tol, w, wtol = attend64(q[b], c.k[b], c.v[b], scale)
        close(out[b], o, tol, f"sequence {b} of {n}")
        if weights is not None and n:
            was = 0.0 if old is None else decay * c.get(b, old.unsqueeze(-1)).squeeze(-1).double()
            new = c.get(b, weights.unsqueeze(-1)).squeeze(-1)
            close(new, was + w, wtol + 2.0 ** -23 * (was + w), f"weights of sequence {b}")


LENS = {"one": [1], "ends": [63, 64, 65, 127, 128, 129], "few": [0, 1, 2, 0, 16, 15, 17], "wide": [1000, 3, 0, 517],
        "long": [9001]}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("nq,nkv,hd,page", [(4, 2, 64, 16), (32, 8, 128, 16), (3, 1, 128, 24), (7, 1, 64, 8), (4, 4, 128, 64),
                                            (16, 1, 64, 128), (9, 1, 128, 32), (48, 12, 128, 40)])
def test_matches_formula(nq, nkv, hd, page, dtype, lens):
    c = Paged(LENS[lens], nkv, hd, page, DT[dtype])
    q = randn(gen(2), len(c.lens), nq, hd, dtype=DT[dtype])
    out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    check(c, q, out)
    weights = torch.full((c.pages, nkv, page), float("nan"), device="cuda")
    again = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, key_weights=weights, decay=0.0)
    assert torch.equal(out, again)  # the weights change no bit of the output
    check(c, q, out, weights)
    rows = sum(c.lens) * nkv
    assert int(torch.isfinite(weights).sum()) == rows  # and no other entry is written
    lps.cache_ops_status()


@pytest.mark.parametrize("decay", [1.0, 0.5, 0.0])
def test_weights_accumulate(decay):
    c = Paged([300, 0, 65, 1], 2, 64, 16, torch.bfloat16)
    q = randn(gen(3), 4, 8, 64, dtype=torch.bfloat16)
    old = torch.rand(c.pages, 2, 16, generator=gen(4), device="cuda")
    new = old.clone()
    out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, key_weights=new, decay=decay)
    check(c, q, out, new, old, decay)
    seen = torch.zeros(c.pages, 2, 16, dtype=torch.bool, device="cuda")
    for b in range(4):
        page, row = c.at(b)
        seen[page, :, row] = True
    assert torch.equal(new[~seen], old[~seen])


@pytest.mark.parametrize("hd", [64, 128])
def test_strided_tensors(hd):
    """q as a column range of a fused projection and out as every second head: the dense call's bits."""
    c = Paged([70, 500], 2, hd, 16, torch.bfloat16)
    fused = randn(gen(5), 2, 12, hd, dtype=torch.bfloat16)
    q = fused[:, 2:10]
    ref = lps.attention_paged_decode(q.contiguous(), c.kp, c.vp, c.table, c.lengths)
    check(c, q, ref)
    assert torch.equal(lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths), ref)
    out = torch.full((2, 16, hd), 7.0, device="cuda", dtype=torch.bfloat16)
    assert lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, out=out[:, ::2]).data_ptr() == out.data_ptr()
    assert torch.equal(out[:, ::2], ref) and (out[:, 1::2] == 7.0).all()


def test_sequences_that_break_the_rules_give_zeros_and_harm_nobody():
    c = Paged([100, 200, 300, 64, 20], 2, 64, 16, torch.bfloat16)
    q = randn(gen(6), 5, 4, 64, dtype=torch.bfloat16)
    room = c.table.shape[1] * 16
    for bad in (-1, room + 1, 2 ** 31 - 1, -2 ** 31):
        out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, i32([100, bad, 300, 64, bad]))
        assert (out[[1, 4]] == 0).all()
        for b in (0, 2, 3):
            o, tol, _, _ = attend64(q[b], c.k[b], c.v[b])
            close(out[b], o, tol, f"sequence {b} beside length {bad}")
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):  # pages that are none: their rows are not seen
        table = c.table.clone()
        table[2, 3:5] = bad
        table[3] = bad
        weights = torch.full((c.pages, 2, 16), 5.0, device="cuda")
        out = lps.attention_paged_decode(q, c.kp, c.vp, table, c.lengths, key_weights=weights, decay=0.0)
        keep = torch.ones(300, dtype=torch.bool, device="cuda")
        keep[48:80] = False
        o, tol, w, wtol = attend64(q[2], c.k[2][:, keep], c.v[2][:, keep])
        close(out[2], o, tol, f"holes of page {bad}")
        close(c.get(2, weights.unsqueeze(-1)).squeeze(-1)[:, keep], w, wtol + 2.0 ** -23 * w, "weights beside the holes")
        assert (out[3] == 0).all()
        page, row = c.at(3)
        assert (weights[page, :, row] == 5.0).all()
    lps.cache_ops_status()


@pytest.mark.parametrize("batch,longest", [(1, 64), (5, 640), (300, 200), (1024, 90)])
def test_shares_of_many_and_of_few(batch, longest):
    """Fewer tiles than CTAs, and CTAs with many short sequences each."""
    lens = torch.randint(0, longest + 1, (batch,), generator=torch.Generator().manual_seed(batch)).tolist()
    lens[0] = longest
    c = Paged(lens, 2, 64, 8, torch.bfloat16)
    q = randn(gen(7), batch, 6, 64, dtype=torch.bfloat16)
    out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    for b in {0, 1, batch // 2, batch - 1} & set(range(batch)):
        o, tol, _, _ = attend64(q[b], c.k[b], c.v[b])
        close(out[b], o, tol, f"sequence {b} of {c.lens[b]}")
    alone = [lps.attention_paged_decode(q[b:b + 1], c.kp, c.vp, c.table[b:b + 1], c.lengths[b:b + 1]) for b in range(0, batch, 37)]
    for b, o in zip(range(0, batch, 37), alone):
        ref, tol, _, _ = attend64(q[b], c.k[b], c.v[b])
        close(o[0], ref, tol, f"sequence {b} alone")


def test_pages_past_two_to_the_31_elements():
    nkv, hd, page = 2, 128, 64
    pages = 2 ** 31 // (nkv * hd * page) + 40
    kp, vp = (torch.zeros(pages, nkv, page, hd, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    c = Paged([150], nkv, hd, page, torch.bfloat16)
    c.table = i32([[pages - 1, 3, pages - 17]])
    c.put(0, kp, c.k[0])
    c.put(0, vp, c.v[0])
    q = randn(gen(8), 1, 8, hd, dtype=torch.bfloat16)
    weights = torch.zeros(pages, nkv, page, device="cuda")
    out = lps.attention_paged_decode(q, kp, vp, c.table, c.lengths, key_weights=weights)
    check(c, q, out, weights)
    assert int((weights != 0).sum()) == 300


@pytest.mark.parametrize("dtype", DT)
def test_extreme_scores(dtype):
    """Scores far apart, equal scores, a heavy key at either end: the maximum moves and the others go to nothing."""
    c = Paged([700], 1, 64, 16, DT[dtype])
    q = randn(gen(9), 1, 2, 64, dtype=DT[dtype])
    for factor in (30.0, 0.0):
        c.put(0, c.kp, c.k[0] * factor)
        c.k[0] = c.get(0, c.kp)
        check(c, q, lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths))
    c = Paged([700], 1, 64, 16, DT[dtype])
    for row in (0, 699, 350):
        k = c.k[0].clone()
        k[:, row] = q[0, 0] * 4
        c.put(0, c.kp, k)
        for scale in (0.5, 1e-30):
            o, tol, _, _ = attend64(q[0], k, c.v[0], scale)
            close(lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, scale=scale)[0], o, tol, f"row {row}, scale {scale}")


def test_infinities():
    """A row all of whose scores are -inf is NaN; one -inf score is no weight; an infinity of V arrives."""
    c = Paged([130], 1, 64, 16, torch.bfloat16)
    q = torch.ones(1, 2, 64, device="cuda", dtype=torch.bfloat16)
    page, row = c.at(0)
    kp = c.kp.clone()
    kp[page, :, row] = -float("inf")
    assert torch.isnan(lps.attention_paged_decode(q, kp, c.vp, c.table, c.lengths)).all()
    kp = c.kp.clone()
    kp[page[:70], :, row[:70]] = -float("inf")
    o, tol, _, _ = attend64(q[0], c.k[0][:, 70:], c.v[0][:, 70:])
    close(lps.attention_paged_decode(q, kp, c.vp, c.table, c.lengths)[0], o, tol, "70 rows of -inf")
    clean = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    for bad in (float("inf"), -float("inf"), float("nan")):
        vp = c.vp.clone()
        vp[page[100], 0, row[100], 5] = bad
        out = lps.attention_paged_decode(q, c.kp, vp, c.table, c.lengths)
        want = torch.full((2,), bad, device="cuda", dtype=torch.bfloat16)
        assert torch.equal(out[0, :, 5], want) if bad == bad else torch.isnan(out[0, :, 5]).all()
        out[0, :, 5] = clean[0, :, 5]
        assert torch.equal(out, clean)
    kp = c.kp.clone()
    kp[page[100], 0, row[100], 5] = float("nan")
    assert torch.isnan(lps.attention_paged_decode(q, kp, c.vp, c.table, c.lengths)).all()


def test_a_captured_call_follows_lengths_tables_and_queries():
    c = Paged([500, 0, 100], 2, 64, 16, torch.bfloat16)
    q = randn(gen(10), 3, 8, 64, dtype=torch.bfloat16)
    lengths, table, weights = c.lengths.clone(), c.table.clone(), torch.zeros(c.pages, 2, 16, device="cuda")
    lps.attention_paged_decode(q, c.kp, c.vp, table, lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lps.attention_paged_decode(q, c.kp, c.vp, table, lengths, key_weights=weights, decay=0.0)
    for lens in ([500, 0, 100], [1, 0, 99], [64, 0, 0], [0, 0, 0], [500, 0, 1]):
        lengths.copy_(i32(lens))
        q.copy_(randn(gen(sum(lens)), 3, 8, 64, dtype=torch.bfloat16))
        graph.replay()
        for b, n in enumerate(lens):
            o, tol, _, _ = attend64(q[b], c.k[b][:, :n], c.v[b][:, :n])
            close(out[b], o, tol, f"replay of {lens}, sequence {b}")
    table[0], table[2] = c.table[2], c.table[0]
    lengths.copy_(i32([100, 0, 500]))
    graph.replay()
    for b, other in ((0, 2), (2, 0)):
        o, tol, _, _ = attend64(q[b], c.k[other], c.v[other])
        close(out[b], o, tol, "tables swapped")


def test_calls_on_two_streams_at_once():
    cs = [Paged([3000, 17], 2, 128, 16, torch.bfloat16, seed=s) for s in (1, 2)]
    qs = [randn(gen(s), 2, 8, 128, dtype=torch.bfloat16) for s in (3, 4)]
    want = [lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths) for q, c in zip(qs, cs)]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(lps.attention_paged_decode(qs[i], cs[i].kp, cs[i].vp, cs[i].table, cs[i].lengths))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.parametrize("cycles", [1, 300, 3000])
def test_a_wait_that_gives_up_is_reported(cycles):
    """Each call is right or reported, and the next one right."""
    c = Paged([9000, 70, 4000], 4, 128, 16, torch.bfloat16)
    q = randn(gen(11), 3, 16, 128, dtype=torch.bfloat16)
    want = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    lps.cache_ops_status()
    L = _capi.load()
    _capi.check(L.cache_ops_set_wait_limit(cycles))
    try:
        out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    finally:
        _capi.check(L.cache_ops_set_wait_limit(0))
    try:
        lps.cache_ops_status()
        assert torch.equal(out, want)
    except lps.LpsError as e:
        assert e.code == lps.LPS_ECUDA and "paged decode attention" in str(e)
    assert torch.equal(lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths), want)
    lps.cache_ops_status()


def test_an_empty_cache_and_math():
    c = Paged([0, 0], 2, 64, 16, torch.float16)
    q = randn(gen(12), 2, 4, 64, dtype=torch.float16)
    assert (lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths) == 0).all()
    assert math.isfinite(float(q.sum()))


@pytest.mark.parametrize("nq,nkv,hd,lens", [(32, 8, 128, [9000]), (32, 8, 128, [1000, 8191, 0, 333, 64, 2000]), (4, 2, 64, [5000, 70]), (32, 32, 64, [700] * 9),
                                            (28, 4, 128, [20000, 1]), (12, 4, 128, [3000] * 3), (8, 1, 128, [12000]), (3, 1, 128, [9000, 100])])
def test_heads_in_parts_are_joined_every_time(nq, nkv, hd, lens):
    """Whichever CTA finishes last, and in every replay: hundreds of calls of few and of many parts a head, two graphs in turn."""
    c = Paged(lens, nkv, hd, 16, torch.bfloat16)
    q = randn(gen(13), len(lens), nq, hd, dtype=torch.bfloat16)
    want = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    check(c, q, want)
    out = torch.empty_like(q)
    wrong = torch.zeros((), device="cuda", dtype=torch.int64)
    for _ in range(300):
        out.fill_(float("nan"))
        lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, out=out)
        wrong += (out != want).any()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(4):
                out.fill_(float("nan"))
                lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, out=out)
                wrong += (out != want).any()
        graphs.append(g)
    for i in range(100):
        graphs[i % 2].replay()
    assert int(wrong) == 0
    lps.cache_ops_status()
