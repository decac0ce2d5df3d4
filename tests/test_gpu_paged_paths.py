"""The two ways through attention over pages, of one size each: heads shared out over all CTAs where the tables have room for many
rows, and a cluster a head where they have not; against the formula in 64 bits, with bad pages, in graphs and with waits that give up."""
import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi

torch = pytest.importorskip("torch")
from paged import Paged, gen, i32, randn  # noqa: E402
from test_gpu_paged_attention import LENS, attend64, check, close  # noqa: E402

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("nq,nkv,hd,page,dtype", [(4, 2, 64, 16, BF), (32, 8, 128, 16, FP), (3, 1, 128, 24, BF), (9, 1, 64, 128, FP), (48, 12, 128, 40, BF)])
def test_tables_with_room_for_many_rows(nq, nkv, hd, page, dtype, lens):
    c = Paged(LENS[lens], nkv, hd, page, dtype, width=10000 // page)
    q = randn(gen(2), len(c.lens), nq, hd, dtype=dtype)
    out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    weights = torch.full((c.pages, nkv, page), float("nan"), device="cuda")
    assert torch.equal(out, lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, key_weights=weights, decay=0.0))
    check(c, q, out, weights)
    assert int(torch.isfinite(weights).sum()) == sum(c.lens) * nkv
    lps.cache_ops_status()


@pytest.mark.parametrize("width", [19, 600])
def test_bad_lengths_and_pages(width):
    c = Paged([100, 200, 300, 64, 20], 2, 64, 16, BF, width=width)
    q = randn(gen(6), 5, 4, 64, dtype=BF)
    for bad in (-1, width * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, i32([100, bad, 300, 64, bad]))
        assert (out[[1, 4]] == 0).all()
        for b in (0, 2, 3):
            o, tol, _, _ = attend64(q[b], c.k[b], c.v[b])
            close(out[b], o, tol, f"sequence {b} beside length {bad}")
        table = c.table.clone()
        table[2, 3:5] = table[3] = bad if bad < 0 else c.pages
        weights = torch.full((c.pages, 2, 16), 5.0, device="cuda")
        out = lps.attention_paged_decode(q, c.kp, c.vp, table, c.lengths, key_weights=weights, decay=0.0)
        keep = torch.ones(300, dtype=torch.bool, device="cuda")
        keep[48:80] = False
        o, tol, w, wtol = attend64(q[2], c.k[2][:, keep], c.v[2][:, keep])
        close(out[2], o, tol, "holes")
        close(c.get(2, weights.unsqueeze(-1)).squeeze(-1)[:, keep], w, wtol + 2.0 ** -23 * w, "weights beside the holes")
        page, row = c.at(3)
        assert (out[3] == 0).all() and (weights[page, :, row] == 5.0).all()
    lps.cache_ops_status()


@pytest.mark.parametrize("nq,nkv,hd,lens", [(16, 4, 128, [8000]), (18, 9, 64, [8192]), (30, 10, 64, [4096]), (32, 8, 128, [900, 0, 1]), (16, 8, 64, [700, 64] * 4),
                                            (16, 8, 64, [500, 1, 65, 1000] * 4), (3, 1, 128, [300] * 133), (2, 1, 128, [300] * 134), (32, 2, 128, [1000])])
def test_heads_of_clusters_are_joined_every_time(nq, nkv, hd, lens):
    """One to eight CTAs a head, and a head more than there is room for: in every call and in graphs that take turns."""
    c = Paged(lens, nkv, hd, 16, BF)
    q = randn(gen(13), len(lens), nq, hd, dtype=BF)
    want = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    check(c, q, want)
    out = torch.empty_like(q)
    wrong = torch.zeros((), device="cuda", dtype=torch.int64)

    def calls(n):
        for _ in range(n):
            out.fill_(float("nan"))
            lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, out=out)
            wrong.add_((out != want).any())

    calls(100)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            calls(4)
    for i in range(50):
        graphs[i % 2].replay()
    assert int(wrong) == 0
    lps.cache_ops_status()


@pytest.mark.parametrize("cycles", [1, 300, 3000])
def test_a_wait_of_a_cluster_that_gives_up_is_reported(cycles):
    c = Paged([1000, 70, 900], 4, 128, 16, BF)
    q = randn(gen(11), 3, 16, 128, dtype=BF)
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
