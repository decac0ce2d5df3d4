"""The operators over pages where tables have room for many rows: evictions by clusters, of more rows than they hold, and key weights
behind the grid of the kernel that sums them, logits by the rows and histories that choose a block's run; and the order of weights that
are no numbers."""
import numpy as np
import pytest

import layer_pipeline_staged_gb300 as lps

torch = pytest.importorskip("torch")
from paged import Paged, gen, i32, randn  # noqa: E402
from test_gpu_paged_attention import attend64, close  # noqa: E402
from test_gpu_paged_ops import ORDER, adjust64, logits_inputs, same_logits  # noqa: E402

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def kept(w, n, budget, recent):
    """The rows that stay of n with weights w, in order: NaN is below every number, of equal ones the lowest row stays."""
    if n <= budget:
        return np.arange(n)
    w, nan = w[: n - recent], np.isnan(w[: n - recent])
    best = np.lexsort((np.arange(n - recent), -np.where(nan, 0.0, w), nan))[: budget - recent]
    return np.concatenate([np.sort(best), np.arange(n - recent, n)])


def check(lens, nkv, hd, page, budget, recent, weights, width=None):
    need = [-(-min(n, budget) // page) for n in lens]
    c = Paged(lens, nkv, hd, page, BF, spare=sum(need) + 2, width=width)
    kw = torch.full((c.pages, nkv, page), 77.0, device="cuda")
    fresh, at = np.full((len(lens), -(-budget // page)), -1, np.int32), 0
    for b, n in enumerate(lens):
        p, j = c.at(b)
        kw[p, :, j] = weights(b, nkv, n).T
        fresh[b, : need[b]] = c.free[at:at + need[b]]
        at += need[b]
    got = [c.kp.clone(), c.vp.clone(), kw.clone()]
    new = lps.kv_pages_evict(*got, c.table, c.lengths, i32(fresh), budget, recent)
    assert new.tolist() == [min(n, budget) for n in lens]
    want = [c.kp.clone(), c.vp.clone(), kw.clone()]
    for b, n in enumerate(lens):
        p, j = c.at(b)
        for h in range(nkv):
            rows = torch.from_numpy(kept(kw[p, h, j].cpu().numpy(), n, budget, recent)).cuda()
            to = torch.arange(len(rows), device="cuda")
            for x, was in zip(want, (c.kp, c.vp, kw)):
                x[i32(fresh)[b].long()[to // page], h, to % page] = was[p[rows], h, j[rows]]
    for g, w in zip(got, want):
        assert torch.equal(torch.nan_to_num(g, nan=-123.0), torch.nan_to_num(w, nan=-123.0))


def spread(b, nkv, n):
    return torch.rand(nkv, n, generator=gen(1 + b), device="cuda") ** 8


def few(b, nkv, n):
    return (torch.rand(nkv, n, generator=gen(1 + b), device="cuda") * 4).floor()


def equal(b, nkv, n):
    return torch.zeros(nkv, n, device="cuda")


def no_numbers(b, nkv, n):
    x = torch.rand(nkv, n, generator=gen(1 + b), device="cuda") - 0.5
    kind = torch.randint(0, 3, (nkv, n), generator=gen(99 + b), device="cuda")
    x[kind == 1], x[kind == 2] = -float("inf"), float("nan")
    return x


WEIGHTS = {"spread": spread, "few": few, "equal": equal, "no_numbers": no_numbers}


@pytest.mark.parametrize("weights", WEIGHTS)
@pytest.mark.parametrize("room", [16384, 32768, 65536])
@pytest.mark.parametrize("lens,budget,recent", [([16001, 5, 0], 4000, 64), ([100], 50, 10), ([16384, 2, 64], 15999, 7), ([9, 3001], 3000, 3000)])
def test_clusters_of_two_to_eight(weights, room, lens, budget, recent):
    """By the tables' room: long sequences, and short ones of which most blocks have no row."""
    check(lens, 2, 64, 16, budget, recent, WEIGHTS[weights], width=room // 16)


@pytest.mark.parametrize("weights", WEIGHTS)
@pytest.mark.parametrize("lens,nkv,hd,page", [([33001], 1, 128, 24), ([65530, 40000], 3, 64, 64), ([40000] + [70] * 40, 2, 64, 8)])
def test_tables_just_as_wide_as_their_sequences(weights, lens, nkv, hd, page):
    check(lens, nkv, hd, page, 9001, 100, WEIGHTS[weights])


@pytest.mark.parametrize("weights", WEIGHTS)
@pytest.mark.parametrize("budget", [1000, 200001])
def test_more_rows_than_a_cluster_holds(weights, budget):
    check([270001], 1, 64, 128, budget, 33, WEIGHTS[weights])


@pytest.mark.parametrize("n", [1501, 1504])
@pytest.mark.parametrize("budget", [300, 700, 1220, 1480])
def test_nan_is_below_minus_infinity(n, budget):
    """Where the budget ends among the numbers, among -inf and among NaN, with eights of rows that are not whole."""
    check([n, 33], 2, 64, 16, budget, 20, no_numbers)


@pytest.mark.parametrize("decay", [0.0, 0.5])
def test_key_weights_behind_the_grid(decay):
    """256 sequences of 8 kv heads: the grid has blocks for 16384 keys of each, and one sequence has 40000."""
    lens = [(i * 37) % 90 for i in range(256)]
    lens[200] = 40000
    c = Paged(lens, 8, 64, 16, BF)
    q = randn(gen(2), 256, 8, 64, dtype=BF)
    old = torch.rand(c.pages, 8, 16, generator=gen(3), device="cuda")
    new = old.clone()
    out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, key_weights=new, decay=decay)
    seen = torch.zeros(c.pages, 16, dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        page, row = c.at(b)
        seen[page, row] = True
        if b in (1, 2, 199, 200, 201, 255):
            o, tol, w, wtol = attend64(q[b], c.k[b], c.v[b])
            close(out[b], o, tol, f"sequence {b} of {n}")
            want = decay * old[page, :, row].T.double() + w
            close(new[page, :, row].T, want, wtol + 2.0 ** -23 * want, f"weights of sequence {b}")
    assert torch.equal(new.transpose(1, 2)[~seen], old.transpose(1, 2)[~seen])
    assert (new != old).transpose(1, 2)[seen].any(-1).all()
    lps.cache_ops_status()


@pytest.mark.parametrize("dtype", [torch.float32, BF, torch.float16])
@pytest.mark.parametrize("batch,vocab,width,entries", [(24, 128256, 300, 8), (27, 128256, 1016, 8), (27, 128256, 1017, 8), (44, 128256, 500, 0),
                                                       (50, 128256, 0, 30), (50, 128256, 5000, 3), (100, 65537, 1000, 0), (12, 128255, 9000, 1)])
def test_logits_of_many_rows(batch, vocab, width, entries, dtype):
    x, d = logits_inputs(batch, vocab, width, entries, dtype)
    kw = {k: v for k, v in d.items() if v is not None}
    ref = adjust64(x, *(kw.get(k) for k in ORDER))
    same_logits(lps.logits_adjust(x, **kw), *ref)
    assert lps.logits_adjust(x, **kw, out=x) is x
    same_logits(x, *ref)
