"""Calls of the operators over pages that their documentation allows and that are easy to forget."""
import pytest

import layer_pipeline_staged_gb300 as lps

torch = pytest.importorskip("torch")
from paged import Paged, gen, i32, randn  # noqa: E402
from test_gpu_paged_attention import attend64, close  # noqa: E402
from test_gpu_paged_large import kept  # noqa: E402

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def none(*shape, dtype=torch.int32):
    return torch.empty(*shape, device="cuda", dtype=dtype)


@pytest.mark.parametrize("width", [0, 4])
def test_a_batch_of_no_sequences(width):
    """A step of a batch that has run empty: every call returns what it has for no sequences, and nothing is written."""
    c = Paged([40], 2, 64, 16, BF)
    kp, vp, w, f = c.kp.clone(), c.vp.clone(), torch.rand(c.pages, 2, 16, generator=gen(1), device="cuda"), lps.rotary_frequencies(64).cuda()
    was, q, k = w.clone(), none(0, 8, 64, dtype=BF), none(0, 2, 64, dtype=BF)
    table, lengths = none(0, width), none(0)
    qo, ko = lps.rotary_rows(q, k, lengths, f)
    assert qo.shape == q.shape and ko.shape == k.shape
    assert lps.rotary_append_paged(q, k, k, None, lengths, table, kp, vp, f, key_weights=w).shape == q.shape
    out = lps.attention_paged_decode(q, kp, vp, table, lengths, key_weights=w)
    assert out.shape == q.shape and out.dtype == BF
    given = none(0, 8, 64, dtype=BF)
    assert lps.attention_paged_decode(q, kp, vp, table, lengths, out=given) is given
    new = lps.kv_pages_evict(kp, vp, w, table, lengths, none(0, 2), 20, 5)
    assert new.shape == (0,) and new.dtype == torch.int32 and new.is_cuda
    assert lps.logits_adjust(none(0, 100, dtype=torch.float32), tokens=none(0, 3), lengths=lengths).shape == (0, 100)
    assert torch.equal(w, was)
    for x, y in ((kp, c.kp), (vp, c.vp)):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())


@pytest.mark.parametrize("width", [None, 700])
def test_sequences_that_share_pages(width):
    """Two sequences with one prefix, and one that has a page of its own twice: each as if alone, by a cluster a head and by shares;
    then an eviction from the shared pages, which stay as they were."""
    nkv, hd, page = 2, 64, 16
    c = Paged([100, 70, 48], nkv, hd, page, BF, spare=12, width=width)
    table = c.table.clone()
    table[1, :3] = table[0, :3]  # 48 rows of the first
    table[2, 2] = table[2, 0]
    q = randn(gen(2), 3, 8, hd, dtype=BF)
    k, v = ([x[0], torch.cat((x[0][:, :48], x[1][:, 48:]), 1), torch.cat((x[2][:, :32], x[2][:, :16]), 1)] for x in (c.k, c.v))
    out = lps.attention_paged_decode(q, c.kp, c.vp, table, c.lengths)
    for b in range(3):
        o, tol, _, _ = attend64(q[b], k[b], v[b])
        close(out[b], o, tol, f"sequence {b}")
    weights = torch.rand(c.pages, nkv, page, generator=gen(3), device="cuda")
    kp, vp, w, fresh = c.kp.clone(), c.vp.clone(), weights.clone(), i32(c.free[:9].reshape(3, 3))
    assert lps.kv_pages_evict(kp, vp, w, table, c.lengths, fresh, 40, 10).tolist() == [40, 40, 40]
    old = table[table >= 0].unique().long()
    for x, was in ((kp, c.kp), (vp, c.vp), (w, weights)):
        assert torch.equal(x[old].nan_to_num(), was[old].nan_to_num())
    for b, n in enumerate(c.lens):
        r = torch.arange(n, device="cuda")
        of_row = weights[table[b].long()[r // page], :, r % page].cpu().numpy()
        i = torch.arange(40, device="cuda")
        at = fresh[b].long()[i // page]
        for h in range(nkv):
            rows = torch.from_numpy(kept(of_row[:, h], n, 40, 10)).cuda()
            assert torch.equal(kp[at, h, i % page], k[b][h, rows]) and torch.equal(vp[at, h, i % page], v[b][h, rows])
