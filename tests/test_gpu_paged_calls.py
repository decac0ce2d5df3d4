"""Calls of the operators over pages that their documentation allows and that are easy to forget."""
import pytest

import layer_pipeline_staged_gb300 as lps

torch = pytest.importorskip("torch")
from paged import Paged, gen, i32, randn  # noqa: E402

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
