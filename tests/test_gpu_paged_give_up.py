"""Attention over pages when waits give up: with a limit of one cycle every wait does so for certain, without a look, and the
call has to say so, end, and leave the next call as it would have been; with other limits each call is right or reported."""
import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi

torch = pytest.importorskip("torch")
from paged import DT, Paged, gen, i32, randn  # noqa: E402

pytestmark = pytest.mark.gpu

# in shares over all CTAs (with pieces of several heads a CTA), and a cluster a head
FORMS = {"shares": ([9000, 70, 4000], 4, 128, 16), "many": ([200, 3, 64, 65] * 40, 2, 64, 8), "cluster": ([1000, 70, 900], 4, 128, 16),
         "one": ([130], 1, 64, 3)}


class limited:
    def __init__(self, cycles):
        self.cycles = cycles

    def __enter__(self):
        _capi.check(_capi.load().cache_ops_set_wait_limit(self.cycles))

    def __exit__(self, *_):
        _capi.check(_capi.load().cache_ops_set_wait_limit(0))


def reported():
    """Whether a call has given up since the last look."""
    try:
        lps.cache_ops_status()
    except lps.LpsError as e:
        assert e.code == lps.LPS_ECUDA and "paged decode attention" in str(e)
        return True
    return False


def form(name, dtype=torch.bfloat16):
    lens, nkv, hd, group = FORMS[name]
    c = Paged(lens, nkv, hd, 16, dtype)
    return c, randn(gen(11), len(lens), nkv * group, hd, dtype=dtype)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("dtype", DT)
def test_a_call_whose_waits_give_up_is_reported(name, dtype, weighted):
    c, q = form(name, DT[dtype])
    weights = torch.zeros(c.pages, c.nkv, 16, device="cuda") if weighted else None
    want = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, key_weights=weights, decay=0.0)
    was = None if weights is None else weights.clone()
    assert not reported()
    for _ in range(3):
        with limited(1):
            lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, key_weights=weights, decay=0.0)
        assert reported() and not reported()
        assert torch.equal(lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths, key_weights=weights, decay=0.0), want)
        assert weights is None or torch.equal(weights, was)
        assert not reported()


def test_a_call_without_rows_waits_for_nothing():
    c, q = form("cluster")
    with limited(1):
        out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, i32([0, -1, 0]))
    assert not reported() and (out == 0).all()


@pytest.mark.parametrize("name", FORMS)
def test_limits_of_all_lengths(name):
    c, q = form(name)
    want = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
    assert not reported()
    for cycles in (2, 50, 200, 500, 1000, 2000, 4000, 8000, 20000):
        with limited(cycles):
            out = lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths)
        assert reported() or torch.equal(out, want)
        assert torch.equal(lps.attention_paged_decode(q, c.kp, c.vp, c.table, c.lengths), want) and not reported()
