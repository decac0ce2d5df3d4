"""The operators over pages where callers meet them: host threads, streams, graphs that take turns, autograd's bookkeeping, both
ways of reading tensors, equal bits for equal calls, and tensors that do not fit."""
import threading

import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import ops

torch = pytest.importorskip("torch")
from paged import Paged, gen, i32, randn  # noqa: E402
from test_gpu_paged_ops import ORDER, adjust64, logits_inputs, same_logits  # noqa: E402

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Step:
    """Inputs of every operator over pages, and one call of each."""

    def __init__(self, seed=1, lens=(200, 3, 0, 65)):
        g = gen(seed)
        self.c = Paged(list(lens), 2, 64, 16, BF, seed=seed, spare=40)
        n = len(lens)
        self.q, self.k, self.v = (randn(g, n, h, 64, dtype=BF) for h in (8, 2, 2))
        self.kp, self.vp = self.c.kp.clone(), self.c.vp.clone()
        self.w = torch.rand(self.c.pages, 2, 16, generator=g, device="cuda")
        self.f = lps.rotary_frequencies(64).cuda()
        self.pos = i32(range(n))
        self.fresh = i32(self.c.free[:4 * n].reshape(n, 4))
        self.x = randn(g, n, 1000, dtype=torch.float32)
        self.tokens = torch.randint(0, 1000, (n, 300), generator=g, device="cuda", dtype=torch.int32)
        self.ids = torch.randint(0, 1000, (n, 20), generator=g, device="cuda", dtype=torch.int32)
        self.bias = randn(g, n, 20, dtype=torch.float32)
        self.count, self.half = torch.full((n,), 300, device="cuda", dtype=torch.int32), torch.full((n,), 0.5, device="cuda")

    def rows(self):
        return lps.rotary_rows(self.q, self.k, self.pos, self.f)

    def append(self):
        kp, vp = self.kp.clone(), self.vp.clone()
        return lps.rotary_append_paged(self.q, self.k, self.v, None, self.c.lengths, self.c.table, kp, vp, self.f), kp, vp

    def attend(self):
        w = self.w.clone()
        return lps.attention_paged_decode(self.q, self.kp, self.vp, self.c.table, self.c.lengths, key_weights=w), w

    def evict(self):
        kp, vp, w = self.kp.clone(), self.vp.clone(), self.w.clone()
        return lps.kv_pages_evict(kp, vp, w, self.c.table, self.c.lengths, self.fresh, 50, 10), kp, vp, w

    def logits(self):
        return (lps.logits_adjust(self.x, tokens=self.tokens, lengths=self.count, repetition=self.half + 1, frequency=self.half,
                                  presence=self.half, bias_ids=self.ids, bias=self.bias),)

    def all(self):
        return [t for f in (self.rows, self.append, self.attend, self.evict, self.logits) for t in f()]


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x.nan_to_num(nan=-9.0) if x.is_floating_point() else x,
                                                y.nan_to_num(nan=-9.0) if y.is_floating_point() else y) for x, y in zip(a, b))


def test_equal_calls_give_equal_bits():
    s = Step(lens=(2000, 3, 0, 65, 900, 1000))
    want = s.all()
    for _ in range(5):
        assert same(s.all(), want)


def test_a_host_threads_first_calls_and_threads_side_by_side():
    steps = [Step(seed) for seed in (1, 2, 3)]
    want = [s.all() for s in steps]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got = steps[i].all()
                torch.cuda.current_stream().synchronize()
                if not same(got, want[i]):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    lps.cache_ops_status()


def test_inputs_made_on_another_stream():
    """The calls run on the current stream, behind what that stream waits for."""
    s = Step()
    want = s.all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        t = Step()
        got = t.all()
    torch.cuda.current_stream().wait_stream(side)
    assert same(got, want)


def test_graphs_that_take_turns_in_one_pool():
    """Two captured steps that share a memory pool, replayed in turn and one after the other without a pause."""
    steps = [Step(1), Step(2, (70, 500, 1))]
    want = [s.all() for s in steps]
    graphs, out = [], []
    pool = torch.cuda.graph_pool_handle()
    for s in steps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            o = s.all()
            keep = [t.clone() for t in o]
        graphs.append(g)
        out.append((o, keep))
    for order in ((0, 1, 0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            graphs[i].replay()
            got = [t.clone() for t in out[i][1]]
            assert same(got, want[i])


def test_both_ways_of_reading_tensors_agree():
    s = Step()
    want = s.all()
    m = ops._ready()
    assert ops._tensors(torch) is not None, "the quick way has not been built for this torch"
    try:
        m.init(lps.LpsError, torch, None)
        assert same(s.all(), want)
        with pytest.raises(ValueError, match="type"):
            lps.rotary_rows(s.q.half(), s.k, s.pos, s.f)
    finally:
        m.init(lps.LpsError, torch, ops._tensors(torch))
    assert same(s.all(), want)

    class Kind(torch.Tensor):
        pass

    q = s.q.as_subclass(Kind)  # read by its attributes
    assert torch.equal(lps.attention_paged_decode(q, s.kp, s.vp, s.c.table, s.c.lengths), s.attend()[0])


def test_autograd_knows_and_is_refused():
    s = Step()
    versions = [t._version for t in (s.kp, s.vp, s.w)]
    lps.rotary_append_paged(s.q, s.k, s.v, None, s.c.lengths, s.c.table, s.kp, s.vp, s.f, key_weights=s.w)
    assert [t._version for t in (s.kp, s.vp, s.w)] == [v + 1 for v in versions]
    out = torch.empty_like(s.q)
    lps.attention_paged_decode(s.q, s.kp, s.vp, s.c.table, s.c.lengths, key_weights=s.w, out=out)
    assert out._version == 1 and s.w._version == versions[2] + 2 and s.kp._version == versions[0] + 1
    lps.kv_pages_evict(s.kp, s.vp, s.w, s.c.table, s.c.lengths, s.fresh, 50)
    assert s.kp._version == versions[0] + 2 and s.w._version == versions[2] + 3
    x = s.x.clone()
    lps.logits_adjust(x, tokens=s.tokens, lengths=s.count, out=x)
    assert x._version == 1
    q = s.q.clone()
    lps.rotary_rows(q, s.k, s.pos, s.f, out=(q, torch.empty_like(s.k)))
    assert q._version == 1

    leaf = s.q.clone().requires_grad_()
    for call in (lambda: lps.rotary_rows(leaf, s.k, s.pos, s.f), lambda: lps.attention_paged_decode(leaf, s.kp, s.vp, s.c.table, s.c.lengths),
                 lambda: lps.attention_paged_decode(s.q, s.kp, s.vp, s.c.table, s.c.lengths, key_weights=s.w.clone().requires_grad_()),
                 lambda: lps.logits_adjust(s.x.clone().requires_grad_()),
                 lambda: lps.logits_adjust(s.x, bias_ids=s.ids, bias=s.bias.clone().requires_grad_())):
        with pytest.raises(ValueError, match="backward"):
            call()
        with torch.no_grad():
            call()
    want = s.all()
    with torch.inference_mode():
        assert same(s.all(), want)


def test_tensors_that_do_not_fit_are_refused():
    s = Step()
    c, wide = s.c, s.c.table.long()
    ok = dict(table=c.table, lengths=c.lengths)

    def attend(q=s.q, kp=s.kp, vp=s.vp, key_weights=None, out=None, **kw):
        a = dict(ok, **kw)
        return lps.attention_paged_decode(q, kp, vp, a["table"], a["lengths"], key_weights=key_weights, out=out)

    attend()
    for kw in (dict(q=s.q[:3]), dict(q=s.q[:, :7]), dict(q=s.q[..., :32]), dict(kp=s.kp[:, :1]), dict(kp=s.kp.transpose(1, 2)), dict(kp=s.kp[::2], vp=s.vp[::2]),
               dict(vp=s.vp.half()), dict(table=wide), dict(table=c.table[:, ::2]), dict(table=c.table[:3]), dict(table=c.table.cpu()),
               dict(lengths=c.lengths[:3]), dict(lengths=c.lengths.cpu()), dict(lengths=c.lengths.float()), dict(key_weights=s.w[:-1]),
               dict(key_weights=s.w.half()), dict(key_weights=s.w.double()), dict(out=s.q[:, :4]), dict(out=s.q.float())):
        with pytest.raises((ValueError, lps.LpsError)):
            attend(**kw)
    with pytest.raises(ValueError, match="freqs"):
        lps.rotary_rows(s.q, s.k, s.pos, s.f.float())
    with pytest.raises(lps.LpsError, match="rot_dim"):
        lps.rotary_rows(s.q, s.k, s.pos, s.f[:20])
    with pytest.raises(ValueError, match="positions"):
        lps.rotary_rows(s.q, s.k, s.pos[:2], s.f)
    with pytest.raises(lps.LpsError, match="one token a sequence"):
        lps.rotary_append_paged(s.q, s.k, s.v, None, c.lengths[:2], c.table[:2], s.kp, s.vp, s.f)
    flat = torch.zeros(s.w.numel() + 1, device="cuda")[1:].view(s.w.shape)
    with pytest.raises(lps.LpsError, match="aligned"):
        lps.kv_pages_evict(s.kp, s.vp, flat, c.table, c.lengths, s.fresh, 50)
    with pytest.raises(lps.LpsError, match="room"):
        lps.kv_pages_evict(s.kp, s.vp, s.w, c.table, c.lengths, s.fresh, 65)
    with pytest.raises(TypeError):
        lps.kv_pages_evict(s.kp, s.vp, s.w, c.table, c.lengths, s.fresh, 50.5)
    for kw in (dict(tokens=s.tokens), dict(lengths=s.count), dict(repetition=s.half), dict(bias=s.bias), dict(allowed=s.tokens),
               dict(tokens=s.tokens.long(), lengths=s.count), dict(bias_ids=s.ids, bias=s.bias[:, :3]), dict(out=s.x.half())):
        with pytest.raises(ValueError):
            lps.logits_adjust(s.x, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        lps.logits_adjust(s.x.t())
    with pytest.raises(ValueError, match="float32"):
        lps.logits_adjust(s.x.double())


def test_empty_calls():
    s = Step()
    q, k = lps.rotary_rows(s.q[:0], s.k[:0], s.pos[:0], s.f)
    assert q.shape == (0, 8, 64) and k.shape == (0, 2, 64)
    off = torch.zeros(5, device="cuda", dtype=torch.int32)
    kp = s.kp.clone()
    assert lps.rotary_append_paged(s.q[:0], s.k[:0], s.v[:0], off, s.c.lengths, s.c.table, kp, s.vp, s.f).shape == (0, 8, 64)
    assert torch.equal(kp.nan_to_num(), s.kp.nan_to_num())
    assert lps.logits_adjust(s.x[:0]).shape == (0, 1000) and lps.logits_adjust(s.x[:, :0]).shape == (4, 0)
    assert torch.equal(lps.logits_adjust(s.x, tokens=s.tokens[:, :0], lengths=s.count, repetition=s.half), s.x)
    assert torch.equal(lps.logits_adjust(s.x, bias_ids=s.ids[:, :0], bias=s.bias[:, :0]), s.x)


FIRST = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import torch
from test_gpu_paged_edges import Step, same
s = Step()
g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    out = [t.clone() for t in s.all()]
g.replay()
torch.cuda.synchronize()
assert same(out, s.all())
print("fine")
"""


def test_a_process_whose_first_calls_are_captured():
    import os
    import subprocess
    import sys
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=os.path.dirname(tests), tests=tests)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("page", [1000, 4096])
def test_caches_of_one_page_a_sequence(page):
    """A contiguous cache [sequences, kv heads, max_ctx, head_dim] is pages of max_ctx rows: what the operators on it give."""
    lens, nkv, hd = [min(page, 900), 1, 300], 2, 128
    g = gen(4)
    kc, vc = (randn(g, 3, nkv, page, hd, dtype=BF) for _ in range(2))
    q = randn(g, 3, 8, hd, dtype=BF)
    table, chain = i32([[0], [1], [2]]), torch.full((3, 1), -1, device="cuda", dtype=torch.int32)
    out = lps.attention_paged_decode(q, kc, vc, table, i32(lens))
    tree = lps.attention_tree_verify(q[:, None], kc, vc, chain, [n - 1 for n in lens], [1, 1, 1])[:, 0]
    assert (out.float() - tree.float()).abs().max() <= 2 * 2.0 ** -8 * tree.float().abs().max()  # two results, rounded once, and weights of 8 bits
    k, v = randn(g, 5, nkv, hd, dtype=BF), randn(g, 5, nkv, hd, dtype=BF)
    a, b, c, d = kc.clone(), vc.clone(), kc.clone(), vc.clone()
    lps.kv_rows_append(k, v, [0, 2, 2, 5], a, b, [10, 0, 296])
    lps.rotary_append_paged(randn(g, 5, 8, hd, dtype=BF), k, v, i32([0, 2, 2, 5]), i32([12, 0, 299]), table, c, d, None)
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("tokens", [3, 400])
def test_many_heads_a_token(tokens):
    """More (token, head) rows than a block places at once: every head as if alone."""
    g, f = gen(6), lps.rotary_frequencies(64).cuda()
    q, k, v = randn(g, tokens, 700, 64, dtype=BF), randn(g, tokens, 130, 64, dtype=BF), randn(g, tokens, 130, 64, dtype=BF)
    pos = torch.arange(50, 50 + tokens, device="cuda", dtype=torch.int32)
    qo, ko = lps.rotary_rows(q, k, pos, f)
    for h in (0, 1, 511, 512, 699):
        one, _ = lps.rotary_rows(q[:, h:h + 1].contiguous(), k[:, :1], pos, f)
        assert torch.equal(qo[:, h:h + 1], one)
    kp, vp = (torch.zeros(tokens // 8 + 1, 130, 8, 64, device="cuda", dtype=BF) for _ in range(2))
    table = torch.arange(kp.shape[0], device="cuda", dtype=torch.int32)[None]
    qa = lps.rotary_append_paged(q, k, v, i32([0, tokens]), i32([tokens]), table, kp, vp, f, positions=pos)
    assert torch.equal(qa, qo)
    assert torch.equal(kp.transpose(1, 2).reshape(-1, 130, 64)[:tokens], ko) and torch.equal(vp.transpose(1, 2).reshape(-1, 130, 64)[:tokens], v)
    same_q, same_k = lps.rotary_rows(q, k, pos, None)  # nothing turns
    assert torch.equal(same_q, q) and torch.equal(same_k, k)


def test_pools_and_logits_past_two_to_the_31_elements():
    nkv, hd, page = 2, 128, 64
    pages = 2 ** 31 // (nkv * hd * page) + 20
    kp, vp = (torch.zeros(pages, nkv, page, hd, device="cuda", dtype=BF) for _ in range(2))
    w = torch.zeros(pages, nkv, page, device="cuda")
    g, f = gen(7), lps.rotary_frequencies(hd).cuda()
    q, k, v = randn(g, 100, 4, hd, dtype=BF), randn(g, 100, nkv, hd, dtype=BF), randn(g, 100, nkv, hd, dtype=BF)
    old, new = i32([[pages - 1, pages - 3]]), i32([[pages - 2]])
    lps.rotary_append_paged(q, k, v, i32([0, 100]), i32([100]), old, kp, vp, f, key_weights=w)
    kr = lps.rotary_rows(q, k, torch.arange(100, device="cuda", dtype=torch.int32), f)[1]
    assert torch.equal(kp[pages - 1].transpose(0, 1), kr[:64]) and torch.equal(vp[pages - 3, :, :36].transpose(0, 1), v[64:])
    w[pages - 1, 0, 5:30] = 2.0
    w[pages - 3, 1, 3:20] = 1.0
    assert lps.kv_pages_evict(kp, vp, w, old, i32([100]), new, 30, 2).tolist() == [30]
    assert torch.equal(kp[pages - 2, 0, :30], torch.cat((kr[0:3, 0], kr[5:30, 0], kr[98:, 0])))
    assert torch.equal(vp[pages - 2, 1, :30], torch.cat((v[0:11, 1], v[67:84, 1], v[98:, 1])))
    assert torch.equal(w[pages - 2, 0, :30], torch.cat((w.new_zeros(3), w.new_full((25,), 2.0), w.new_zeros(2))))
    assert not kp[0].any() and not vp[1].any()
    del kp, vp, w
    torch.cuda.empty_cache()
    x = torch.zeros(40000, 65536, device="cuda", dtype=BF)
    x[39999, 7] = 3.0
    n = torch.ones(40000, device="cuda", dtype=torch.int32)
    seven = torch.full((40000, 1), 7, device="cuda", dtype=torch.int32)
    out = lps.logits_adjust(x, tokens=seven, lengths=n, presence=torch.ones(40000, device="cuda"), out=x)
    assert float(out[39999, 7]) == 2.0 and float(out[39998, 7]) == -1.0 and float(out[0, 7]) == -1.0
    assert int((out[39990:] != 0).sum()) == 10 and int((out[:10] != 0).sum()) == 10


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("batch,vocab,width,entries", [(2, 1000, 1500, 0), (3, 5000, 16383, 4), (3, 40001, 16384, 4), (20, 65537, 100, 5),
                                                       (20, 65537, 9000, 5), (20, 65537, 16400, 600), (80, 65537, 60, 3), (80, 65537, 5000, 0)])
def test_logits_of_few_and_many_rows_with_short_and_long_histories(batch, vocab, width, entries, dtype):
    x, d = logits_inputs(batch, vocab, width, entries, dtype, 2)
    d["allowed"] |= i32([[0x0FF0FF0F] * d["allowed"].shape[1]])
    kw = {k: v for k, v in d.items() if v is not None}
    ref = adjust64(x, *(kw.get(k) for k in ORDER))
    got = lps.logits_adjust(x, **kw)
    same_logits(got, *ref)
    same = x.clone()
    assert lps.logits_adjust(same, **kw, out=same) is same and torch.equal(same, got)


@pytest.mark.parametrize("width", [16383, 16384, 70000])
def test_logits_of_a_history_of_one_token(width):
    """As many counts as the history has room for, of a token whose neighbours are in the history too."""
    x = torch.zeros(2, 9000, device="cuda")
    tokens = torch.full((2, width), 4001, device="cuda", dtype=torch.int32)
    tokens[1, :2] = i32([4000, 4002])
    out = lps.logits_adjust(x, tokens=tokens, lengths=i32([width, width]), frequency=torch.ones(2, device="cuda"),
                            bias_ids=i32([[4002], [4003]]), bias=torch.full((2, 1), 0.5, device="cuda"))
    assert out[0, 3999:4004].tolist() == [0.0, 0.0, -width, 0.5, 0.0] and out[1, 3999:4004].tolist() == [0.0, -1.0, 2.0 - width, -1.0, 0.5]
    assert int((out != 0).sum()) == 2 + 4
