"""The operators over a caller-owned cache at the edges of what a caller may do: host threads, values and
tensors that are rare but allowed, and calls that are refused."""
import threading

import numpy as np
import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def _randn(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def _status():
    return _capi.load().cache_ops_status(torch.cuda.current_stream().cuda_stream)


# ---- host threads ---------------------------------------------------------------------------------

@pytest.mark.parametrize("op", ["prompt", "tree", "append", "accept"])
def test_a_threads_first_call_on_the_device(op):
    """A host thread that has made no call on the device yet: the call is enqueued like any other's."""
    q, k, v = _randn(1, 70, 8, 128), _randn(2, 70, 2, 128), _randn(3, 70, 2, 128)
    kc, vc, tq = _randn(4, 1, 2, 100, 128), _randn(5, 1, 2, 100, 128), _randn(6, 1, 3, 8, 128)
    par = torch.tensor([[-1, 0, -1]], dtype=torch.int32, device="cuda")
    path, taken = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    po, to = torch.zeros_like(q), torch.zeros_like(tq)

    def call():
        if op == "prompt":
            lps.attention_prompt_packed(q, k, v, [0, 30, 70], out=po)
        elif op == "tree":
            lps.attention_tree_verify(tq, kc, vc, par, [90], [3], out=to)
        elif op == "append":
            lps.kv_rows_append(k, v, [0, 70], kc, vc, [20])
        else:
            lps.kv_rows_accept(kc, vc, [90], path, taken)

    state = (po, to, kc, vc)
    before = [t.clone() for t in state]
    call()
    want = [t.clone() for t in state]
    for t, b in zip(state, before):
        t.copy_(b)
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call()
        except Exception as e:  # reported by the main thread
            errors.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(torch.equal(t, w) for t, w in zip(state, want))


# ---- weights far apart ------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("above", [14.0, 16.0, 17.5, 20.0])
def test_many_small_weights_beside_a_large_one(above, hd, dtype):
    """One key (the first, or one in the middle) whose score is far above those of 8000 others, which are all
    equal: their share of the output arrives. With v = 0 at the large key and 1 elsewhere the output is that
    share, s = n e^-above / (1 + n e^-above).

    Tolerance: u = eps / 2; the result is rounded once, u s; a weight above the type's smallest normal number is
    off by u of itself, a smaller one by half of the smallest number; in fp16 the weights of 2^7 to 2^15 that
    the largest key gets make that at most 2^-25 2^-7 of the denominator each, together n 2^-32; fp32: the
    exponent's argument is at most 1.45 above + 7, rounded twice, and exp2 is off by 2^-22, sums over n keys are
    off by 2 n 2^-24 of themselves."""
    n = 8001
    u = torch.finfo(dtype).eps / 2
    share = (n - 1) * np.exp(-above) / (1 + (n - 1) * np.exp(-above))
    tol = 2 * u * share + ((n * 2.0 ** -32) if dtype == FP else 0.0) + share * (2.0 ** -21 + 4 * (1.45 * above + 7) * 2.0 ** -24 + 2 * n * 2.0 ** -24)
    for at in (0, 4000):
        q = torch.ones(n, 4, hd, device="cuda", dtype=dtype)
        k, v = torch.zeros(n, 2, hd, device="cuda", dtype=dtype), torch.ones(n, 2, hd, device="cuda", dtype=dtype)
        k[at], v[at] = above / 8, 0.0
        scale = 8.0 / hd  # the score of the large key: hd (above / 8) scale
        out = lps.attention_prompt_packed(q, k, v, [0, n], scale=scale)
        kc, vc = (t.transpose(0, 1).contiguous()[None] for t in (k, v))
        tree = lps.attention_tree_verify(q[None, :3].contiguous(), kc, vc, torch.tensor([[-1, 0, 1]], dtype=torch.int32, device="cuda"),
                                         [n - 3], [3], scale=scale)
        for got in (out[-1], tree[0, 2]):
            assert ((got.double() - share).abs() <= tol).all(), (at, got.double().mean().item() / share, tol / share)


# ---- infinities ---------------------------------------------------------------------------------------

def _chain(batch, width):
    return torch.arange(-1, width - 1, device="cuda", dtype=torch.int32).repeat(batch, 1)


# trees whose keys one CTA has alone, that two slots share, that clusters share, and wide ones
TREES = [(1, 1, 0, 8, 2), (2, 9, 60, 8, 2), (1, 5, 3000, 8, 2), (1, 64, 2000, 8, 2), (60, 64, 40, 16, 4)]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hd", [64, 128])
def test_a_row_whose_scores_are_all_minus_infinity(hd, dtype):
    """0 / 0 by the formula: NaN from a prompt and from every tree, however its keys are shared out; with one
    finite score among them the row is that key's value. A draft of a broken chain stays zero."""
    q, k, v = _randn(1, 300, 8, hd, dtype=dtype).abs() + 1, _randn(2, 300, 2, hd, dtype=dtype), _randn(3, 300, 2, hd, dtype=dtype)
    k[:140] = -float("inf")
    out = lps.attention_prompt_packed(q, k, v, [0, 300])
    assert out[:140].isnan().all() and not out[140:].isnan().any()
    assert torch.equal(out[140].view(2, 4, hd), v[140][:, None].expand(2, 4, hd))
    for batch, width, pos, nq, nkv in TREES:
        tq, kc, vc = _randn(4, batch, width, nq, hd, dtype=dtype).abs() + 1, _randn(5, batch, nkv, pos + width, hd, dtype=dtype), _randn(6, batch, nkv, pos + width, hd, dtype=dtype)
        parents = _chain(batch, width)
        if width > 2:
            parents[:, width - 1] = 77  # the last draft's chain is broken
        kc[:] = -float("inf")
        out = lps.attention_tree_verify(tq, kc, vc, parents, [pos] * batch, [width] * batch)
        whole = out[:, :width - 1] if width > 2 else out
        assert whole.isnan().all()
        assert width <= 2 or (out[:, width - 1] == 0).all()
        for at in {0, pos // 2, pos}:  # one key that is seen by all drafts
            kc2 = kc.clone()
            kc2[:, :, at] = 0.5
            out = lps.attention_tree_verify(tq, kc2, vc, parents, [pos] * batch, [width] * batch)
            want = vc[:, :, at].repeat_interleave(nq // nkv, 1)[:, None].expand(batch, width, nq, hd)
            whole = slice(0, width - 1 if width > 2 else width)
            assert torch.equal(out[:, whole], want[:, whole]), (width, pos, at)
            assert width <= 2 or (out[:, width - 1] == 0).all()


FAR = {BF: 100.0, FP: 30.0}  # a score so far below the largest has a weight of zero in the element type


def _far_case(seed, n, nq, nkv, hd, dtype, peak):
    """q, k, v of one sequence whose key `peak` has a score FAR above all others', which are equal; by the formula
    every weight is positive."""
    q = torch.ones(n, nq, hd, device="cuda", dtype=dtype)
    k = torch.zeros(n, nkv, hd, device="cuda", dtype=dtype)
    k[peak] = FAR[dtype] / 8
    return q, k, _randn(seed, n, nkv, hd, dtype=dtype), 8.0 / hd


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("peak,at", [(0, 70), (70, 0), (300, 20), (20, 300), (500, 501), (599, 3), (3, 598)])
def test_prompt_infinity_seen_with_a_weight_next_to_nothing(peak, at, hd, dtype):
    """A positive weight times infinity is infinite, however small the weight and wherever the key lies: in a block
    that all rows see whole or one that they do not, before or behind the key that outweighs it."""
    n, inf = 600, float("inf")
    q, k, v, scale = _far_case(7, n, 8, 2, hd, dtype, peak)
    clean = lps.attention_prompt_packed(q, k, v, [0, n], scale=scale)
    assert torch.isfinite(clean).all()
    v2 = v.clone()
    v2[at, :, 3], v2[at, :, 40] = inf, -inf
    v2[at, :, 50], v2[max(at - 9, 1), :, 50] = inf, -inf
    v2[at, :, 60] = float("nan")
    got = lps.attention_prompt_packed(q, k, v2, [0, n], scale=scale)
    assert (got[at:, :, 3] == inf).all() and (got[at:, :, 40] == -inf).all()
    both = max(at, at - 9, 1)
    assert got[both:, :, [50, 60]].isnan().all()
    others = [d for d in range(hd) if d not in (3, 40, 50, 60)]
    assert torch.equal(got[:, :, others], clean[:, :, others]) and torch.equal(got[:at, :, 3], clean[:at, :, 3])
    # a weight that is zero by the formula, at a score of -inf: 0 x inf
    k[at] = -inf
    clean = lps.attention_prompt_packed(q, k, v, [0, n], scale=scale)
    got = lps.attention_prompt_packed(q, k, v2, [0, n], scale=scale)
    assert got[at:, :, [3, 40, 50, 60]].isnan().all()
    assert torch.equal(got[at + 1:, :, others], clean[at + 1:, :, others])
    # and a NaN score makes the whole row NaN
    k[at] = float("nan")
    assert lps.attention_prompt_packed(q, k, v2, [0, n], scale=scale)[at:].isnan().all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("tree", range(len(TREES)))
def test_tree_infinity_seen_with_a_weight_next_to_nothing(tree, hd, dtype):
    """The same over a cache, with the two keys in one CTA's part, in the parts of two slots or of two CTAs."""
    batch, width, pos, nq, nkv = TREES[tree]
    n, inf = pos + width, float("inf")
    parents = _chain(batch, width)
    for peak, at in {(0, n - 1), (n - 1, 0), (n // 2, n // 3), (n // 3, n // 2), (0, min(130, n - 1)), (min(130, n - 1), 0)}:
        if peak == at:
            continue
        q1, k, v, scale = _far_case(8, n, nq, nkv, hd, dtype, peak)
        q = q1[:width][None].repeat(batch, 1, 1, 1)
        kc, vc = (t.transpose(0, 1)[None].repeat(batch, 1, 1, 1) for t in (k, v))
        call = lambda: lps.attention_tree_verify(q, kc, vc, parents, [pos] * batch, [width] * batch, scale=scale)  # noqa: E731
        clean = call()
        assert torch.isfinite(clean).all()
        vc[:, :, at, 3], vc[:, :, at, 40], vc[:, :, at, 50] = inf, -inf, float("nan")
        got = call()
        first = max(0, at - pos)  # the first draft that sees it
        assert (got[:, first:, :, 3] == inf).all() and (got[:, first:, :, 40] == -inf).all() and got[:, first:, :, 50].isnan().all(), (peak, at)
        others = [d for d in range(hd) if d not in (3, 40, 50)]
        assert torch.equal(got[..., others], clean[..., others]) and torch.equal(got[:, :first], clean[:, :first])
        kc[:, :, at] = -inf
        got = call()
        assert got[:, first:, :, [3, 40, 50]].isnan().all(), (peak, at)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_all_infinite_or_nan(bad):
    """A cache or a long prompt full of them is answered like any other, well within the kernels' waits."""
    for n, hd in ((8184, 128), (3000, 64)):
        q, k, v = _randn(1, n, 8, hd), _randn(2, n, 2, hd), torch.full((n, 2, hd), bad, device="cuda", dtype=BF)
        out = lps.attention_prompt_packed(q, k, v, [0, n])
        lps.cache_ops_status()
        assert out.isnan().all() if bad != bad else (out == bad).all()
        k[n // 2] = -float("inf")  # a NaN score, or one of either infinity, makes NaN of the rows that see it
        out = lps.attention_prompt_packed(q, k, v, [0, n])
        lps.cache_ops_status()
        assert out[n // 2:].isnan().all() and (bad != bad or (out[:n // 2] == bad).all())
    kc, vc, tq = _randn(3, 2, 2, 100064, 128), torch.full((2, 2, 100064, 128), bad, device="cuda", dtype=BF), _randn(4, 2, 40, 8, 128)
    out = lps.attention_tree_verify(tq, kc, vc, _chain(2, 40), [100000, 7], [40, 40])
    lps.cache_ops_status()
    assert out.isnan().all() if bad != bad else (out == bad).all()


@pytest.mark.parametrize("dtype", [BF, FP])
def test_values_near_the_types_end(dtype):
    """Large finite values stay what they are (a mean of them): o is summed in fp32 with weights of up to 2^8 a key
    (2^15 in fp16) before it is divided."""
    top = torch.finfo(dtype).max / (2.0 ** 30 if dtype == BF else 2.0)
    q, k = _randn(1, 200, 4, 64, dtype=dtype), _randn(2, 200, 2, 64, dtype=dtype)
    v = torch.full_like(k, top)
    out = lps.attention_prompt_packed(q, k, v, [0, 200]).double()
    # the weights are rounded for the product and not for the sum: off by eps / 2, and the result by as much again
    assert ((out - top).abs() <= 1.01 * torch.finfo(dtype).eps * top).all()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale", [1e-45, 1e-38, 1e-30])
def test_scales_next_to_nothing(scale, dtype):
    """All scores come to nothing: the mean of the values seen, also where scores of -inf come first. The mean is off
    by one rounding and by fp32 sums over n keys."""
    n, hd = 700, 64
    q, k, v = _randn(1, n, 4, hd, dtype=dtype).abs() + 1, _randn(2, n, 2, hd, dtype=dtype), _randn(3, n, 2, hd, dtype=dtype)
    k[:200] = -float("inf")
    kc, vc = (t.transpose(0, 1).contiguous()[None] for t in (k, v))
    prompt = lps.attention_prompt_packed(q, k, v, [0, n], scale=scale)
    tree = lps.attention_tree_verify(q[None, :5].contiguous(), kc, vc, _chain(1, 5), [n - 5], [5], scale=scale)
    for got, last in ((prompt[-1], n), (prompt[400], 401), (tree[0, 4], n), (tree[0, 0], n - 4)):
        want = v[200:last].double().mean(0)[:, None].expand(2, 2, hd).reshape(4, hd)
        tol = torch.finfo(dtype).eps / 2 * want.abs() + (2 * n + 16) * 2.0 ** -24 * v[200:last].double().abs().mean()
        assert ((got.double() - want).abs() <= tol + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps).all()


# ---- autograd ---------------------------------------------------------------------------------------

def _writers():
    """Each call that writes a given tensor, and the tensors that it writes."""
    q, k, v = _randn(1, 20, 4, 64), _randn(2, 20, 2, 64), _randn(3, 20, 2, 64)
    kc, vc, tq = _randn(4, 1, 2, 50, 64), _randn(5, 1, 2, 50, 64), _randn(6, 1, 3, 4, 64)
    path, taken = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda")
    po, to = torch.zeros_like(q), torch.zeros_like(tq)
    return {"prompt": (lambda: lps.attention_prompt_packed(q, k, v, [0, 20], out=po), [po]),
            "tree": (lambda: lps.attention_tree_verify(tq, kc, vc, _chain(1, 3), [40], [3], out=to), [to]),
            "append": (lambda: lps.kv_rows_append(k, v, [0, 20], kc, vc, [5]), [kc, vc]),
            "accept": (lambda: lps.kv_rows_accept(kc, vc, [40], path, taken), [kc, vc])}


@pytest.mark.parametrize("op", ["prompt", "tree", "append", "accept"])
def test_what_a_call_writes_is_known_to_autograd(op):
    """A tensor that an earlier product saved for its backward and a call then writes: the backward refuses, as after
    any operation in place, instead of using the new values."""
    call, outs = _writers()[op]
    for t in outs:
        w = torch.ones_like(t, requires_grad=True)
        loss = (w * t).float().sum()
        with torch.no_grad():
            call()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
        version = t._version
        with pytest.raises(lps.LpsError):  # a refused call writes nothing
            if op == "prompt":
                lps.attention_prompt_packed(t, t[:, :3], t[:, :3], [0, 20], out=t)
            elif op == "tree":
                lps.attention_tree_verify(t, _randn(4, 1, 2, 50, 64), _randn(5, 1, 2, 50, 64), _chain(1, 3), [49], [3], out=t)
            elif op == "append":
                lps.kv_rows_append(_randn(2, 20, 2, 64), _randn(3, 20, 2, 64), [0, 20], t, t.clone(), [31])
            else:
                lps.kv_rows_accept(t, t.clone(), [51], torch.zeros(1, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
        assert t._version == version
    with torch.inference_mode():  # whose tensors have no version
        call, outs = _writers()[op]
        call()
    lps.cache_ops_status()


def test_forward_derivatives_are_refused_on_the_gpu():
    import torch.autograd.forward_ad as fwd
    q, k = _randn(1, 20, 4, 64), _randn(2, 20, 2, 64)
    with fwd.dual_level():
        with pytest.raises(ValueError, match="forward derivative"):
            lps.attention_prompt_packed(fwd.make_dual(q, torch.ones_like(q)), k, k, [0, 20])
        inside = lps.attention_prompt_packed(q, k, k, [0, 20])
    assert torch.equal(inside, lps.attention_prompt_packed(q, k, k, [0, 20]))


# ---- caches in one buffer ------------------------------------------------------------------------------

def test_caches_side_by_side_in_one_buffer():
    """K and V caches as the halves of one tensor touch but do not overlap; shifted by a row they do, and are refused."""
    both = torch.zeros(2, 2, 2, 50, 64, device="cuda", dtype=FP)
    k, v = _randn(1, 20, 2, 64, dtype=FP), _randn(2, 20, 2, 64, dtype=FP)
    lps.kv_rows_append(k, v, [0, 12, 20], both[0], both[1], [3, 40])
    want = torch.zeros_like(both)
    for half, t in enumerate((k, v)):
        want[half, 0, :, 3:15], want[half, 1, :, 40:48] = t[:12].transpose(0, 1), t[12:].transpose(0, 1)
    assert torch.equal(both, want)
    path = torch.tensor([[1, 3, 0, 0], [0, 2, 0, 0]], dtype=torch.int32, device="cuda")  # draft rows below the width
    taken = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    lps.kv_rows_accept(both[0], both[1], [4, 41], path, taken)
    for b, pos in enumerate((4, 41)):
        rows = want[:, b, :, [pos + int(x) for x in path[b, :2]]].clone()
        want[:, b, :, pos:pos + 2] = rows
    assert torch.equal(both, want)
    flat = torch.zeros(2 * 2 * 2 * 50 * 64 + 64, device="cuda", dtype=FP)
    n = 2 * 2 * 50 * 64
    a, b = flat[:n].view(2, 2, 50, 64), flat[64:64 + n].view(2, 2, 50, 64)
    with pytest.raises(lps.LpsError, match="overlap"):
        lps.kv_rows_append(k, v, [0, 12, 20], a, b, [3, 40])
    with pytest.raises(lps.LpsError, match="overlap"):
        lps.kv_rows_accept(a, b, [4, 41], path, taken)
    assert not flat.any()


# ---- outputs on 16 and on 32 bytes -----------------------------------------------------------------------

def _spaced(shape, hd, shift, dtype):
    """A view of `shape` whose rows lie `shift` elements apart (8: on 16 bytes, 16: on 32), and its buffer."""
    *outer, heads, _ = shape
    buf = torch.full((*outer, heads * (hd + shift) + shift), 3.0, device="cuda", dtype=dtype)
    return buf[..., shift:].unflatten(-1, (heads, hd + shift))[..., :hd], buf


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("nq,nkv", [(3, 1), (8, 2), (14, 2)])
@pytest.mark.parametrize("hd", [64, 128])
def test_output_rows_on_16_and_on_32_bytes(hd, nq, nkv, dtype):
    """The same bits from every way out, with ragged last tiles, and with an infinity and a NaN of V that are seen;
    nothing between the rows is touched."""
    off, inf = [0, 70, 71, 331], float("inf")
    q, k, v = _randn(1, 331, nq, hd, dtype=dtype), _randn(2, 331, nkv, hd, dtype=dtype), _randn(3, 331, nkv, hd, dtype=dtype)
    kc, vc, tq = _randn(4, 2, nkv, 300, hd, dtype=dtype), _randn(5, 2, nkv, 300, hd, dtype=dtype), _randn(6, 2, 41, nq, hd, dtype=dtype)
    par = _chain(2, 41)
    for plant in (False, True):
        if plant:
            v[75, :, 5], v[200, :, hd - 1], vc[0, :, 3, 7], vc[1, :, 255, hd - 2] = inf, float("nan"), -inf, inf
        want = lps.attention_prompt_packed(q, k, v, off)
        tree = lps.attention_tree_verify(tq, kc, vc, par, [200, 240], [41, 30], out=torch.full_like(tq, 3.0))
        if plant:
            assert (want[75:, :, 5] == inf).all() and want[200:, :, hd - 1].isnan().all()
            assert (tree[0, :, :, 7] == -inf).all() and (tree[1, 15:30, :, hd - 2] == inf).all()
        for shift in (8, 16):
            out, buf = _spaced(q.shape, hd, shift, dtype)
            lps.attention_prompt_packed(q, k, v, off, out=out)
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
            out.fill_(3.0)
            assert (buf == 3.0).all()
            out, buf = _spaced(tq.shape, hd, shift, dtype)
            lps.attention_tree_verify(tq, kc, vc, par, [200, 240], [41, 30], out=out)
            assert torch.equal(out.view(torch.int16), tree.view(torch.int16))
            out.fill_(3.0)
            assert (buf == 3.0).all()


# ---- row moves of either type --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("hd", [64, 128])
def test_accept_moves_bits_of_either_type(hd, dtype):
    kc, vc = (torch.randint(-2**15, 2**15, (3, 4, 3, 90, hd), device="cuda", dtype=torch.int16).view(dtype) for _ in range(2))
    paths, pos = [[0, 3, 4, 11], [], [5], list(range(1, 12))], [70, 5, 0, 33]
    want = [kc.clone(), vc.clone()]
    path = torch.full((4, 12), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
        for w, c in zip(want, (kc, vc)):
            for i, x in enumerate(p):
                w[:, b, :, pos[b] + i] = c[:, b, :, pos[b] + x]
    lps.kv_rows_accept(kc, vc, pos, path.cuda(), torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"))
    for got, w in zip((kc, vc), want):
        assert torch.equal(got.view(torch.int16), w.view(torch.int16))


def test_a_range_of_offsets():
    q, k = _randn(1, 50, 4, 64), _randn(2, 50, 2, 64)
    got = lps.attention_prompt_packed(q, k, k, range(0, 51, 10))
    assert torch.equal(got, lps.attention_prompt_packed(q, k, k, [0, 10, 20, 30, 40, 50]))
    assert not torch.equal(got, lps.attention_prompt_packed(q, k, k, [0, 50]))
