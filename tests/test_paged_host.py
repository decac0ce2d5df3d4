"""The argument checks of the operators over pages and of the logits' adjustment, and the frequencies, on the CPU: every
refusal is decided from the arguments alone. The addresses passed here are never dereferenced (each call is refused
first), so the refusals run only where there is no device."""
import ctypes
import math
import os

import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi
from layer_pipeline_staged_gb300 import build as lps_build

torch = pytest.importorskip("torch")
no_device = pytest.mark.skipif(torch.cuda.is_available(), reason="addresses here are placeholders: CPU-only test")

A = [0x100000 * (i + 1) for i in range(20)]


@pytest.fixture(scope="module", autouse=True)
def built():
    lps_build.build()


def _i64(x):
    return None if x is None else (ctypes.c_int64 * len(x))(*x)


def rows(q=A[0], k=A[1], qo=A[2], ko=A[3], type=0, tokens=5, pos=A[4], freqs=A[5], rot=64, inter=0, mag=1.0, nq=8, nkv=2, hd=64,
         strides=None):
    return _capi.load().rotary_rows(q, k, qo, ko, type, tokens, pos, freqs, rot, inter, mag, nq, nkv, hd, _i64(strides), None)


def append(q=A[0], k=A[1], v=A[2], qo=A[3], type=0, tokens=5, seqs=2, off=A[4], len=A[5], table=A[6], width=4, kp=A[7], vp=A[17],
           pages=10, page=16, pos=None, freqs=A[9], rot=64, inter=0, mag=1.0, kw=None, nq=8, nkv=2, hd=64, strides=None):
    return _capi.load().rotary_append_paged(q, k, v, qo, type, tokens, seqs, off, len, table, width, kp, vp, pages, page, pos, freqs,
                                            rot, inter, mag, kw, nq, nkv, hd, _i64(strides), None)


def decode(q=A[0], kp=A[1], vp=A[2], out=A[3], type=0, batch=2, len=A[4], table=A[5], width=4, pages=10, page=16, nq=8, nkv=2,
           hd=64, strides=None, scale=0.0, kw=None, decay=1.0, ws=A[6], bytes=0):
    return _capi.load().attention_paged_decode(q, kp, vp, out, type, batch, len, table, width, pages, page, nq, nkv, hd, _i64(strides),
                                               scale, kw, decay, ws, bytes, None)


def evict(kp=A[0], vp=A[10], kw=A[2], pages=10, page=16, nkv=2, hd=64, batch=2, len=A[3], table=A[4], width=4, fresh=A[5], fw=2,
          new=A[6], budget=32, recent=4, ws=A[7], bytes=1 << 20):
    return _capi.load().kv_pages_evict(kp, vp, kw, pages, page, nkv, hd, batch, len, table, width, fresh, fw, new, budget, recent, ws,
                                       bytes, None)


def logits(x=A[0], out=A[1], type=2, batch=2, vocab=100, strides=None, tokens=A[2], width=8, len=A[3], prompt=None, rep=None,
           freq=None, pres=None, ids=A[4], bias=A[5], n=3, allowed=None):
    return _capi.load().logits_adjust(x, out, type, batch, vocab, _i64(strides), tokens, width, len, prompt, rep, freq, pres, ids,
                                      bias, n, allowed, None)


HEADS = [dict(nkv=0), dict(nkv=65536), dict(hd=32), dict(hd=256), dict(type=2), dict(type=-1)]
PAGES = [dict(pages=0), dict(page=0), dict(page=4), dict(page=20), dict(page=65544), dict(width=0), dict(width=2 ** 27)]
TURN = [dict(rot=-16), dict(rot=8), dict(rot=80), dict(rot=24), dict(freqs=None), dict(mag=math.inf), dict(mag=math.nan)]


@no_device
@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(tokens=-1), dict(nq=0),
                                dict(q=A[0] + 8), dict(ko=A[3] + 2), dict(strides=[512, 64, 128, 64, 512, 63, 128, 64]),
                                dict(strides=[512, 64, 128, 64, 512, 64, 100, 64]), *HEADS, *TURN])
def test_rows_refused(kw):
    assert rows(**kw) == lps.LPS_EINVAL and "rotary_rows" in _capi.load().last_error_string().decode()


@no_device
@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(len=None), dict(table=None), dict(kp=None),
                                dict(vp=None), dict(off=None), dict(tokens=-1), dict(seqs=0), dict(nq=0), dict(v=A[2] + 4),
                                dict(kp=A[7] + 8), dict(vp=A[7]), dict(vp=A[7] + 10 * 16 * 2 * 64 * 2 - 16), dict(strides=[8] * 8),
                                *HEADS, *PAGES, *TURN])
def test_append_refused(kw):
    assert append(**kw) == lps.LPS_EINVAL and "rotary_append_paged" in _capi.load().last_error_string().decode()


@no_device
@pytest.mark.parametrize("kw", [dict(q=None), dict(kp=None), dict(vp=None), dict(out=None), dict(len=None), dict(table=None), dict(ws=None),
                                dict(batch=0), dict(batch=1025), dict(nq=0), dict(nq=9), dict(nq=34), dict(out=A[3] + 2), dict(out=A[0]), dict(ws=A[6] + 8),
                                dict(strides=[512, 64, 512, 60]), dict(scale=-1.0), dict(scale=math.nan), dict(scale=3e38),
                                dict(decay=-0.1), dict(decay=1.1), dict(decay=math.nan), dict(nq=65528, nkv=65528, width=2 ** 22, page=64),
                                *HEADS, *PAGES])
def test_decode_refused(kw):
    assert decode(**kw) == lps.LPS_EINVAL and "attention_paged_decode" in _capi.load().last_error_string().decode()


@no_device
@pytest.mark.parametrize("args", [(0, 8, 2, 64, 16, 4, 0), (1025, 8, 2, 64, 16, 4, 0), (1, 8, 3, 64, 16, 4, 0), (1, 8, 2, 80, 16, 4, 1),
                                  (1, 8, 2, 64, 12, 4, 0), (1, 8, 2, 64, 16, 0, 0)])
def test_workspace_refused(args):
    assert _capi.load().attention_paged_decode_workspace(*args) == lps.LPS_EINVAL


@no_device
@pytest.mark.parametrize("kw", [dict(kp=None), dict(vp=None), dict(kw=None), dict(len=None), dict(table=None), dict(fresh=None), dict(new=None),
                                dict(ws=None), dict(batch=0), dict(batch=65536), dict(budget=0), dict(budget=33), dict(recent=-1),
                                dict(recent=33), dict(fw=0), dict(new=A[3]), dict(fresh=A[4]), dict(ws=A[7] + 2), dict(bytes=2 * 2 * 32 * 4 - 1),
                                dict(kp=A[0] + 8), dict(vp=A[0] + 16), dict(kw=A[2] + 8), *[h for h in HEADS if "type" not in h], *PAGES])
def test_evict_refused(kw):
    assert evict(**kw) == lps.LPS_EINVAL and "kv_pages_evict" in _capi.load().last_error_string().decode()
    assert _capi.load().kv_pages_evict_workspace(1, 2, 0) == lps.LPS_EINVAL
    assert _capi.load().kv_pages_evict_workspace(3, 2, 100000) == 3 * 2 * 100000 * 4


@no_device
@pytest.mark.parametrize("kw", [dict(x=None), dict(out=None), dict(type=3), dict(type=-1), dict(batch=0), dict(batch=65536), dict(vocab=0),
                                dict(vocab=2 ** 31 - 1), dict(width=-1), dict(n=-1), dict(tokens=None), dict(len=None), dict(ids=None),
                                dict(bias=None), dict(width=0, rep=A[6]), dict(width=0, freq=A[6]), dict(width=0, pres=A[6]),
                                dict(strides=[99, 100]), dict(strides=[100, 2 ** 38]), dict(x=A[0] + 2), dict(type=0, out=A[1] + 1)])
def test_logits_refused(kw):
    assert logits(**kw) == lps.LPS_EINVAL and "logits_adjust" in _capi.load().last_error_string().decode()


def test_frequencies():
    f = lps.rotary_frequencies(64, 10000.0)
    assert f.dtype == torch.float64 and f.shape == (32,) and f[0] == 1.0
    assert abs(float(f[16]) - 0.01) < 1e-17 and (f[1:] < f[:-1]).all()
    assert torch.equal(lps.rotary_frequencies(64, 10000.0, "linear", 4.0), f / 4.0)
    ntk = lps.rotary_frequencies(64, 10000.0, "ntk", 4.0)
    assert ntk[0] == 1.0 and abs(float(ntk[-1] * 4.0 / f[-1]) - 1.0) < 1e-12
    parts = lps.rotary_frequencies(64, 10000.0, "parts", 4.0, original=2048, slow=1.0, fast=32.0)
    turns = 2048 * f / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], f[turns >= 32]) and torch.allclose(parts[turns <= 1], f[turns <= 1] / 4, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and (parts[between] < f[between]).all() and (parts[between] > f[between] / 4).all()
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=64, theta=0.0), dict(rot_dim=64, theta=math.inf), dict(rot_dim=64, factor=0.5),
                dict(rot_dim=64, scaling="parts"), dict(rot_dim=64, scaling="parts", original=10, slow=4.0, fast=4.0),
                dict(rot_dim=64, scaling="more"), dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            lps.rotary_frequencies(**bad)


def _calls():
    """(call, its tensors) of every operator on CPU tensors, which are refused because they are on no GPU."""
    bf = torch.bfloat16
    q, k, pool = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(2, 2, 64, dtype=bf), torch.zeros(5, 2, 16, 64, dtype=bf)
    i = torch.zeros(2, dtype=torch.int32)
    tab, f, kw = torch.zeros(2, 3, dtype=torch.int32), torch.ones(32, dtype=torch.float64), torch.zeros(5, 2, 16)
    return [(lambda q, k: lps.rotary_rows(q, k, i, f), [q, k]),
            (lambda q, k, qo, ko: lps.rotary_rows(q, k, i, f, out=(qo, ko)), [q, k, q.clone(), k.clone()]),
            (lambda q, k, v, kp, vp, o: lps.rotary_append_paged(q, k, v, None, i, tab, kp, vp, f, key_weights=kw, q_out=o),
             [q, k, k.clone(), pool, pool.clone(), q.clone()]),
            (lambda q, kp, vp, o: lps.attention_paged_decode(q, kp, vp, tab, i, key_weights=kw, out=o), [q, pool, pool.clone(), q.clone()]),
            (lambda kp, vp: lps.kv_pages_evict(kp, vp, kw, tab, i, tab.clone(), 16), [pool, pool.clone()]),
            (lambda x, o: lps.logits_adjust(x, out=o), [torch.zeros(2, 50), torch.zeros(2, 50)])]


def test_tensors_off_the_gpu_and_of_other_kinds_are_refused():
    import torch.autograd.forward_ad as fwd
    for call, tensors in _calls():
        with pytest.raises(ValueError, match="CUDA"):
            call(*tensors)
        for n in range(len(tensors)):
            for wrong in (None, 3, torch.zeros(2), tensors[n].double()):
                with pytest.raises((ValueError, TypeError)):
                    call(*[wrong if m == n else t for m, t in enumerate(tensors)])
            with fwd.dual_level(), pytest.raises(ValueError, match="forward derivative"):
                call(*[fwd.make_dual(t, torch.ones_like(t)) if m == n else t for m, t in enumerate(tensors)])


def test_the_quick_way_of_reading_tensors_is_for_one_torch(monkeypatch):
    from layer_pipeline_staged_gb300 import ops
    if lps_build._torch() is None:
        pytest.skip("this torch has no headers")
    assert ops._tensors(torch) is not None
    monkeypatch.setattr(torch, "__version__", "0.1.2+other")
    assert ops._tensors(torch) is None


@pytest.mark.parametrize("cxx", ["/bin/false", "/no/such/compiler"])
def test_a_build_without_the_quick_way_of_reading_tensors(monkeypatch, tmp_path, capfd, cxx):
    """It is left out where it does not compile, an older one too, and the library is built all the same."""
    if lps_build._torch() is None:
        pytest.skip("this torch has no headers")
    older = tmp_path / "_tensors.so"
    older.write_bytes(b"")
    os.utime(older, (0, 0))
    monkeypatch.setattr(lps_build, "TENSORS", str(older))
    monkeypatch.setenv("CXX", cxx)
    assert lps_build.build() == lps_build.LIB and os.path.exists(lps_build.LIB)
    assert list(tmp_path.iterdir()) == [] and "Python interface" in capfd.readouterr().err
