"""The argument checks of the operators over a caller-owned cache, on the CPU: every refusal is decided
from the arguments alone, before the device is asked for anything. The addresses passed here are never
dereferenced (each call is refused first), so the test runs only where there is no device."""
import ctypes

import numpy as np
import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi
from layer_pipeline_staged_gb300 import build as lps_build


def _has_gpu() -> bool:
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


pytestmark = pytest.mark.skipif(_has_gpu(), reason="addresses here are placeholders: CPU-only test")

Q, K, V, OUT, DEV = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


@pytest.fixture(scope="module", autouse=True)
def built():
    lps_build.build()


def _i32(x):
    return (ctypes.c_int32 * max(len(x), 1))(*x)


def _i64(x):
    return None if x is None else (ctypes.c_int64 * len(x))(*x)


def prompt(q=Q, k=K, v=V, out=OUT, type=0, n=2, offsets=(0, 5, 9), nq=32, nkv=8, hd=128, strides=None, scale=0.0):
    off = None if offsets is None else _i32(offsets)
    return _capi.load().attention_prompt_packed(q, k, v, out, type, n, off, nq, nkv, hd, _i64(strides), scale, None)


def tree(q=Q, k=K, v=V, out=OUT, type=0, batch=2, width=8, pos=(3, 4), rows=(8, 1), parents=DEV, nq=32, nkv=8, hd=128,
         max_ctx=64, strides=None, scale=0.0):
    return _capi.load().attention_tree_verify(q, k, v, out, type, batch, width, None if pos is None else _i32(pos),
                                              None if rows is None else _i32(rows), parents, nq, nkv, hd, max_ctx,
                                              _i64(strides), scale, None)


def append(k=K, v=V, n=2, offsets=(0, 5, 9), kc=OUT, vc=Q, start=(0, 60), nkv=8, hd=128, max_ctx=64, strides=None):
    return _capi.load().kv_rows_append(k, v, n, None if offsets is None else _i32(offsets), kc, vc,
                                       None if start is None else _i32(start), nkv, hd, max_ctx, _i64(strides), None)


def accept(kc=K, vc=V, layers=2, batch=2, nkv=8, hd=128, max_ctx=64, pos=(0, 64), width=8, path=DEV, accepted=DEV):
    return _capi.load().kv_rows_accept(kc, vc, layers, batch, nkv, hd, max_ctx, None if pos is None else _i32(pos), width,
                                       path, accepted, None)


D8 = (4096, 128, 1024, 128, 1024, 128, 4096, 128)
CASES = [(prompt, kw, what) for kw, what in [
    (dict(q=None), "required"), (dict(k=None), "required"), (dict(v=None), "required"), (dict(out=None), "required"),
    (dict(offsets=None), "required"), (dict(n=0), "n_seqs"), (dict(n=-1), "n_seqs"), (dict(type=2), "type"),
    (dict(type=-1), "type"), (dict(hd=96), "head_dim"), (dict(nkv=0), "n_q_heads"), (dict(nq=0), "n_q_heads"),
    (dict(nq=12), "n_q_heads"), (dict(nq=34, nkv=2), "n_q_heads"), (dict(nq=70000, nkv=70000), "n_q_heads"),
    (dict(offsets=(-1, 5, 9)), "offsets"), (dict(offsets=(0, 5, 4)), "offsets"), (dict(offsets=(0, 5, 2**31 - 1)), "offsets"), (dict(scale=-0.5), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(q=Q + 2), "aligned"), (dict(k=K + 8), "aligned"), (dict(v=V + 1), "aligned"), (dict(out=OUT + 4), "aligned"),
    *[(dict(strides=D8[:i] + (bad,) + D8[i + 1:]), "strides") for i in range(8) for bad in (0, -128, 132, 64, 1 << 40)],
]] + [(tree, kw, what) for kw, what in [
    (dict(q=None), "required"), (dict(k=None), "required"), (dict(out=None), "required"), (dict(pos=None), "required"),
    (dict(rows=None), "required"), (dict(parents=None), "required"), (dict(type=7), "type"), (dict(hd=32), "head_dim"),
    (dict(nq=24, nkv=16), "n_q_heads"), (dict(batch=0), "batch"), (dict(batch=257, pos=(0,) * 257, rows=(1,) * 257), "batch"),
    (dict(width=0), "width"), (dict(width=65), "width"), (dict(max_ctx=0), "max_ctx"), (dict(pos=(-1, 0)), "pos"),
    (dict(rows=(9, 1)), "rows"), (dict(rows=(1, -1)), "rows"), (dict(pos=(57, 0)), "max_ctx"),
    (dict(pos=(0, 2**31 - 1)), "max_ctx"), (dict(max_ctx=2**31 - 1), "max_ctx"), (dict(scale=-1.0), "scale"), (dict(k=K + 2), "aligned"),
    (dict(strides=(4096, 4096, 100, 32768, 4096, 128)), "strides"), (dict(strides=(0, 4096, 128, 32768, 4096, 128)), "strides"),
]] + [(append, kw, what) for kw, what in [
    (dict(k=None), "required"), (dict(kc=None), "required"), (dict(start=None), "required"), (dict(n=0), "n_seqs"),
    (dict(offsets=(3, 2, 9)), "offsets"), (dict(start=(0, 61)), "start"), (dict(start=(-1, 0)), "start"),
    (dict(start=(65, 0), offsets=(0, 0, 1)), "start"), (dict(start=(0, 2**31 - 1)), "start"), (dict(hd=80), "head_dim"),
    (dict(nkv=0), "n_q_heads"), (dict(max_ctx=0), "max_ctx"), (dict(kc=OUT + 2), "aligned"), (dict(vc=OUT), "differ"),
    (dict(strides=(1024, 128, 1024, 4)), "strides"),
]] + [(accept, kw, what) for kw, what in [
    (dict(kc=None), "required"), (dict(path=None), "required"), (dict(accepted=None), "required"), (dict(pos=None), "required"),
    (dict(layers=0), "n_layers"), (dict(layers=32768), "n_layers"), (dict(batch=0), "batch"), (dict(width=65), "width"),
    (dict(width=0), "width"), (dict(pos=(0, 65)), "pos"), (dict(pos=(-1, 0)), "pos"), (dict(hd=256), "head_dim"),
    (dict(vc=V + 4), "aligned"), (dict(vc=K), "differ"), (dict(max_ctx=2**31 - 1), "max_ctx"),
]]


@pytest.mark.parametrize("call,kw,what", CASES, ids=[f"{c.__name__}-{i}" for i, (c, _, _) in enumerate(CASES)])
def test_refused_before_the_device(call, kw, what):
    assert call(**kw) == lps.LPS_EINVAL
    err = _capi.load().last_error_string().decode()
    assert what in err, err


def test_wrappers_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    q, k = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        lps.attention_prompt_packed(q, k, k, [0, 4])
    with pytest.raises(ValueError, match="tokens"):
        lps.attention_prompt_packed(q, k[:3], k, [0, 4])
    with pytest.raises(ValueError, match="bfloat16"):
        lps.attention_prompt_packed(q.float(), k.float(), k.float(), [0, 4])
    kc = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lps.kv_rows_append(k, k, [0, 2, 4], kc, kc[:1], [0, 0])
    with pytest.raises(ValueError):
        lps.kv_rows_accept(kc, kc[:1], [0, 0], np.zeros((2, 4), np.int32), np.zeros(2, np.int32))


def test_wrappers_read_host_integers():
    """Lists, arrays of 32 and 64 bits, strided arrays and CPU tensors are host integers; floats, booleans, two
    axes, too many values and values past 32 bits are not. Each call is refused for its tensors or for its
    integers, so what the message names tells which was reached."""
    torch = pytest.importorskip("torch")
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    kc = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16)
    from layer_pipeline_staged_gb300 import ops
    ops._ready()
    # CPU tensors are refused before the integers are read, by every wrapper
    for call in (lambda: lps.kv_rows_append(k, k, [0, 2, 4], kc, kc.clone(), [0, 0]),
                 lambda: lps.attention_prompt_packed(k, k, k, np.array([0, 4])),
                 lambda: lps.attention_tree_verify(kc, kc, kc, torch.zeros(2, 2, dtype=torch.int32), [0, 0], [1, 1]),
                 lambda: lps.kv_rows_accept(kc, kc.clone(), [0, 0], torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    for bad in (None, 3, "q", np.zeros((4, 2, 64))):
        with pytest.raises(TypeError):
            lps.attention_prompt_packed(bad, k, k, [0, 4])
