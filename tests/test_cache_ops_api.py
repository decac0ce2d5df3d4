"""The package's face of the operators over a caller-owned cache, as far as it shows without a GPU."""
import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import build as lps_build
from layer_pipeline_staged_gb300 import ops


@pytest.fixture(scope="module", autouse=True)
def built():
    lps_build.build()


def test_every_operator_and_the_status_are_exported():
    for name in ops.__all__:
        assert name in lps.__all__ and getattr(lps, name) is getattr(ops, name)
    assert "cache_ops_status" in ops.__all__
    for name in ("attention_prompt_packed", "attention_tree_verify"):
        assert "cache_ops_status" in getattr(ops, name).__doc__


def test_status_raises_what_the_library_says(monkeypatch):
    """The status call goes to the library with the stream's handle on the stream's device, and its refusal is raised."""
    torch = pytest.importorskip("torch")
    from contextlib import contextmanager

    from layer_pipeline_staged_gb300 import _capi
    seen = []

    class Stream:
        device, cuda_stream = "the device", 77

    class Library:
        rc = lps.LPS_ECUDA

        def cache_ops_status(self, stream):
            seen.append(stream)
            return self.rc

        def last_error_string(self):
            return b"gave up"

    @contextmanager
    def on(device):
        seen.append(device)
        yield

    library = Library()
    monkeypatch.setattr(_capi, "load", lambda: library)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream)
    with pytest.raises(lps.LpsError, match="gave up") as e:
        lps.cache_ops_status()
    assert e.value.code == lps.LPS_ECUDA and seen == ["the device", 77]
    library.rc = lps.LPS_OK
    assert lps.cache_ops_status(Stream) is None


def _calls(torch, mark):
    """Every operator's call on CPU tensors, with `mark` applied to one tensor argument after the other. Unmarked
    they are refused because the tensors are not on a GPU."""
    bf = torch.bfloat16
    q, k = torch.zeros(4, 4, 64, dtype=bf), torch.zeros(4, 2, 64, dtype=bf)
    tq, kc = torch.zeros(2, 3, 4, 64, dtype=bf), torch.zeros(2, 2, 8, 64, dtype=bf)
    par, path, taken = torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for fn, tensors, call in (
            (lps.attention_prompt_packed, [q, k, k.clone(), q.clone()], lambda f, q, k, v, o: f(q, k, v, [0, 4], out=o)),
            (lps.attention_tree_verify, [tq, kc, kc.clone(), tq.clone()], lambda f, q, k, v, o: f(q, k, v, par, [0, 0], [1, 1], out=o)),
            (lps.kv_rows_append, [k, k.clone(), kc, kc.clone()], lambda f, k, v, kc, vc: f(k, v, [0, 2, 4], kc, vc, [0, 0])),
            (lps.kv_rows_accept, [kc, kc.clone()], lambda f, kc, vc: f(kc, vc, [0, 0], path, taken))):
        with pytest.raises(ValueError, match="CUDA"):
            call(fn, *tensors)
        for i in range(len(tensors)):
            marked = [mark(t) if i == j else t for j, t in enumerate(tensors)]
            yield lambda: call(fn, *marked)


def test_forward_derivatives_are_refused():
    """A dual tensor has requires_grad False and its primal's memory: its tangent would be lost without a word."""
    torch = pytest.importorskip("torch")
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level():
        for call in _calls(torch, lambda t: fwd.make_dual(t, torch.ones_like(t))):
            with pytest.raises(ValueError, match="forward derivative"):
                call()
            with torch.no_grad(), pytest.raises(ValueError, match="forward derivative"):
                call()
        for call in _calls(torch, lambda t: fwd.unpack_dual(fwd.make_dual(t, torch.ones_like(t))).primal):
            with pytest.raises(ValueError, match="CUDA"):
                call()


def test_negative_views_are_refused():
    """A view whose sign is still to be changed (the imaginary part of a conjugate) holds other values than it shows."""
    torch = pytest.importorskip("torch")
    lazy = torch.zeros(2, 2, dtype=torch.complex64).conj().imag
    assert lazy.is_neg()
    for call in _calls(torch, torch._neg_view):
        with pytest.raises(ValueError, match="resolve_neg"):
            call()
    for call in _calls(torch, lambda t: torch._neg_view(t).resolve_neg()):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.mark.parametrize("scale", [1e-46, 2.0 ** -150, 5e-324, -1e-50])
def test_a_scale_that_32_bits_do_not_hold_is_refused(scale):
    """It would come to 0, which stands for 1/sqrt(head_dim)."""
    torch = pytest.importorskip("torch")
    q, kc = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    par = torch.zeros(2, 3, dtype=torch.int32)
    for call in (lambda s: lps.attention_prompt_packed(q[0], q[0], q[0], [0, 3], scale=s),
                 lambda s: lps.attention_tree_verify(q, kc, kc, par, [0, 0], [1, 1], scale=s)):
        with pytest.raises(ValueError, match="scale"):
            call(scale)
        for fits in (0, 0.0, 2.0 ** -149, 0.1):
            with pytest.raises(ValueError, match="CUDA"):
                call(fits)


# ---- host integers -------------------------------------------------------------------------------------------

class _Int:
    def __init__(self, x):
        self.x = x

    def __index__(self):
        return self.x


def _ints(values, n=-1):
    return ops._ready().host_ints(values, n)


def test_host_integers_are_read_from_every_kind():
    """Lists, tuples, ranges, arrays of several types, byte orders, strides and directions, CPU tensors, and any
    object with __index__."""
    np, torch = pytest.importorskip("numpy"), pytest.importorskip("torch")
    want, wide = [-5, 0, 2**31 - 1, -2**31], np.zeros((4, 3), np.int64)
    wide[:, 1] = want
    for values in (want, tuple(want), np.array(want), np.array(want, np.int32), np.array(want, np.int32)[::-1][::-1], wide[:, 1],
                   np.array(want[::-1])[::-1], np.array(want, ">i4"), np.array(want, ">i8"), np.array(want, "<i8"), torch.tensor(want),
                   torch.tensor(want, dtype=torch.int32), torch.tensor(wide[:, 1]), [_Int(x) for x in want], [np.int64(x) for x in want]):
        assert _ints(values) == want and _ints(values, 4) == want
    assert _ints(range(0, 51, 10)) == [0, 10, 20, 30, 40, 50]
    for t in (np.uint8, np.int8, np.uint16, np.int16, np.uint32, np.uint64):
        assert _ints(np.array([0, 3, 100], t)) == [0, 3, 100]
    many = list(range(1000))  # more than the call's own room
    assert _ints(many) == _ints(np.array(many)) == _ints(np.array(many, np.int32)[:], 1000) == many
    assert _ints([]) == _ints(np.zeros(0, np.int32)) == _ints((), 0) == []


def test_what_is_not_a_row_of_host_integers_is_refused():
    np, torch = pytest.importorskip("numpy"), pytest.importorskip("torch")
    for values in ([0.0, 1.0], np.array([0.0, 1.0]), np.array([0, 1], np.float16), np.array([False, True]), np.array([[0, 1]]), np.array(3),
                   [0, 2**31], [-2**31 - 1, 0], np.array([0, 2**31]), np.array([0, 2**32 - 1], np.uint32), np.array([2**63], np.uint64),
                   [2**70], ["0"], [None], torch.tensor([0.5]), torch.tensor([[1, 2]]), np.array([1j])):
        with pytest.raises(ValueError):
            _ints(values)
    for values in (None, 7, object()):
        with pytest.raises(TypeError):
            _ints(values)
    for values in ([0, 1], np.array([0, 1]), np.array([0, 1], np.int16)):
        for n in (0, 1, 3):
            with pytest.raises(ValueError, match="must hold"):
                _ints(values, n)

    class Emptying:
        def __index__(self):
            values.clear()
            return 0

    values = [Emptying()] + [1] * 40
    with pytest.raises(ValueError, match="changed"):
        _ints(values)

    class Failing:
        def __index__(self):
            raise KeyError("no")

    with pytest.raises(ValueError, match="integers"):
        _ints([0, Failing()])


# ---- the library's own refusals, with addresses that are never dereferenced ------------------------------

def _no_gpu():
    try:
        import torch
        return not torch.cuda.is_available()
    except Exception:
        return True


cpu_only = pytest.mark.skipif(not _no_gpu(), reason="addresses here are placeholders")


def _i32(*x):
    import ctypes
    return (ctypes.c_int32 * len(x))(*x)


def _refused(rc, what):
    from layer_pipeline_staged_gb300 import _capi
    assert rc == lps.LPS_EINVAL
    err = _capi.load().last_error_string().decode()
    assert what in err, err


@cpu_only
@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_a_scale_whose_product_overflows_is_refused(scale):
    L = lps.load()
    _refused(L.attention_prompt_packed(0x10000, 0x20000, 0x30000, 0x40000, 0, 1, _i32(0, 5), 8, 2, 64, None, scale, None), "scale")
    _refused(L.attention_tree_verify(0x10000, 0x20000, 0x30000, 0x40000, 0, 1, 4, _i32(3), _i32(4), 0x50000, 8, 2, 64, 64, None, scale,
                                     None), "scale")


@cpu_only
def test_caches_that_overlap_are_refused():
    """Rows of both would be moved at once: which of them stays would be a matter of time."""
    L, one, base = lps.load(), 2 * 2 * 64 * 64 * 2, 0x1000000  # bytes of [2][2][64][64]
    for other in (base + 16, base + one - 16, base - 16, base - one + 16):
        _refused(L.kv_rows_append(0x10000, 0x20000, 2, _i32(0, 5, 9), base, other, _i32(0, 0), 2, 64, 64, None, None), "overlap")
        _refused(L.kv_rows_accept(base, other, 1, 2, 2, 64, 64, _i32(0, 0), 8, 0x30000, 0x40000, None), "overlap")
    _refused(L.kv_rows_accept(base, base + one, 3, 2, 2, 64, 64, _i32(0, 0), 8, 0x30000, 0x40000, None), "overlap")


# ---- the marshalling extension ---------------------------------------------------------------------------

def test_the_extension_is_named_for_its_python():
    import os
    import sysconfig
    assert lps_build.MARSHAL.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.exists(lps_build.MARSHAL)
    assert not os.path.exists(os.path.join(lps_build.HERE, "_marshal.so"))
    ops._ready()
    assert os.path.samefile(ops._m.__file__, lps_build.MARSHAL)


def test_without_python_headers_the_library_is_built(monkeypatch, tmp_path, capsys):
    """The C library needs no Python: its build goes on without the extension, and the wrappers say what is missing."""
    import os
    import sys
    import sysconfig
    paths = sysconfig.get_paths()
    monkeypatch.setattr(lps_build.sysconfig, "get_paths", lambda: dict(paths, include=str(tmp_path)))
    monkeypatch.setattr(lps_build, "MARSHAL", str(tmp_path / "_marshal.so"))
    assert lps_build.build() == lps_build.LIB and os.path.exists(lps_build.LIB)
    assert not os.path.exists(tmp_path / "_marshal.so") and "Python.h" in capsys.readouterr().err
    monkeypatch.setitem(sys.modules, "layer_pipeline_staged_gb300._marshal", None)
    monkeypatch.delattr(lps, "_marshal", raising=False)
    monkeypatch.setattr(ops, "_m", None)
    with pytest.raises(RuntimeError, match="build it first"):
        lps.kv_rows_append(None, None, [0], None, None, [])
