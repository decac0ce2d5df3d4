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
