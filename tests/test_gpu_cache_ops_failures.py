"""What the operators over a caller-owned cache do when one of their bounded waits gives up: the call ends,
says so in the status word, and leaves the GPU as it found it for the next call."""
import re

import numpy as np
import pytest

import layer_pipeline_staged_gb300 as lps
from layer_pipeline_staged_gb300 import _capi

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _status():
    return _capi.load().cache_ops_status(torch.cuda.current_stream().cuda_stream)


def _prompt(hd):
    """More items than SMs, so that CTAs take others over, of very different lengths."""
    g = torch.Generator("cuda").manual_seed(7)
    off = np.concatenate([[0], np.cumsum([2100, 33, 700, 129, 1, 1000, 64])]).astype(np.int32)
    q, k, v = (torch.randn(int(off[-1]), h, hd, generator=g, device="cuda").to(torch.bfloat16) for h in (32, 8, 8))
    return lambda: lps.attention_prompt_packed(q, k, v, off)


def _tree(width, batch, pos, nq, nkv, hd):
    g = torch.Generator("cuda").manual_seed(8)
    rng = np.random.default_rng(8)
    q = torch.randn(batch, width, nq, hd, generator=g, device="cuda").to(torch.float16)
    kc, vc = (torch.randn(batch, nkv, pos + width, hd, generator=g, device="cuda").to(torch.float16) for _ in range(2))
    par = torch.from_numpy(np.stack([rng.integers(-1, t, size=batch) for t in range(width)], 1).astype(np.int32)).cuda()
    at = [pos if b % 2 == 0 else pos // 3 for b in range(batch)]
    return lambda: lps.attention_tree_verify(q, kc, vc, par, at, [width] * batch)


CASES = {
    "prompt-128": lambda: _prompt(128),
    "prompt-64": lambda: _prompt(64),
    "tree-solo": lambda: _tree(26, 2, 4000, 32, 8, 128),  # one tile over both slots, joined over a cluster
    "tree-pair": lambda: _tree(64, 3, 3000, 32, 8, 128),  # two tiles, joined over a cluster
    "tree-many": lambda: _tree(64, 40, 300, 16, 4, 64),   # clusters of one, not joined
}


@pytest.mark.parametrize("cycles", [1, 500, 2000, 5000, 20000])
@pytest.mark.parametrize("name", CASES)
def test_a_wait_that_gives_up_is_reported(name, cycles):
    """With a wait limit too short for some or all of a call's waits, the call ends; either nothing gave up and its
    output is right, or the status word says which kernel did. The next call, with the default limit, is right."""
    L, call = _capi.load(), CASES[name]()
    assert _status() == lps.LPS_OK
    ref = call()
    assert _status() == lps.LPS_OK
    given_up = 0
    try:
        assert L.cache_ops_set_wait_limit(cycles) == lps.LPS_OK
        for _ in range(3):
            out = call()
            rc = _status()
            if rc == lps.LPS_OK:
                assert torch.equal(out, ref)
            else:
                assert rc == lps.LPS_ECUDA
                err = L.last_error_string().decode()
                assert "packed-prompt / drafted-tree attention" in err and "timed out" in err, err
                kinds = int(re.search(r"status 0x([0-9a-f]+)", err).group(1), 16)
                assert kinds and not kinds & 4, err  # what the CTAs had issued has landed before they ended
                given_up += 1
    finally:
        assert L.cache_ops_set_wait_limit(0) == lps.LPS_OK
    assert given_up == 3 or cycles > 1, "a wait of one cycle is too short for a copy from memory"
    assert torch.equal(call(), ref)
    assert _status() == lps.LPS_OK


def test_wait_limit_is_the_calling_threads():
    import threading
    call = CASES["prompt-64"]()
    ref, got, rc = call(), [], []

    def other():
        torch.cuda.synchronize()
        got.append(call())
        rc.append(_status())

    L = _capi.load()
    try:
        assert L.cache_ops_set_wait_limit(1) == lps.LPS_OK
        t = threading.Thread(target=other)
        t.start()
        t.join()
    finally:
        assert L.cache_ops_set_wait_limit(0) == lps.LPS_OK
    assert rc == [lps.LPS_OK] and torch.equal(got[0], ref)
    assert L.cache_ops_set_wait_limit(-1) == lps.LPS_EINVAL


def test_the_package_reports_a_wait_that_gave_up():
    """cache_ops_status of the package raises once, on the stream it is asked about, and then is clear."""
    L, call = _capi.load(), CASES["prompt-128"]()
    side = torch.cuda.Stream()
    call()
    lps.cache_ops_status()
    side.wait_stream(torch.cuda.current_stream())
    try:
        assert L.cache_ops_set_wait_limit(1) == lps.LPS_OK
        with torch.cuda.stream(side):
            call()
    finally:
        assert L.cache_ops_set_wait_limit(0) == lps.LPS_OK
    with pytest.raises(lps.LpsError, match="output is invalid") as e:
        lps.cache_ops_status(side)
    assert e.value.code == lps.LPS_ECUDA
    lps.cache_ops_status(side)
    lps.cache_ops_status()
