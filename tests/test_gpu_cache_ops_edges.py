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
