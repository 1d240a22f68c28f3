"""What the Python binding of the 4-bit KV cache keeps from one call for the next, and the streams it runs on, with the
library replaced by one that writes down what it is given (no GPU needed)."""
import ctypes as C

import numpy as np
import pytest
import torch

from block_scaled_fp4_fp4q_amd import binding as B


class Recorder:
    """Stands for the library: remembers the attention calls, succeeds, and asks for max_kv bytes of workspace."""

    def __init__(self):
        self.calls = []

    def fp4q_attend_workspace_bytes(self, spec, cache, call):
        return call._obj.max_kv

    def fp4q_attend(self, spec, cache, call, space, need, stream):
        c = call._obj
        self.calls.append(dict(max_kv=c.max_kv, max_q=c.max_q, window=c.window, causal=c.causal, scale=c.scale, need=need))
        return 0


@pytest.fixture
def lib(monkeypatch):
    lib = Recorder()
    monkeypatch.setattr(B, "_lib_handle", lambda: lib)
    monkeypatch.setattr(B, "_current_stream", lambda index: 0)
    return lib


def cache():
    t = [torch.zeros(4, 2, 16, 64, dtype=torch.uint8), torch.zeros(4, 2, 16, 8, dtype=torch.uint8), torch.ones(1)]
    return B.KvCache(*t, *[x.clone() for x in t], require_cuda=False)


def args():
    return dict(q=torch.zeros(4, 8, 128), kv_lens=torch.zeros(4, dtype=torch.int32),
                q_starts=torch.zeros(5, dtype=torch.int32))


def test_numbers_changed_in_place_are_read_again(lib):
    """0-dimensional tensors and arrays count as numbers: their values at the call, not their identity."""
    c, a = cache(), args()
    for make in (torch.tensor, np.array):
        kv, q, win, scale, causal = make(100), make(2), make(5), make(0.5), make(True)
        B.attend(c, max_kv=kv, max_q=q, window=win, scale=scale, causal=causal, **a)
        assert lib.calls[-1] == dict(max_kv=100, max_q=2, window=5, causal=1, scale=0.5, need=100)
        kv += 28
        q += 1
        scale *= 0.5
        win *= 0
        causal &= False
        B.attend(c, max_kv=kv, max_q=q, window=win, scale=scale, causal=causal, **a)
        assert lib.calls[-1] == dict(max_kv=128, max_q=3, window=0, causal=0, scale=0.25, need=128)
    kept = [x for key in c._calls for x in key if not isinstance(x, (tuple, int, float, type(None)))]
    assert not kept, f"objects of the caller kept: {kept}"


def test_sizes_that_are_no_integers_are_refused(lib):
    c, a = cache(), args()
    B.attend(c, max_kv=64, max_q=2, window=4, **a)  # an equal key where 64.0 is taken for 64
    for kw in (dict(max_kv=64.0), dict(max_q=2.0), dict(window=4.0), dict(max_kv="64"), dict(scale="1")):
        with pytest.raises((TypeError, ValueError)):
            B.attend(c, **{**a, **dict(max_kv=64, max_q=2, window=4), **kw})
    for kw in (dict(max_kv=64.0), dict(max_q=2.0), dict(window=4.0)):
        with pytest.raises(TypeError):
            B.attend_workspace_bytes(c, a["q"], a["kv_lens"], q_starts=a["q_starts"], **kw)


def test_streams_of_another_device_are_refused(monkeypatch):
    """Such a stream would make its device the current one, and the call would run on the cache's device's own stream."""
    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)

    c = cache()
    monkeypatch.setattr(c, "device", torch.device("cuda", 0))
    slots, x = torch.zeros(2, dtype=torch.int64), torch.zeros(2, 2, 128)
    for call in (lambda s: B.kv_write(c, x, x, slots, stream=s), lambda s: B.kv_read(c, slots, stream=s),
                 lambda s: B.attend(c, torch.zeros(2, 2, 128), torch.zeros(2, dtype=torch.int32), stream=s)):
        with pytest.raises(ValueError, match="stream"):
            call(Stream(1))
    B._on(torch.device("cuda", 0), Stream(0))  # nothing is entered yet
