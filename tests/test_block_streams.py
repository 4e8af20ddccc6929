"""The block operators with a stream of their own: what a call copies or
allocates on the way is the stream's."""
import contextlib

import pytest
import torch

from dispatch_combine_gb300 import _lib


@pytest.fixture
def trace(monkeypatch):
    """Calls of the binding on CPU tensors, with the stream that was current
    when memory was allocated or copied."""
    seen, current = [], ["current"]

    @contextlib.contextmanager
    def using(stream):
        current.append(stream)
        yield
        current.pop()

    real_empty, real_contiguous = torch.empty, torch.Tensor.contiguous

    def empty(*a, **kw):
        seen.append(("empty", current[-1]))
        return real_empty(*a, **kw)

    def contiguous(t):
        if not t.is_contiguous():
            seen.append(("copy", current[-1]))
        return real_contiguous(t)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.Tensor, "contiguous", contiguous)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: seen.append(("kept for", s)))
    monkeypatch.setattr(torch.cuda, "stream", using)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("stream", handle))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(_lib, "_dense", lambda t, *a: None if t is None else t.data_ptr())
    monkeypatch.setattr(_lib, "_rows", lambda t, *a: (t.data_ptr(), t.stride(0)))
    monkeypatch.setattr(_lib, "_heads", lambda t, *a: (t.data_ptr(), t.stride(0)))
    monkeypatch.setattr(_lib, "_fn", lambda name: lambda *args: 0)
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    return seen


def calls(stream):
    f = torch.zeros(32, 64, dtype=torch.bfloat16)
    gate = torch.zeros(32, 4, dtype=torch.bfloat16)[:, 1]
    kv = _lib.kv_struct(4, 2, 64, 16, 4)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(3, dtype=torch.int32)

    class Space:
        ptr, nbytes = 0, 0

    return {
        "norm_in": lambda: _lib.moe_norm_in(f, stream=stream),
        "norm_out": lambda: _lib.moe_norm_out(f, f, gate=gate, next_norm=True, stream=stream),
        "append": lambda: _lib.moe_kv_append(kv, q, k, k, i32, i32, None, cache, cache, stream=stream),
        "attention": lambda: _lib.moe_prefix_attention(kv, q, cache, cache, None, 0, None, i32, Space(),
                                                       want_lse=True, stream=stream),
    }


@pytest.mark.parametrize("name,allocations,copies", [("norm_in", 1, 0), ("norm_out", 2, 1), ("append", 1, 0),
                                                     ("attention", 2, 0)])
def test_memory_of_a_call_belongs_to_its_stream(trace, name, allocations, copies):
    run = calls(1234)[name]
    del trace[:]
    run()
    want = [("empty", ("stream", 1234))] * allocations + [("copy", ("stream", 1234))] * copies
    assert sorted(trace) == sorted(want + [("kept for", "current")] * allocations)
    run = calls(None)[name]
    del trace[:]
    run()
    assert sorted(trace) == sorted([("empty", "current")] * allocations + [("copy", "current")] * copies)
