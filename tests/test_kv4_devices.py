"""The calls of the 4-bit cache and of the drafts' verification refuse every tensor, and
a workspace, that is not on the current device, before anything is launched."""
import pytest
import torch

from dispatch_combine_gb300 import _lib


class There(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    device_index = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.device_index


def there(t, index):
    t = t.as_subclass(There)
    t.device_index = index
    return t


class Space:
    """A workspace as the calls see it."""
    ptr, nbytes = 0, 1 << 20

    def __init__(self, index=0):
        self.buf = there(torch.zeros(256, dtype=torch.uint8), index)


def arguments(name):
    """(the call's fixed arguments, its tensors by name)"""
    kv = _lib.kv_struct(4, 2, 64, 16, 4)
    q, k = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cache, i32 = torch.zeros(4, 2, 576, dtype=torch.uint8), torch.zeros(3, dtype=torch.int32)
    pages16, p, u = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(3, 10), torch.zeros(3)
    return {
        "moe_kv4_append": (dict(kv=kv), dict(q=q, k=k, v=k, positions=i32, slots=i32, inv_freq=torch.zeros(32),
                                             k_cache=cache, v_cache=cache, q_out=q)),
        "moe_kv4_read": (dict(kv=kv), dict(slots=i32, k_cache=cache, v_cache=cache, k_out=pages16, v_out=pages16,
                                           dst_slots=i32)),
        "moe_kv4_attention": (dict(kv=kv, max_q=1), dict(q=q, k_cache=cache, v_cache=cache,
                                                         page_table=torch.zeros(3, 4, dtype=torch.int32), kv_lens=i32,
                                                         q_offsets=torch.zeros(4, dtype=torch.int32), out=q,
                                                         lse=torch.zeros(3, 4))),
        "moe_verify_drafts": ({}, dict(target=p, tokens=i32, uniforms=u, offsets=i32, draft=p,
                                       accepted=torch.zeros(2, dtype=torch.int32), out_tokens=i32)),
    }[name]


CALLS = ["moe_kv4_append", "moe_kv4_read", "moe_kv4_attention", "moe_verify_drafts"]


@pytest.fixture
def two_devices(monkeypatch):
    launched = []
    monkeypatch.setattr(_lib, "_one_device", lambda: False)
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    monkeypatch.setattr(_lib, "_fn", lambda name: lambda *args: launched.append(name) or 0)
    monkeypatch.setattr(_lib, "_stream", lambda s: 0)
    return launched


def call(name, elsewhere=None):
    fixed, tensors = arguments(name)
    tensors = {k: there(t, 1 if k == elsewhere else 0) for k, t in tensors.items()}
    getattr(_lib, name)(**fixed, **tensors, ws=Space(1 if elsewhere == "ws" else 0))


@pytest.mark.parametrize("name", CALLS)
def test_tensors_of_the_current_device_pass(two_devices, name):
    call(name)
    assert two_devices == [name]


@pytest.mark.parametrize("name,argument", [(n, a) for n in CALLS for a in [*arguments(n)[1], "ws"]])
def test_a_tensor_of_another_device_is_refused(two_devices, name, argument):
    with pytest.raises(ValueError, match="current device"):
        call(name, argument)
    assert two_devices == []
