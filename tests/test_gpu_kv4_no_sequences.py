"""moe_kv4_attention of tokens without a sequence: what the offsets hold is checked
where no sequence reads them, too."""
import math

import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def attend(offset, T=3):
    """num_seqs = 0, q_offsets = [offset]; (rows in front, rows of the tokens, rows behind) of o and lse."""
    kv = moe.kv_struct(8, 2, 64, 16, 0)
    ws = moe.Workspace(moe.moe_kv4_attention_workspace_size(kv, T, 0, 1))
    none = torch.empty(0, 2, moe.moe_kv4_page_bytes(kv), dtype=torch.uint8, device="cuda")
    q = torch.ones(T, 8, 64, dtype=torch.bfloat16, device="cuda")
    room = 64
    o = torch.full((T + 2 * room, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 2 * room, 8), 7.0, device="cuda")
    offsets = torch.tensor([offset], dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    moe.moe_kv4_attention(kv, q, none, none, None, lens, ws, q_offsets=offsets, out=o[room:room + T],
                          lse=lse[room:room + T])
    status = moe.moe_get_device_status(ws)
    return status, [(t[:room], t[room:room + T], t[room + T:]) for t in (o, lse)]


@pytest.mark.parametrize("offset", [0, 1, 3])
def test_tokens_see_nothing(offset):
    status, (o, lse) = attend(offset)
    assert status == 0
    assert (o[1] == 0).all() and (lse[1] == -math.inf).all()
    for t in (*o[::2], *lse[::2]):
        assert (t == 7.0).all()


@pytest.mark.parametrize("offset", [4, 40, -1, -40])
def test_offsets_outside_are_reported(offset):
    """Offsets that leave [0, T], by no more than the room around the outputs."""
    status, (o, lse) = attend(offset)
    assert status == 1
    for t in (*o[::2], *lse[::2]):
        assert (t == 7.0).all()
