"""One workspace, sized for the largest batch, through every smaller one."""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_prefix_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def test_a_batch_that_drains():
    hq, hkv, D, page = 32, 4, 128, 16
    kv = moe.kv_struct(hq, hkv, D, page, 1, torch.bfloat16)
    ws = moe.Workspace(moe.moe_prefix_attention_workspace_size(kv, 90, 9, 10, 700))
    for qs, prefix in [([10] * 9, 700), ([1] * 9, 700), ([1] * 5, 700), ([1] * 4, 700), ([1], 700), ([2], 40),
                       ([9, 1], 0), ([8, 1], 0), ([4] * 2, 0), ([1], 0), ([10] * 9, 700)]:
        c = Case(qs, [17 * (b + 1) for b in range(len(qs))], prefix, hq=hq, hkv=hkv, D=D, page=page)
        need = moe.moe_prefix_attention_workspace_size(c.kv, c.T, len(qs), c.max_q, prefix)
        assert need <= ws.nbytes
        c.check(ws=ws)
