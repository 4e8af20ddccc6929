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


def test_one_workspace_for_attention_and_layer():
    # calls of one stream may share a workspace: neither relies on what the other leaves
    g = torch.Generator(device="cuda").manual_seed(3)

    def w(*s, std):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(torch.bfloat16)

    T, d, E, inter = 2048, 1024, 8, 512
    shape = dict(T=T, d=d, E=E, G=4, topk_group=2, k=2, inter=inter, score=moe.MOE_SCORE_SIGMOID_BIAS)
    x, w_r, bias = w(T, d, std=1.0), w(d, E, std=0.02), torch.randn(E, generator=g, device="cuda")
    w_gu, w_dn = w(E, 2 * inter, d, std=d ** -0.5), w(E, d, inter, std=inter ** -0.5)
    want = moe.moe_layer(shape, x, w_r, bias, w_gu, w_dn, moe.Workspace(moe.moe_workspace_size(shape)))
    c = Case([1] * 40, [30 + b for b in range(40)], 300, hq=16, hkv=2, D=128)
    need = moe.moe_prefix_attention_workspace_size(c.kv, c.T, 40, 1, 300)
    ws = moe.Workspace(max(moe.moe_workspace_size(shape), need))
    for _ in range(3):
        c.check(ws=ws)
        assert torch.equal(moe.moe_layer(shape, x, w_r, bias, w_gu, w_dn, ws), want)
    assert moe.moe_get_device_status(ws) == 0
