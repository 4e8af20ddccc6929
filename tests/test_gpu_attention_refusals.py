"""moe_prefix_attention without a page table: the lengths and offsets that it is
given are still looked at."""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_prefix_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


@pytest.mark.parametrize("prefix,hq", [(0, 8), (50, 8), (300, 64)])   # nothing to attend, few rows, many
def test_bad_lengths_and_offsets_without_a_table(prefix, hq):
    def run(name=None, index=0, value=0, **kw):
        c = Case([1, 2], [0, 0], prefix, hq=hq, hkv=2)
        c.table = None
        if name:
            getattr(c, name)[index] = value
        c.run(**kw)
        return moe.moe_get_device_status(c.ws)

    assert run() == 0
    assert run("lens", 0, 1) == 1
    assert run("lens", 1, -3) == 1
    assert run("off", 1, -7) == 1
    assert run("off", 1, 3000) == 1
    assert run("off", 2, 3000) == 1
    assert run("off", 2, 0) == 1
    assert run(max_q=1) == 1
