"""moe_verify_drafts: every draft outside the vocabulary is reported, wherever it
stands among the drafts and whatever becomes of those before it."""
import pytest
import torch

import dispatch_combine_gb300 as moe
from tests.gpu_common import ensure_lib
from tests.test_gpu_verify_drafts import BF16, FP32, check, probs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _lib():
    ensure_lib()


def batch(counts, V, dtype, seed=1):
    """Drafts that all stand: a uniform number of 0 lets every one with a probability through."""
    T = sum(counts)
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda").to(torch.int32)
    off = torch.tensor([sum(counts[:b]) for b in range(len(counts) + 1)], dtype=torch.int32, device="cuda")
    return probs(T, V, seed, dtype, spread=0.5), tokens, torch.zeros(T, device="cuda"), off, probs(T, V, seed + 1, dtype,
                                                                                             spread=0.5)


@pytest.mark.parametrize("at", [1, 2, 3, 17, 31, 32, 33, 63, 64, 65, 80])
@pytest.mark.parametrize("bad", [-1, 100, 2 ** 31 - 1, -2 ** 31])
def test_one_bad_draft(at, bad):
    target, tokens, u, off, draft = batch([81, 2], 100, FP32)
    acc = check(target, tokens, u, off, draft)
    assert acc.tolist() == [80, 1]
    tokens[at] = bad
    for d in (draft, None):
        acc = check(target, tokens, u, off, d, status=1)
        assert acc.tolist() == [at - 1, 1]


@pytest.mark.parametrize("at", [2, 31, 40, 79])
def test_a_bad_draft_behind_one_that_falls(at):
    target, tokens, u, off, draft = batch([80], 100, FP32)
    target[0, tokens[1]] = 0.0
    tokens[at] = 100
    acc = check(target, tokens, u, off, draft, status=1)
    assert acc.item() == 0


@pytest.mark.parametrize("counts,V", [([4] * 37, 32000), ([3, 1, 2] * 100, 9001), ([2] * 700, 64)])
def test_one_bad_draft_among_many_sequences(counts, V):
    target, tokens, u, off, draft = batch(counts, V, BF16)
    check(target, tokens, u, off, draft)
    last = sum(counts) - 1              # the last draft of the last sequence
    tokens[last] = V
    acc = check(target, tokens, u, off, draft, status=1)
    assert acc[-1].item() == counts[-1] - 2


def test_what_is_no_draft_is_not_looked_at():
    """The first token of a sequence has been decided: it is nothing to the verification."""
    target, tokens, u, off, draft = batch([3, 1, 4], 100, FP32)
    tokens[0], tokens[3], tokens[4] = -1, 100, 2 ** 31 - 1
    check(target, tokens, u, off, draft)
