"""TreeStep.accept: what it keeps, and what it leaves out and reports."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import TreeStep, ffd

pytestmark = pytest.mark.gpu
FORMATS = [ffd.FFD_CACHE_BF16, ffd.FFD_CACHE_BYTE]
B, N, CAP = 4, 5, 128


def _step(fmt, lengths):
    s = su.shape(B, 2, 2, CAP)
    cache = ffd.KVCache.empty(s, fmt)
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        if t is not None:
            t.view(torch.uint8).fill_(0x22)
    step = TreeStep(s, cache, torch.tensor(lengths, dtype=torch.int32).cuda(), N)
    step.q.copy_(su.randn(1, B, N, 4, 128))
    step.k_new.copy_(su.randn(2, B, N, 2, 128))
    step.v_new.copy_(su.randn(3, B, N, 2, 128))
    return step


def _accept(step, nodes, counts):
    step.accept(torch.tensor(nodes).cuda(), torch.tensor(counts, dtype=torch.int32).cuda())
    return step.lengths.tolist()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("nodes,count", [([0, 1, 2], 4), ([0, 1, 2], -1), ([0, 5, 1], 2), ([0, -1, 1], 2),
                                         ([0, 1, 2], 2 ** 31 - 1), ([0, 1, 2], -2 ** 31)])
def test_a_list_that_cannot_be_kept(fmt, nodes, count):
    """One sequence's list is longer than given, negative, or names a node that is
    not there: its length stays, nothing of it is written, the flag is set; the others
    go on."""
    step = _step(fmt, [10, 20, 30, 40])
    step.step()
    before = step.cache.k.view(torch.uint8).clone()
    assert _accept(step, [[0, 1, 2], nodes, [1, 0, 0], [0, 0, 0]], [3, count, 1, 0]) == [13, 20, 31, 40]
    assert torch.equal(step.cache.k.view(torch.uint8)[1], before[1])
    assert torch.equal(step.cache.k.view(torch.uint8)[3], before[3])
    assert step.check() == ffd.FFD_DEVICE_FLAG_BAD_LENGTH
    assert step.check() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_no_room(fmt):
    step = _step(fmt, [CAP - 2, CAP - 3, 0, CAP])
    step.sizes.copy_(torch.tensor([2, 3, 5, 0], dtype=torch.int32))
    step.step()
    assert step.check() == 0
    lists = [[0, 1, 0], [0, 1, 2], [0, 1, 2], [0, 1, 2]]
    assert _accept(step, lists, [2, 3, 3, 0]) == [CAP, CAP, 3, CAP]
    assert step.check() == 0
    step.sizes.fill_(N)  # (room for one sequence only, whatever the lists say)
    assert _accept(step, lists, [1, 1, 1, 1]) == [CAP, CAP, 4, CAP]
    assert step.check() == ffd.FFD_DEVICE_FLAG_BAD_LENGTH


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_node_beyond_the_sequences_own(fmt):
    """Nodes are those that the step had of that sequence, not those of the buffers."""
    step = _step(fmt, [10, 20, 30, 40])
    step.sizes.copy_(torch.tensor([2, 3, 5, 0], dtype=torch.int32))
    step.step()
    assert _accept(step, [[0, 1, 2]] * 4, [3, 3, 3, 0]) == [10, 23, 33, 40]
    assert step.check() == ffd.FFD_DEVICE_FLAG_BAD_LENGTH


def test_refusals_leave_the_lengths():
    step = _step(FORMATS[0], [10, 20, 30, 40])
    counts = torch.ones(B, dtype=torch.int32).cuda()
    for nodes, c in [(torch.zeros(B, 2).cuda(), counts), (torch.zeros(B - 1, 2, dtype=torch.int64).cuda(), counts),
                     (torch.zeros(B, 2, dtype=torch.int64), counts), (torch.zeros(B, dtype=torch.int64).cuda(), counts),
                     (torch.zeros(B, 2, dtype=torch.int64).cuda(), counts.long()),
                     (torch.zeros(B, 2, dtype=torch.int64).cuda(), counts[:1]),
                     (torch.zeros(B, 2, dtype=torch.int64).cuda(), counts.cpu())]:
        with pytest.raises(ValueError):
            step.accept(nodes, c)
    with pytest.raises((ValueError, ffd.FFDError)):
        step.accept(torch.zeros(B, CAP + 1, dtype=torch.int64).cuda(), counts)
    assert step.lengths.tolist() == [10, 20, 30, 40]
    step.accept(torch.zeros(B, 0, dtype=torch.int64).cuda(), torch.zeros_like(counts))
    assert step.lengths.tolist() == [10, 20, 30, 40] and step.check() == 0
