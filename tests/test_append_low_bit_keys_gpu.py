"""Several rows written at once and the low-bit key copy that ffd_decode selects by:
the blocks that changed are quantised again from the first of them on."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import TreeStep, ffd

pytestmark = pytest.mark.gpu
T, CAP = 64, 512


def _quantised(s, k, lengths, block_begin=0, bufs=None):
    bufs = bufs or ffd.DecodeBuffers(s)
    ffd.quantize_keys(s, k, lengths, block_begin, bufs.k_packed, bufs.k_scales)
    return bufs


def _blocks(s, bufs, lengths):
    """Codes and scales of each sequence's blocks, whole ones and the last."""
    packed = bufs.k_packed.view(s.batch, s.num_kv_heads, CAP, 64)
    scales = bufs.k_scales.view(s.batch, s.num_kv_heads, CAP // T, 128).view(torch.int16)
    return [(packed[b, :, :-(-n // T) * T], scales[b, :, :-(-n // T)]) for b, n in enumerate(lengths.tolist())]


def _same(s, a, b, lengths):
    return all(torch.equal(x, y) for p, q in zip(_blocks(s, a, lengths), _blocks(s, b, lengths)) for x, y in zip(p, q))


@pytest.mark.parametrize("start,new", [([100, 190], 50), ([64, 65], 64), ([1, 300], 130), ([63, 127], 1)])
def test_from_the_first_changed_block_on(start, new):
    s = su.shape(2, 2, 2, CAP)
    cache = ffd.KVCache.empty(s)
    lengths = torch.tensor(start, dtype=torch.int32).cuda()
    k0, v0 = su.randn(1, 2, max(start), 2, 128).cuda(), su.randn(2, 2, max(start), 2, 128).cuda()
    ffd.append_tokens(s, cache, k0, v0, lengths, new_lengths=lengths)
    bufs, last = _quantised(s, cache.k, lengths), _quantised(s, cache.k, lengths)
    first = min(start) // T
    lengths += new
    k, v = su.randn(3, 2, new, 2, 128).cuda(), su.randn(4, 2, new, 2, 128).cuda()
    ffd.append_tokens(s, cache, k, v, lengths)
    whole = _quantised(s, cache.k, lengths)
    assert _same(s, _quantised(s, cache.k, lengths, first, bufs), whole, lengths)
    # only the last block: right for one token, stale for several that cross a block
    crosses = any((n + new - 1) // T > n // T for n in start)
    assert _same(s, _quantised(s, cache.k, lengths, ffd.FFD_LAST_BLOCK, last), whole, lengths) == (not crosses)


def test_after_accepted_drafts():
    """A dense-selecting decode (large delta) and a sparse one agree with a cache whose
    keys were quantised from the start."""
    s = su.shape(2, 2, 2, CAP)
    cache = ffd.KVCache.empty(s)
    start = [125, 60]
    lengths = torch.tensor(start, dtype=torch.int32).cuda()
    k0, v0 = su.randn(1, 2, 125, 2, 128).cuda(), su.randn(2, 2, 125, 2, 128).cuda()
    ffd.append_tokens(s, cache, k0, v0, lengths, new_lengths=lengths)
    bufs = _quantised(s, cache.k, lengths)
    step = TreeStep(s, cache, lengths, 9)
    for t, seed, h in ((step.q, 3, 4), (step.k_new, 4, 2), (step.v_new, 5, 2)):
        t.copy_(su.randn(seed, 2, 9, h, 128))
    step.step()
    step.accept(torch.arange(9).repeat(2, 1).cuda(), torch.tensor([9, 7], dtype=torch.int32).cuda())
    assert step.check() == 0 and lengths.tolist() == [134, 67]
    _quantised(s, cache.k, lengths, min(start) // T, bufs)
    whole = _quantised(s, cache.k, lengths)
    q = su.randn(6, 2, 4, 128).cuda()
    for delta in (0.5, 4.0, float("inf")):
        results = []
        for b in (bufs, whole):
            ffd.decode(s, q, cache.k, cache.v, b.k_packed, b.k_scales, lengths, delta, b.out, b.mask, b.workspace)
            results.append((b.out.clone(), b.mask.clone()))
        assert all(torch.equal(x, y) for x, y in zip(*results))
