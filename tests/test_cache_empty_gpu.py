"""KVCache.empty after memory that held NaN: no token of the cache, none of a decode."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [ffd.FFD_CACHE_BF16, ffd.FFD_CACHE_BYTE])
def test_is_finite_throughout(fmt):
    s = su.shape(2, 2, 2, 512)
    n = 2 * 2 * 512 * 128
    old = [torch.full((n,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    old += [torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    old += [torch.full((n // 128,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del old
    cache = ffd.KVCache.empty(s, fmt)
    for t in (cache.k, cache.v, cache.k_scales, cache.v_scales):
        assert t is None or (t.view(torch.uint8) == 0).all()
    assert cache.format == fmt
    if fmt == ffd.FFD_CACHE_BYTE:
        return
    lengths = torch.tensor([134, 67], dtype=torch.int32).cuda()
    rows = su.randn(1, 2, 134, 2, 128).cuda()
    ffd.append_tokens(s, cache, rows, rows, lengths, new_lengths=lengths)
    b = ffd.DecodeBuffers(s)
    ffd.quantize_keys(s, cache.k, lengths, 0, b.k_packed, b.k_scales)
    ffd.decode(s, su.randn(2, 2, 4, 128).cuda(), cache.k, cache.v, b.k_packed, b.k_scales, lengths, 4.0, b.out,
               b.mask, b.workspace)
    assert b.out.isfinite().all()
