"""Python entry points of the multi-token operators: tensors of a wrong number of
dimensions, type or size are refused by name, before anything is launched."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import TreeStep, ffd

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
B, N, HQ, HKV, CAP = 2, 3, 4, 2, 64


def _t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _parts(fmt=ffd.FFD_CACHE_BF16):
    s = su.shape(B, HQ // HKV, HKV, CAP)
    return s, ffd.KVCache.empty(s, fmt), torch.full((B,), N, dtype=I32, device="cuda")


@pytest.mark.parametrize("shape", [(), (4,), (B, N), (B, N, HQ), (B, N, HQ, 64), (B, N, HQ, 128, 1)])
def test_tree_queries(shape):
    s, cache, lengths = _parts()
    q = _t(*shape)
    with pytest.raises(ValueError, match="q"):
        ffd.decode_tree(s, cache, q, lengths, torch.zeros_like(q), ffd.tree_workspace(s, N))


@pytest.mark.parametrize("shape", [(), (4,), (B, N), (B, N, HKV), (B, N, HKV, 64), (B, N, HKV, 128, 1)])
def test_new_rows(shape):
    s, cache, lengths = _parts()
    with pytest.raises(ValueError, match="k_new"):
        ffd.append_tokens(s, cache, _t(*shape), _t(*shape), lengths)


@pytest.mark.parametrize("shape", [(), (4,), (B, HKV), (B, HKV, 5), (B, HKV, 5, 64), (B, HKV, 5, 128, 1)])
def test_read_outputs(shape):
    s, cache, lengths = _parts(ffd.FFD_CACHE_BYTE)
    with pytest.raises(ValueError, match="k_out"):
        ffd.read_cache(s, cache, lengths, 0, k_out=_t(*shape))
    with pytest.raises(ValueError, match="v_out"):
        ffd.read_cache(s, cache, lengths, 0, v_out=_t(*shape))


@pytest.mark.parametrize("lengths", [torch.zeros(1, dtype=I32), torch.zeros(B, dtype=torch.int64),
                                     torch.zeros((B, 1), dtype=I32)])
def test_step_lengths(lengths):
    s, cache, _ = _parts()
    with pytest.raises(ValueError, match="lengths"):
        TreeStep(s, cache, lengths.cuda(), N)
    with pytest.raises(ValueError):
        TreeStep(s, cache, lengths, N)


def test_step_cache_of_another_shape():
    s, _, lengths = _parts()
    other = ffd.KVCache.empty(su.shape(B, 2, HKV, 2 * CAP))
    with pytest.raises(ValueError, match="cache"):
        TreeStep(s, other, lengths, N)
