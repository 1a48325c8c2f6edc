"""ffd_decode_tree reads what the work before it in the stream leaves, also where
that work lets the next kernel start early."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("capacity", [0, 64])
@pytest.mark.parametrize("stale,fresh", [(70, 0), (0, 70)])
def test_lengths_that_a_rotation_writes(capacity, stale, fresh):
    """The lengths lie in the output of a rotation by angle 0, which copies its
    input's bits: of a long one, whose successor may start while it runs.  With an empty
    cache the call has one kernel only.  No sequence can have 70 tokens."""
    B, n, tokens = 2, 3, 8192
    s = su.shape(B, 2, 2, capacity)
    cache = ffd.KVCache.empty(s)
    q, out = (torch.ones((B, n, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = ffd.tree_workspace(s, n)
    sizes = torch.zeros(B, dtype=torch.int32, device="cuda")
    x = torch.zeros((tokens, 8, 128), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros_like(x)
    at = (x.numel() - 128) // 2
    x.view(-1).view(torch.int32)[at:at + B] = fresh
    lengths = y.view(-1).view(torch.int32)[at:at + B]
    positions = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    rope = ffd.Rope(128)
    for _ in range(20):
        lengths.fill_(stale)
        out.fill_(9.0)
        ffd.rotate(rope, positions, x, y)
        ffd.decode_tree(s, cache, q, lengths, out, ws, tree_sizes=sizes)
        good = fresh == 0
        assert ffd.check_device_status(ws) == (0 if good else ffd.FFD_DEVICE_FLAG_BAD_LENGTH)
        assert (out == (9.0 if good else 0.0)).all()
