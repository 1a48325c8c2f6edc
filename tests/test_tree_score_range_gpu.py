"""Attention of drafted tokens with scores from ordinary to far beyond what fp32
tells apart: right up to the documented size, and then right or NaN, never a
plausible number that is wrong."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd
from test_tree_gpu import FORMATS, Case

pytestmark = pytest.mark.gpu
ROWS = [(3, 1), (4, 4), (6, 4), (12, 4), (14, 8), (30, 8)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G", ROWS)
@pytest.mark.parametrize("power", [0, 8, 14, 19, 21, 23, 25, 28, 31, 34, 40, 60])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_scores(fmt, n, G, power, sign):
    """Queries 2^power times as large as ordinary ones (scores up to about 4 x
    2^power), over several tiles and a CTA each; sign -1: every score of a row far
    below zero.  Where the highest score leads by more than 64 and its error, its
    weight is all there is: the row is that token's value, of which a weight with 8
    significant bits and the rounding to bf16 take up to 2^-8 each, together at most
    2^-7 + 2^-16.  A row is NaN only if a score passes 2^18 (8-bit
    cache) or 2^29."""
    c = Case(fmt, 1, n, G, 1, 640, [601], kind="chain", seed=120 + n)
    if sign < 0:
        c.q, k = c.q.abs(), -c.wide()[0].nan_to_num(0.0).abs()
        if fmt == ffd.FFD_CACHE_BF16:
            c.k = k.to(torch.bfloat16)
        else:
            c.k, c.ks = su.quantise64(k.float())
    c.q *= 2.0 ** power
    got = c.device().run()[0].double()
    k, v = (x[0, 0, :601] for x in c.wide())
    limit = 2.0 ** (29 if fmt == ffd.FFD_CACHE_BF16 else 18)
    sharp = 0
    for i in range(n):
        L = 601 - n + i + 1
        for h in range(G):
            q = c.q[0, i, h].double()
            s = k[:L] @ q / 128 ** 0.5
            if s.abs().max() > limit and got[i, h].isnan().all():
                continue
            assert got[i, h].isfinite().all(), (i, h)
            ds = float((k[:L].abs() @ q.abs()).max()) / 128 ** 0.5 * 2.0 ** -20 + 2.0 ** -18
            top = s.topk(2)
            if top.values[0] - top.values[1] > 64 + 2 * ds:
                want = v[top.indices[0]]
                assert ((got[i, h] - want).abs() <= want.abs() * (2.0 ** -7 + 2.0 ** -15)).all(), (i, h, float(s.abs().max()))
                sharp += 1
    assert ffd.check_device_status(c.ws) == 0
    if power == 14:
        assert sharp > 0
