"""Over the 8-bit cache each query row has a scale of its own: what other heads
or drafted tokens ask with does not change a row's result."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd
from test_tree_gpu import Case

pytestmark = pytest.mark.gpu
BYTE = ffd.FFD_CACHE_BYTE


def _check_rows(c, rows):
    """The given (node, head) rows against their 64-bit form; the bound of
    serve_util.tree64 counts what a row's own query rounds to."""
    got = c.device().run()
    want, tol = c.want()
    for i, h in rows:
        err = (got[0, i, h].double() - want[0, i, h]).abs()
        assert (err <= tol[0, i, h]).all(), f"row {i}, {h}: {float((err / tol[0, i, h]).max()):.1f} of its bound"
    assert ffd.check_device_status(c.ws) == 0


# 16 query rows a kv-head are the most of the one kernel, 17 the least of the other
@pytest.mark.parametrize("n,G", [(4, 1), (4, 4), (16, 1), (17, 1), (5, 8)])
@pytest.mark.parametrize("power", [-30, -12, 8, 12, 15, 18, 21, 60])
def test_one_row_of_another_magnitude(n, G, power):
    """One row 2^power times as large: the others are as accurate as without it.
    (It may itself be NaN where its scores pass 2^18: test_tree_score_range_gpu.)"""
    c = Case(BYTE, 1, n, G, 1, 640, [601], seed=40 + n)
    c.q[0, 1, G - 1] *= 2.0 ** power
    far = float((c.wide()[0][0, 0, :601] @ c.q[0, 1, G - 1].double()).abs().max()) / 128 ** 0.5 > 2.0 ** 18
    _check_rows(c, [(i, h) for i in range(n) for h in range(G) if (i, h) != (1, G - 1) or not far])


@pytest.mark.parametrize("n,G", [(6, 2), (17, 1)])
@pytest.mark.parametrize("value", [3.0e38, float("inf"), float("nan")])
def test_a_row_that_nobody_sees(n, G, value):
    """The last node of a chain, seen by none but itself, asks with the type's
    largest values, infinities or NaN."""
    c = Case(BYTE, 1, n, G, 1, 640, [601], kind="chain", seed=50)
    c.q[0, n - 1] = value
    _check_rows(c, [(i, h) for i in range(n - 1) for h in range(G)])


@pytest.mark.parametrize("n", [8, 32])
def test_rows_of_falling_magnitude(n):
    """Rows 1, 2^-3, 2^-6, ...: scores from about 30 down to nothing."""
    c = Case(BYTE, 1, n, 2, 1, 640, [601], seed=60, q_scale=8.0)
    c.q *= torch.exp2(-3.0 * torch.arange(n)).view(1, n, 1, 1).to(c.q.dtype)
    _check_rows(c, [(i, h) for i in range(n) for h in range(2)])
