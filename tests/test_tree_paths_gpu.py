"""Attention of drafted tokens where a CTA's running softmax reference moves, and
where a CTA goes through several units: paths that random scores and few units do
not reach."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd
from test_tree_gpu import FORMATS, Case

pytestmark = pytest.mark.gpu
TILE = 128
# (nodes, heads of a group): 1 to 504 query rows a kv-head, each form of the kernels
ROWS = [(1, 4), (2, 8), (3, 8), (8, 8), (16, 8), (32, 8), (63, 8)]


def _want(c, b):
    """Sequence b of a Case in 64 bits on the GPU, [Hkv, size, G, D], and a bound
    on its error: weights with 8 significant bits (half a step is up to 2^-8 of each),
    the output in bf16 (likewise); a score is 128 fp32 products and sums, each off by at most
    2^-23 of the magnitudes' sum (2^-20 with the ones of the weights), and moves its
    weight by as much; over the 8-bit cache a weight times its V scale is at most
    half of 2^-16 of the row's largest off, and meets codes of up to 448."""
    n, L, m = c.n, c.lengths[b], c.sizes[b]
    k, v = (x[b, :, :L].cuda() for x in c.wide())
    Hkv = k.shape[0]
    G = c.q.shape[2] // Hkv
    q = c.q[b, :m].double().cuda().view(m, Hkv, G, 128).permute(1, 0, 2, 3).reshape(Hkv, m * G, 128)
    words = c.words[b] if c.words is not None else su.chain_words(n)
    seen = torch.ones((m, L), dtype=torch.bool)
    for i in range(m):
        for j in range(m):
            seen[i, L - m + j] = bool(words[i] >> j & 1)
    seen = seen.cuda()[None, :, None, :].expand(Hkv, m, G, L).reshape(Hkv, m * G, L)
    s = (q @ k.transpose(1, 2) / 128 ** 0.5).masked_fill(~seen, -float("inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - top.masked_fill(top == -float("inf"), 0.0))
    total = p.sum(-1, keepdim=True).clamp(min=1e-300)
    y, mag = p @ v / total, p @ v.abs() / total
    ds = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) / 128 ** 0.5 * 2.0 ** -20 + 2.0 ** -18
    tol = y.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + 2 * ds)
    if c.vs is not None:
        w = p * c.vs[b, :, :L].double().cuda()[:, None, :]
        tol = tol + w.amax(-1, keepdim=True) / total * seen.sum(-1, keepdim=True) * 2.0 ** -17 * 448
    return y.view(Hkv, m, G, 128), tol.view(Hkv, m, G, 128)


def _check(c, skip=lambda b: False):
    got = c.device().run()
    for b, m in enumerate(c.sizes):
        assert (got[b, m:] == 9.0).all(), "rows past the tree are left as they were"
        if m == 0 or skip(b):
            continue
        want, tol = _want(c, b)
        Hkv, _, G, _ = want.shape
        mine = got[b, :m].cuda().double().view(m, Hkv, G, 128).permute(1, 0, 2, 3)
        err = (mine - want).abs()
        assert torch.isfinite(mine).all(), f"sequence {b}: not finite"
        assert (err <= tol).all(), f"sequence {b}: {float((err / tol.clamp(min=1e-30)).max()):.2f} of its bound"
    assert ffd.check_device_status(c.ws) == 0
    return got


def _fill_past(c):
    for b, L in enumerate(c.lengths):
        for t in (c.k, c.v, c.ks, c.vs):
            if t is not None and t.dtype == torch.float8_e4m3fn:
                t[b, :, L:].view(torch.uint8).fill_(0x7F)
            elif t is not None:
                t[b, :, L:] = float("nan")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G", ROWS)
@pytest.mark.parametrize("form", ["rising", "falling", "both"])
def test_the_reference_moves(fmt, n, G, form):
    """One key in each tile whose score is 6.5 (2^9.4 in weight) above or below the
    one of the tile before, for two rows of three, so that a CTA's reference moves
    several times in its 8 or 9 tiles, and earlier tokens still count after it."""
    B, Hkv, tiles = 2, (4 if n * G > 256 else 8), 74
    lengths = [tiles * TILE, tiles * TILE - 77]
    c = Case(fmt, B, n, G, Hkv, tiles * TILE, lengths, seed=70 + n)
    gen = torch.Generator().manual_seed(n)
    u = 2.0 * (torch.randint(0, 2, (128,), generator=gen).double() * 2 - 1)  # |u|^2 = 512
    row = torch.arange(n * G * Hkv).view(n, G * Hkv)
    c.q += ((row % 3 != 0)[None, :, :, None] * u).to(c.q.dtype)
    k = c.wide()[0].nan_to_num(0.0)
    for b, L in enumerate(lengths):
        for t in range((L + TILE - 1) // TILE):
            step = {"rising": t % 9, "falling": 8 - t % 9, "both": abs(t % 9 - 4) * 2}[form]
            at = min(t * TILE + int(torch.randint(0, TILE, (1,), generator=gen)), L - n - 1)
            k[b, :, at] = u * (5 + 6.5 * step) * 128 ** 0.5 / 512
    if fmt == ffd.FFD_CACHE_BF16:
        c.k = k.to(torch.bfloat16)
    else:
        c.k, c.ks = su.quantise64(k.float())
    _fill_past(c)
    _check(c)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G", [(5, 2), (20, 1), (40, 1), (40, 2), (40, 8)])
def test_tiles_of_which_a_row_sees_nothing(fmt, n, G):
    """The second of a unit's two tiles holds only drafted tokens, of which the
    first nodes of a chain see none; 160 units, so that most CTAs have both."""
    first = 128 - n // 5
    c = Case(fmt, 1, n, G, 160, 192, [first + n], kind="chain", seed=80 + n)
    _check(c)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G", [(6, 2), (3, 8), (6, 8), (13, 8), (32, 8), (63, 8)])
def test_many_ragged_sequences(fmt, n, G):
    """More sequences than are cut into equal pieces: CTAs end one unit and
    begin others, whole ones among them."""
    B = 40
    lengths = [(131 * i + 7 * n) % 700 + n for i in range(B)]
    sizes = [n - i % 3 if n > 3 else n for i in range(B)]
    sizes[7] = sizes[8] = 0
    lengths[9], sizes[9] = 1, 1
    _check(Case(fmt, B, n, G, 3, 768, lengths, sizes=sizes, seed=90 + n))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G", [(4, 4), (6, 8), (16, 8), (32, 8), (63, 8)])
def test_more_units_than_ctas(fmt, n, G):
    """192 units of a few tiles, or 384: their parts straddle the CTAs."""
    lengths = [512, 400, 511, 300, 129, 385, 640, 64]
    _check(Case(fmt, 8, n, G, 24, 640, lengths, seed=100 + n))


@pytest.mark.parametrize("n,G", [(6, 2), (6, 8), (13, 8), (32, 8), (63, 8)])
@pytest.mark.parametrize("fmt,what", [(FORMATS[0], "value"), (FORMATS[1], "value"), (FORMATS[1], "scale")])
def test_a_value_that_is_not_finite_stays_in_its_unit(fmt, n, G, what):
    """V of one drafted token of one head of some sequences is NaN: who sees it is
    NaN there; every other row, and the units before and after it in a CTA, are the
    same bit for bit (a row's reference and weights are its own)."""
    B, Hkv, node = 40, 3, n // 2
    lengths = [(131 * i + 5) % 500 + n for i in range(B)]
    c = Case(fmt, B, n, G, Hkv, 768, lengths, kind="chain", seed=110 + n)
    clean = _check(c)
    for b in range(0, B, 4):
        slot = lengths[b] - n + node
        if what == "scale":
            c.vs[b, 1, slot] = float("nan")
        elif fmt == ffd.FFD_CACHE_BYTE:
            c.v[b, 1, slot].view(torch.uint8)[5] = 0x7F
        else:
            c.v[b, 1, slot, 5] = float("nan")
    got = c.device().run()
    for b in range(B):
        same = torch.ones((n, Hkv, G, 128), dtype=torch.bool)
        if b % 4 == 0:
            same[node:, 1, :, slice(None) if what == "scale" else 5] = False
            assert got[b].view(n, Hkv, G, 128)[~same].isnan().all()
        assert torch.equal(got[b].view(n, Hkv, G, 128)[same], clean[b].view(n, Hkv, G, 128)[same])
    assert ffd.check_device_status(c.ws) == 0
