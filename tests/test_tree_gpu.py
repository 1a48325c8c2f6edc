"""Attention of drafted tokens over the cache, against its 64-bit form."""
import random

import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
FORMATS = [ffd.FFD_CACHE_BF16, ffd.FFD_CACHE_BYTE]


def _words(kind, n, sizes, seed):
    """Per sequence, node words: chains, random trees, or any sets at all."""
    r = random.Random(seed)
    out = []
    for m in sizes:
        if kind == "chain":
            w = su.chain_words(m)
        elif kind == "tree":
            w = []
            for i in range(m):
                parent = r.randint(-1, i - 1)
                w.append((w[parent] if parent >= 0 else 0) | 1 << i)
        elif kind == "none":
            w = [0] * m
        else:
            w = [r.getrandbits(64) for _ in range(m)]  # bits of nodes that are not there too
        out.append(w + [r.getrandbits(64) for _ in range(n - len(w))])
    return out


class Case:
    def __init__(self, fmt, B, n, G, Hkv, cap, lengths, sizes=None, kind="tree", seed=0, q_scale=1.0,
                 spread=0.0, fill=float("nan")):
        self.shape = su.shape(B, G, Hkv, cap)
        self.fmt, self.n, self.lengths = fmt, n, lengths
        self.sizes = [n] * B if sizes is None else sizes
        self.given = sizes is not None
        self.q = su.randn(seed + 1, B, n, G * Hkv, 128, scale=q_scale)
        k, v = su.randn(seed + 2, B, Hkv, cap, 128), su.randn(seed + 3, B, Hkv, cap, 128)
        if spread:
            v = (v.double() * torch.exp2(su.randn(seed + 4, B, Hkv, cap, 1, dtype=torch.float64) * spread)).to(BF16)
        self.ks = self.vs = None
        if fmt == ffd.FFD_CACHE_BYTE:
            (k, self.ks), (v, self.vs) = su.quantise64(k.float()), su.quantise64(v.float())
        for b, L in enumerate(lengths):  # what lies past a sequence must not matter
            if 0 <= L < cap:
                for t in (k, v, self.ks, self.vs):
                    if t is not None:
                        if t.dtype == torch.float8_e4m3fn:
                            t[b, :, L:].view(torch.uint8).fill_(0x7F)
                        else:
                            t[b, :, L:] = fill
        self.k, self.v = k, v
        self.words = None if kind == "null" else _words(kind, n, self.sizes, seed)

    def wide(self):
        if self.ks is None:
            return self.k.double(), self.v.double()
        return (self.k.double() * self.ks.double()[..., None], self.v.double() * self.vs.double()[..., None])

    def want(self):
        k, v = self.wide()
        words = self.words or [su.chain_words(m) for m in self.sizes]
        return su.tree64(self.q, k, v, self.lengths, self.sizes, words,
                         weight_scale=None if self.vs is None else self.vs.double())

    def device(self):
        self.cache = ffd.KVCache(*(t.cuda() for t in (self.k, self.v, self.ks, self.vs) if t is not None))
        self.mask = None if self.words is None else torch.tensor([su.signed(w) for w in self.words]).cuda()
        self.d_lengths = torch.tensor(self.lengths, dtype=torch.int32).cuda()
        self.d_sizes = torch.tensor(self.sizes, dtype=torch.int32).cuda() if self.given else None
        self.out = torch.full_like(self.q, 9.0).cuda()
        self.ws = ffd.tree_workspace(self.shape, self.n)
        self.ws[256:] = 0xFF  # NaN: what the workspace holds must not matter
        return self

    def run(self):
        ffd.decode_tree(self.shape, self.cache, self.q.cuda(), self.d_lengths, self.out, self.ws,
                        tree_mask=self.mask, tree_sizes=self.d_sizes)
        return self.out.cpu()

    def check(self):
        self.device()
        got = self.run()
        want, tol = self.want()
        for b, m in enumerate(self.sizes):
            assert (got[b, m:] == 9.0).all(), "rows past the tree are left as they were"
            err = (got[b, :m].double() - want[b, :m]).abs()
            assert torch.isfinite(got[b, :m]).all(), f"sequence {b}: not finite"
            assert (err <= tol[b, :m]).all(), (
                f"sequence {b}: worst {float((err / tol[b, :m].clamp(min=1e-30)).max()):.2f} of its bound, "
                f"error {float(err.max()):.3e}")
        assert ffd.check_device_status(self.ws) == 0
        return got


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("n", [1, 3, 8, 16, 17, 64])
def test_groups_and_nodes(fmt, G, n):
    """Every tile of query rows: replicated, whole, two, and several."""
    Case(fmt, 1, n, G, 1, 320, [300], seed=n * 8 + G).check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("length", [1, 2, 63, 64, 127, 128, 129, 255, 256, 257, 383, 1000, 1024])
def test_lengths(fmt, length):
    n = min(length, 5)
    Case(fmt, 1, n, 2, 2, 1024, [length], seed=length).check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("kind", ["chain", "tree", "any", "none", "null"])
@pytest.mark.parametrize("length", [20, 130, 400])
def test_masks(fmt, kind, length):
    Case(fmt, 2, 20, 4, 2, 448, [length, length - 0], kind=kind, seed=length).check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_that_see_nothing(fmt):
    """The tree is the whole sequence and some nodes see none of it."""
    c = Case(fmt, 2, 7, 4, 2, 64, [7, 7], kind="any", seed=3)
    c.words[0][0] = c.words[0][3] = c.words[1][6] = 0
    c.words[1][2] = 1 << 60  # a node that is not there
    got = c.check()
    assert (got[0, [0, 3]] == 0).all() and (got[1, [2, 6]] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_ragged(fmt):
    Case(fmt, 5, 12, 4, 2, 640, [0, 1, 12, 333, 640], sizes=[0, 1, 5, 12, 0], seed=5).check()


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_sequences(fmt):
    B = 70
    lengths = [(37 * i) % 250 + 3 for i in range(B)]
    Case(fmt, B, 3, 2, 3, 256, lengths, sizes=[i % 4 for i in range(B)], seed=6).check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("q_scale", [0.0, 8.0, 60.0])
def test_flat_and_peaked_scores(fmt, q_scale):
    Case(fmt, 1, 6, 4, 1, 1280, [1277], q_scale=q_scale, seed=7).check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("where", [0, 640, 1270])
def test_one_token_far_above_the_rest(fmt, where):
    """A score 20 above all others, early, in the middle or late, so that the
    running reference falls or rises by that much; the rest still count."""
    c = Case(fmt, 1, 6, 4, 1, 1280, [1277], seed=8)
    k = c.k.double() if c.ks is None else c.k.double() * c.ks.double()[..., None]
    k[0, 0, where] = c.q[0, 0, 0].double() * (20 * 128 ** 0.5 / float((c.q[0, 0, 0].double() ** 2).sum()))
    if c.ks is None:
        c.k = k.to(BF16)
    else:
        c.k, c.ks = su.quantise64(k.float())
        c.k[0, :, 1277:].view(torch.uint8).fill_(0x7F)
    c.check()


@pytest.mark.parametrize("spread", [2.0, 8.0])
def test_value_rows_of_very_different_magnitudes(spread):
    Case(ffd.FFD_CACHE_BYTE, 2, 6, 4, 1, 640, [500, 640], spread=spread, seed=9).check()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_unseen_slots_do_not_matter(fmt, bad):
    """K and V of a drafted token that one node does not see hold NaN or
    infinities; the others see it and are NaN."""
    c = Case(fmt, 1, 6, 2, 1, 320, [300], kind="chain", seed=10)
    slot = 300 - 6 + 4  # node 4: seen by nodes 4 and 5
    want, tol = c.want()
    for t in (c.k, c.v) if fmt == ffd.FFD_CACHE_BF16 else ():
        t[0, 0, slot] = bad
    if fmt == ffd.FFD_CACHE_BYTE:
        for t, s in ((c.k, c.ks), (c.v, c.vs)):
            t[0, 0, slot].view(torch.uint8).fill_(0x7F)
            s[0, 0, slot] = bad
    c.device()
    got = c.run()
    err = (got[0, :4].double() - want[0, :4]).abs()
    assert (err <= tol[0, :4]).all()
    assert got[0, 4:].isnan().any(-1).all()


def test_unseen_infinite_value_alone():
    """Only V of one channel is infinite: who sees the token has an infinity
    in that channel alone."""
    c = Case(ffd.FFD_CACHE_BF16, 1, 6, 2, 1, 320, [300], kind="chain", seed=11)
    want, tol = c.want()
    c.v[0, 0, 300 - 6 + 2, 77] = float("-inf")
    c.device()
    got = c.run()
    rest = [i for i in range(128) if i != 77]
    assert ((got[0].double() - want[0]).abs()[..., rest] <= tol[0][..., rest]).all()
    assert (got[0, 2:, :, 77] == float("-inf")).all()
    assert ((got[0, :2].double() - want[0, :2]).abs() <= tol[0, :2]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_before_the_tree_reaches_everyone(fmt):
    c = Case(fmt, 1, 3, 2, 1, 320, [300], seed=12)
    if fmt == ffd.FFD_CACHE_BF16:
        c.v[0, 0, 10, 5] = float("nan")
    else:
        c.v[0, 0, 10].view(torch.uint8)[5] = 0x7F
    c.device()
    got = c.run()
    assert got[..., 5].isnan().all() and got[..., 6:].isfinite().all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("length,size", [(-1, 1), (321, 1), (100, -1), (100, 5), (2, 3)])
def test_bad_lengths_are_flagged(fmt, length, size):
    c = Case(fmt, 2, 4, 2, 1, 320, [300, 300], sizes=[4, 4], seed=13)
    want, tol = c.want()
    c.lengths, c.sizes = [length, 300], [size, 4]
    c.device()
    got = c.run()
    assert (got[0] == 0).all()
    assert ((got[1].double() - want[1]).abs() <= tol[1]).all()
    assert ffd.check_device_status(c.ws) == ffd.FFD_DEVICE_FLAG_BAD_LENGTH
    assert ffd.check_device_status(c.ws) == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_same_results_every_time_and_in_a_graph(fmt):
    c = Case(fmt, 3, 9, 4, 2, 2048, [2048, 1111, 30], seed=14).device()
    q = c.q.cuda()
    first = c.run()
    for _ in range(3):
        assert torch.equal(c.run().view(torch.int16), first.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ffd.decode_tree(c.shape, c.cache, q, c.d_lengths, c.out, c.ws, tree_mask=c.mask, tree_sizes=c.d_sizes)
    c.out.zero_()
    graph.replay()
    assert torch.equal(c.out.cpu().view(torch.int16), first.view(torch.int16))
    c.d_lengths.copy_(torch.tensor([700, 2000, 9], dtype=torch.int32))
    graph.replay()
    replayed = c.out.cpu()
    c.lengths = [700, 2000, 9]
    assert torch.equal(c.run().view(torch.int16), replayed.view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
def test_two_streams_with_a_workspace_each(fmt):
    cases = [Case(fmt, 2, 9, 4, 2, 1024, [1024, 700], seed=20 + i).device() for i in range(2)]
    want = [c.run() for c in cases]
    qs = [c.q.cuda() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, q in zip(cases, streams, qs):
            with torch.cuda.stream(s):
                ffd.decode_tree(c.shape, c.cache, q, c.d_lengths, c.out, c.ws, tree_mask=c.mask)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert torch.equal(c.out.cpu().view(torch.int16), w.view(torch.int16))


def test_single_token_equals_dense_decode():
    """One node over a bf16 cache: ffd_decode at delta infinity."""
    c = Case(ffd.FFD_CACHE_BF16, 2, 1, 4, 2, 1024, [1024, 515], seed=15, fill=1000.0).device()
    got = c.run()
    bufs = ffd.DecodeBuffers(c.shape)
    ffd.decode(c.shape, c.q[:, 0].cuda().contiguous(), c.cache.k, c.cache.v, None, None, c.d_lengths,
               float("inf"), bufs.out, bufs.mask, bufs.workspace)
    _, tol = c.want()
    assert ((got[:, 0].double() - bufs.out.cpu().double()).abs() <= 2 * tol[:, 0]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_cache(fmt):
    """Many splits: offsets past 32 bits of bytes are not reached, but every
    CTA has a part; checked on the GPU in 64 bits."""
    B, n, G, Hkv, cap = 2, 4, 2, 3, 40000 // 64 * 64
    c = Case(fmt, B, n, G, Hkv, cap, [cap, cap - 77], seed=16).device()
    got = c.run().double()
    k, v = c.wide()
    for b, L in enumerate(c.lengths):
        for h in range(G * Hkv):
            kk, vv = k[b, h // G, :L].cuda(), v[b, h // G, :L].cuda()
            s = c.q[b, :, h].double().cuda() @ kk.T / 128 ** 0.5
            for i in range(n):
                for j in range(n):
                    if not c.words[b][i] >> j & 1:
                        s[i, L - n + j] = -float("inf")
            p = torch.softmax(s, -1)
            want, mag = (p @ vv).cpu(), (p @ vv.abs()).cpu()
            tol = want.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -10)
            assert ((got[b, :, h] - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G", [(1, 4), (7, 8), (16, 4), (13, 8), (64, 4), (63, 8)])
def test_long_cache_row_tiles(fmt, n, G):
    """Every tile of query rows over caches long enough that the copies, not
    the products, set the pace; checked on the GPU in 64 bits."""
    B, Hkv, cap = 2, 4, 65536
    c = Case(fmt, B, n, G, Hkv, 256, [256, 256 - 77], seed=17)
    s = su.shape(B, G, Hkv, cap)
    gen = torch.Generator(device="cuda").manual_seed(n)
    k, v = (torch.randn((B, Hkv, cap, 128), generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    if fmt == ffd.FFD_CACHE_BYTE:
        (kc, ks), (vc, vs) = su.quantise64(k.float()), su.quantise64(v.float())
        cache = ffd.KVCache(kc, vc, ks, vs)
        k, v = kc.double() * ks.double()[..., None], vc.double() * vs.double()[..., None]
    else:
        cache = ffd.KVCache(k, v)
    lengths = [cap, cap - 12345]
    q, out, ws = c.q.cuda(), torch.zeros_like(c.q).cuda(), ffd.tree_workspace(s, n)
    mask = torch.tensor([su.signed(w) for w in c.words]).cuda()
    ln = torch.tensor(lengths, dtype=torch.int32).cuda()
    for _ in range(3):
        ffd.decode_tree(s, cache, q, ln, out, ws, tree_mask=mask)
    assert ffd.check_device_status(ws) == 0
    for b, L in enumerate(lengths):
        seen = torch.ones((n, L), dtype=torch.bool, device="cuda")
        seen[:, L - n:] = (mask[b][:, None] >> torch.arange(n, device="cuda")) & 1 != 0
        for h in range(G * Hkv):
            kk, vv = k[b, h // G, :L].double(), v[b, h // G, :L].double()
            p = torch.softmax((q[b, :, h].double() @ kk.T / 128 ** 0.5).masked_fill(~seen, -float("inf")), -1)
            want, mag = p @ vv, p @ vv.abs()
            tol = want.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -10)
            assert ((out[b, :, h].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("fmt,n", [(f, n) for f in FORMATS for n in (2, 20)])
def test_behind_and_before_other_work_in_a_graph(fmt, n):
    """Inputs that a copy, a fill and a kernel of the same graph leave just
    before the call, results that one takes just after it; twice in a row."""
    c = Case(fmt, 2, n, 4, 2, 1024, [900, 333], seed=30).device()
    want = c.run()
    q, lengths = c.q.cuda(), c.d_lengths.clone()
    late_q, late_lengths, after = torch.zeros_like(q), torch.zeros_like(lengths), [torch.zeros_like(c.out) for _ in range(2)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(2):
            late_lengths.zero_()
            late_q.copy_(q)
            torch.add(late_lengths, lengths, out=late_lengths)
            ffd.decode_tree(c.shape, c.cache, late_q, late_lengths, c.out, c.ws, tree_mask=c.mask)
            after[i].copy_(c.out)
            late_q.zero_()
    for _ in range(3):
        for t in (c.out, *after):
            t.zero_()
        graph.replay()
        for t in after:
            assert torch.equal(t.cpu().view(torch.int16), want.view(torch.int16))
