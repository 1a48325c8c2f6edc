"""Rotary positions, the cache write of several tokens and the 8-bit cache's
read-back, against their 64-bit forms."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _close(got, want, bound, tag=""):
    err = (got.double() - want).abs()
    worst = (err - bound).max()
    assert worst <= 0, f"{tag}: error {err.max():.3e}, {int((err > bound).sum())} past their bound"


def _positions(seed, *shape, low=-5, high=1 << 20):
    return torch.randint(low, high, shape, generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rotary", [2, 6, 32, 80, 96, 120, 128])
def test_rotate_layouts(layout, rotary):
    o = su.options(rotary, layout)
    q, k, pos = su.randn(1, 37, 8, 128), su.randn(2, 37, 3, 128), _positions(3, 37)
    qo, ko = torch.full_like(q, float("nan")).cuda(), torch.full_like(k, float("nan")).cuda()
    ffd.rotate(ffd.Rope(**o), pos.cuda(), q.cuda(), qo, k.cuda(), ko)
    for x, y in ((q, qo), (k, ko)):
        want = su.rotate64(x, pos, o)
        _close(y.cpu(), want, su.rotate_bound(x, want, o))
        assert torch.equal(y.cpu()[..., rotary:], x[..., rotary:])


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "by_parts"])
@pytest.mark.parametrize("tokens", [1, 2047, 2049])
def test_rotate_scalings_and_sizes(scaling, tokens):
    o = su.options(64, "half", scaling)
    q, pos = su.randn(4, tokens, 5, 128), _positions(5, tokens, low=0)
    pos[0] = 2 ** 31 - 1
    out = torch.empty_like(q).cuda()
    ffd.rotate(ffd.Rope(**o), pos.cuda(), q.cuda(), out)
    want = su.rotate64(q, pos, o)
    _close(out.cpu(), want, su.rotate_bound(q, want, o))


@pytest.mark.parametrize("layout,rotary", [("half", 128), ("interleaved", 64), ("half", 20)])
def test_rotate_in_place_and_back(layout, rotary):
    o = su.options(rotary, layout)
    q, pos = su.randn(6, 300, 4, 128), _positions(7, 300)
    rope, dq, dpos = ffd.Rope(**o), q.cuda(), pos.cuda()
    there = torch.empty_like(dq)
    ffd.rotate(rope, dpos, dq, there)
    ffd.rotate(rope, dpos, dq, dq)
    assert torch.equal(there, dq)
    ffd.rotate(rope, dpos, dq, dq, inverse=True)
    want = su.rotate64(there.cpu(), pos, o, inverse=True)
    _close(dq.cpu(), want, su.rotate_bound(there.cpu(), want, o))
    # two roundings of magnitudes up to the pair's
    assert (dq.cpu().double() - q.double()).abs().max() <= float(q.abs().max()) * 2 * 2 * 2.0 ** -8


def test_rotate_inverse_is_the_gradient():
    """<g, J x> = <J^T g, x>, and the directional difference of the forward form."""
    o = su.options(96, "half", "by_parts")
    x, g, pos = su.randn(8, 9, 2, 128), su.randn(9, 9, 2, 128), _positions(10, 9)
    out = torch.empty_like(g).cuda()
    ffd.rotate(ffd.Rope(**o), pos.cuda(), g.cuda(), out, inverse=True)
    want = su.rotate64(g, pos, o, inverse=True)
    _close(out.cpu(), want, su.rotate_bound(g, want, o))
    step = 1e-3
    up = su.rotate64(x.double() + step, pos, o)
    down = su.rotate64(x.double() - step, pos, o)
    difference = ((up - down) / (2 * step) * g.double()).sum()
    gradient = out.cpu().double().sum()
    assert abs(difference - gradient) <= float(su.rotate_bound(g, want, o).sum())


def test_rotate_nothing():
    q = torch.empty((0, 4, 128), dtype=BF16, device="cuda")
    ffd.rotate(ffd.Rope(), torch.empty(0, dtype=torch.int32, device="cuda"), q, q.clone())


def _cache(shape, fmt, seed):
    c = ffd.KVCache.empty(shape, fmt)
    g = torch.Generator().manual_seed(seed)
    for t in (c.k, c.v, c.k_scales, c.v_scales):
        if t is not None:
            t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, dtype=torch.uint8))
    return c


def _bytes(c):
    return [t.view(torch.uint8).cpu().clone() for t in (c.k, c.v, c.k_scales, c.v_scales) if t is not None]


APPENDS = [
    # B, n, G, Hkv, cap, lengths, counts, rotary, layout, positions given
    (1, 1, 1, 1, 64, [1], None, 128, "half", False),
    (3, 5, 4, 2, 192, [5, 100, 192], None, 128, "half", False),
    (3, 5, 4, 2, 192, [4, 100, 192], [4, 0, 5], 64, "interleaved", True),
    (2, 64, 8, 3, 256, [64, 200], [17, 64], 18, "half", True),
    (2, 1100, 2, 2, 1152, [1100, 1152], [1100, 999], 128, "half", False),
    (4, 3, 1, 4, 64, [3, -1, 65, 2], [3, 1, 1, 3], 0, "half", False),   # bad lengths and counts are left out
    (1, 2, 2, 1, 64, [0], [0], 128, "half", False),
]


@pytest.mark.parametrize("fmt", [ffd.FFD_CACHE_BF16, ffd.FFD_CACHE_BYTE])
@pytest.mark.parametrize("case", APPENDS)
def test_append(case, fmt):
    B, n, G, Hkv, cap, lengths, counts, rotary, layout, given = case
    s = su.shape(B, G, Hkv, cap)
    o = su.options(rotary, layout) if rotary else None
    cache = _cache(s, fmt, 11)
    before = _bytes(cache)
    q, k, v = su.randn(12, B, n, G * Hkv, 128), su.randn(13, B, n, Hkv, 128), su.randn(14, B, n, Hkv, 128, scale=3)
    v[0, 0, 0] = 0
    pos = _positions(15, B, n) if given else None
    q_out = torch.full_like(q, 7.0).cuda()
    ffd.append_tokens(s, cache, k.cuda(), v.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(),
                      rope=ffd.Rope(**o) if o else None, positions=None if pos is None else pos.cuda(),
                      new_lengths=None if counts is None else torch.tensor(counts, dtype=torch.int32).cuda(),
                      q=q.cuda(), q_out=q_out)
    after = _bytes(cache)
    touched = torch.zeros((B, Hkv, cap), dtype=torch.bool)
    for b in range(B):
        m = n if counts is None else counts[b]
        if not 0 <= lengths[b] <= cap or not 0 <= m <= min(n, lengths[b]):
            m = 0
        slots = torch.arange(lengths[b] - m, lengths[b])
        assert (q_out[b, m:] == 7.0).all()
        if m == 0:
            continue
        touched[b, :, slots] = True
        p = pos[b, :m] if given else slots

        def rot(x):
            return su.rotate64(x, p, o) if o else x.double()

        bound = (lambda x, w: su.rotate_bound(x, w, o)) if o else (lambda x, w: w.abs() * 0)
        want_q, want_k = rot(q[b, :m]), rot(k[b, :m])
        _close(q_out[b, :m].cpu(), want_q, bound(q[b, :m], want_q))
        got = [t[b, :, slots].transpose(0, 1).cpu() for t in (cache.k, cache.v)]
        if fmt == ffd.FFD_CACHE_BF16:
            _close(got[0], want_k, bound(k[b, :m], want_k))
            assert torch.equal(got[1], v[b, :m])
            continue
        scales = [t[b, :, slots].transpose(0, 1).cpu() for t in (cache.k_scales, cache.v_scales)]
        codes, want_s = su.quantise64(v[b, :m].float())
        assert torch.equal(scales[1], want_s)
        assert torch.equal(got[1].view(torch.uint8), codes.view(torch.uint8))
        # k: the scale is the largest magnitude / 448 to one rounding to bf16 (fp32
        # rotation before it), a value half an e4m3 step off, or half the smallest
        # step (2^-10 of the scale)
        top = want_k.abs().amax(-1) / 448
        assert ((scales[0].double() - top).abs() <= top * (2.0 ** -8 + 2.0 ** -20)).all()
        held = got[0].double() * scales[0].double()[..., None]
        room = want_k.abs() * 2.0 ** -4 + scales[0].double()[..., None] * 2.0 ** -10
        slack = bound(k[b, :m], want_k) - want_k.abs() * 2.0 ** -8 if o else 0
        _close(held, want_k, room + slack)
    for x, y in zip(before, after):
        keep = ~touched
        assert torch.equal(x.view(B, Hkv, cap, -1)[keep], y.view(B, Hkv, cap, -1)[keep])


def test_append_matches_decode_append_slots():
    """One token a sequence without rotation: the rows decode_append writes."""
    s = su.shape(2, 4, 2, 128)
    cache = _cache(s, ffd.FFD_CACHE_BF16, 1)
    k, v = su.randn(1, 2, 1, 2, 128).cuda(), su.randn(2, 2, 1, 2, 128).cuda()
    lengths = torch.tensor([70, 128], dtype=torch.int32).cuda()
    ffd.append_tokens(s, cache, k, v, lengths)
    k2, v2 = torch.zeros_like(cache.k), torch.zeros_like(cache.v)
    b = ffd.DecodeBuffers(s)
    ffd.quantize_keys(s, k2, lengths, 0, b.k_packed, b.k_scales)
    q = su.randn(3, 2, 8, 128).cuda()
    ffd.decode_append(s, q, k[:, 0].contiguous(), v[:, 0].contiguous(), k2, v2, b.k_packed, b.k_scales, lengths,
                      1.0, b.out, b.mask, b.workspace)
    for i, slot in enumerate((69, 127)):
        assert torch.equal(cache.k[i, :, slot], k2[i, :, slot]) and torch.equal(cache.v[i, :, slot], v2[i, :, slot])


def test_append_query_in_place():
    s = su.shape(2, 4, 2, 128)
    o = su.options(128, "interleaved")
    q, k = su.randn(1, 2, 3, 8, 128).cuda(), su.randn(2, 2, 3, 2, 128).cuda()
    lengths = torch.tensor([10, 128], dtype=torch.int32).cuda()
    out = torch.empty_like(q)
    cache = _cache(s, ffd.FFD_CACHE_BYTE, 3)
    ffd.append_tokens(s, cache, k, k.clone(), lengths, rope=ffd.Rope(**o), q=q, q_out=out)
    ffd.append_tokens(s, cache, k, k.clone(), lengths, rope=ffd.Rope(**o), q=q, q_out=q)
    assert torch.equal(out, q)


def test_append_odd_rows():
    """Zeros, the smallest magnitudes, infinities and NaN in a row."""
    s = su.shape(1, 1, 1, 64)
    x = su.randn(1, 1, 6, 1, 128)
    x[0, 0] = 0
    x[0, 1] = 2.0 ** -133
    x[0, 2] *= 2.0 ** -124
    x[0, 3, 0, 5] = float("inf")
    x[0, 4, 0, 77] = float("nan")
    x[0, 5] *= 2.0 ** 120
    cache = _cache(s, ffd.FFD_CACHE_BYTE, 2)
    ffd.append_tokens(s, cache, x.cuda(), x.cuda().clone(), torch.tensor([6], dtype=torch.int32).cuda())
    codes, scales = su.quantise64(x[0, :, 0].float())
    for i in (0, 1, 2, 5):
        for c, sc in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
            assert torch.equal(c[0, 0, i].view(torch.uint8).cpu(), codes[i].view(torch.uint8)), i
            assert torch.equal(sc[0, 0, i].cpu(), scales[i]), i
    out = torch.zeros((1, 1, 6, 128), dtype=BF16, device="cuda")
    ffd.read_cache(s, cache, torch.tensor([6], dtype=torch.int32).cuda(), 0, k_out=out)
    assert out[0, 0, [3, 4]].isnan().all() and out[0, 0, [0, 1, 2, 5]].isfinite().all()


@pytest.mark.parametrize("B,Hkv,cap,lengths,begin,count", [
    (1, 1, 64, [64], 0, 64), (3, 2, 192, [0, 101, 192], 33, 100), (2, 3, 1024, [1000, 7], 5, 900),
    (3, 1, 64, [-1, 65, 64], 0, 64), (1, 2, 128, [128], 127, 1), (1, 1, 64, [64], 64, 0)])
@pytest.mark.parametrize("which", ["both", "k", "v"])
def test_read(B, Hkv, cap, lengths, begin, count, which):
    s = su.shape(B, 2, Hkv, cap)
    codes = [su.randn(i, B, Hkv, cap, 128, dtype=torch.float32, scale=60).clamp(-448, 448).to(torch.float8_e4m3fn)
             for i in (1, 2)]
    scales = [su.randn(i, B, Hkv, cap, scale=0.1) for i in (3, 4)]
    cache = ffd.KVCache(*(t.cuda() for t in (*codes, *scales)))
    outs = [torch.full((B, Hkv, count, 128), 5.0, dtype=BF16).cuda() for _ in range(2)]
    ffd.read_cache(s, cache, torch.tensor(lengths, dtype=torch.int32).cuda(), begin,
                   outs[0] if which != "v" else None, outs[1] if which != "k" else None)
    for i, (c, sc) in enumerate(zip(codes, scales)):
        got = outs[i].cpu()
        want = torch.full_like(got, 5.0)
        if which == "both" or which == "kv"[i]:
            for b in range(B):
                m = max(0, min(lengths[b] - begin, count)) if 0 <= lengths[b] <= cap else 0
                at = slice(begin, begin + m)
                want[b, :, :m] = (c[b, :, at].double() * sc[b, :, at].double()[..., None]).to(BF16)
        assert torch.equal(got, want)


def test_all_codes_read_back():
    s = su.shape(1, 1, 1, 64)
    codes = torch.arange(256, dtype=torch.uint8).view(1, 1, 2, 128).repeat(1, 1, 32, 1).view(torch.float8_e4m3fn)
    scales = (2.0 ** torch.arange(-20, 44, dtype=torch.float32) * 1.40625).to(BF16).view(1, 1, 64)
    out = torch.empty((1, 1, 64, 128), dtype=BF16, device="cuda")
    cache = ffd.KVCache(codes.cuda(), codes.cuda().clone(), scales.cuda(), scales.cuda().clone())
    ffd.read_cache(s, cache, torch.tensor([64], dtype=torch.int32).cuda(), 0, k_out=out)
    want = (codes.double() * scales.double()[..., None]).to(BF16)
    assert torch.equal(out.cpu().isnan(), want.isnan())
    assert torch.equal(out.cpu().nan_to_num(), want.nan_to_num())


def test_other_stream_and_graph():
    """On a side stream, then captured and replayed with other contents."""
    s = su.shape(2, 4, 2, 128)
    o = su.options(128, "half")
    rope = ffd.Rope(**o)
    q, k, v = (su.randn(i, 2, 4, h, 128).cuda() for i, h in ((1, 8), (2, 2), (3, 2)))
    lengths = torch.tensor([50, 128], dtype=torch.int32).cuda()
    cache, out = _cache(s, ffd.FFD_CACHE_BYTE, 5), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ffd.append_tokens(s, cache, k, v, lengths, rope=rope, q=q, q_out=out)
    side.synchronize()
    want = out.clone(), _bytes(cache)
    graph = torch.cuda.CUDAGraph()
    back = torch.empty((2, 2, 128, 128), dtype=BF16, device="cuda")
    with torch.cuda.graph(graph):
        ffd.append_tokens(s, cache, k, v, lengths, rope=rope, q=q, q_out=out)
        ffd.read_cache(s, cache, lengths, 0, k_out=back)
    q2, l2 = su.randn(9, 2, 4, 8, 128).cuda(), torch.tensor([60, 90], dtype=torch.int32).cuda()
    q.copy_(q2)
    lengths.copy_(l2)
    graph.replay()
    got = out.clone()
    eager = torch.empty_like(out)
    other = _cache(s, ffd.FFD_CACHE_BYTE, 5)
    ffd.append_tokens(s, other, k, v, l2, rope=rope, q=q2, q_out=eager)
    assert torch.equal(got, eager) and not torch.equal(got, want[0])
