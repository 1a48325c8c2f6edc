"""Multi-token operators at their outer sizes: caches whose offsets pass 32 bits, more
sequences than a CTA has threads, more heads than a block's table has rows."""
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd
from test_tree_gpu import FORMATS, Case
from test_tree_paths_gpu import _check

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,G", [(2, 4), (5, 8), (33, 8)])
def test_more_sequences_than_threads(fmt, n, G):
    """900 sequences, most of them without tokens."""
    B = 900
    lengths = [(29 * b) % 150 + n if b % 7 == 3 else 0 for b in range(B)]
    lengths[-1] = 192
    sizes = [n if L else 0 for L in lengths]
    sizes[3] = 0
    _check(Case(fmt, B, n, G, 1, 192, lengths, sizes=sizes, seed=200 + n))


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_long_sequence_behind_many_empty_ones(fmt):
    B = 700
    lengths = [0] * (B - 1) + [1000]
    _check(Case(fmt, B, 4, 8, 1, 1024, lengths, sizes=[0] * (B - 1) + [4], seed=210))


@pytest.mark.parametrize("tokens", [3, 2050])
@pytest.mark.parametrize("layout,rotary", [("half", 128), ("half", 24), ("interleaved", 64)])
def test_more_heads_than_a_table_holds(tokens, layout, rotary):
    o = su.options(rotary, layout)
    q, k = su.randn(1, tokens, 300, 128), su.randn(2, tokens, 11, 128)
    positions = torch.randint(0, 100000, (tokens,), generator=torch.Generator().manual_seed(3), dtype=torch.int32)
    q_out, k_out = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    ffd.rotate(ffd.Rope(**o), positions.cuda(), q.cuda(), q_out, k.cuda(), k_out)
    for x, got in ((q, q_out), (k, k_out)):
        want = su.rotate64(x, positions, o)
        assert ((got.cpu().double() - want).abs() <= su.rotate_bound(x, want, o)).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_offsets_beyond_32_bits(fmt):
    """33.6 million rows: the last sequence's lie beyond 2^32 bytes (8-bit: elements)
    of the cache.  Rows appended there are read back, and a tree attends over them."""
    B, G, Hkv, cap, n, new = 2, 2, 8, 64 * 32800, 6, 100
    s = su.shape(B, G, Hkv, cap)
    assert B * Hkv * cap * 128 > 2 ** 32
    cache = ffd.KVCache.empty(s, fmt)
    lengths = torch.tensor([300, cap - 5], dtype=torch.int32).cuda()
    # the last sequence's last head has a cache of values; the others are zero
    gen = torch.Generator(device="cuda").manual_seed(5)
    L = cap - 5
    for t, scales in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        x = torch.randn((L, 128), generator=gen, device="cuda", dtype=BF16)
        if fmt == ffd.FFD_CACHE_BYTE:
            scales[1, 7, :L] = 2.0 ** -6  # (7 standard deviations are e4m3's 448)
            t[1, 7, :L] = (x.float() * 64).to(t.dtype)
        else:
            t[1, 7, :L] = x
        del x
    q, k, v = su.randn(6, B, new, G * Hkv, 128).cuda(), su.randn(7, B, new, Hkv, 128).cuda(), su.randn(8, B, new, Hkv, 128).cuda()
    q_out = torch.empty_like(q)
    ffd.append_tokens(s, cache, k, v, lengths, q=q, q_out=q_out)
    assert torch.equal(q_out.view(torch.int16), q.view(torch.int16))
    for b, end in enumerate(lengths.tolist()):
        for t, scales, rows in ((cache.k, cache.k_scales, k), (cache.v, cache.v_scales, v)):
            rows = rows[b].transpose(0, 1)
            if fmt == ffd.FFD_CACHE_BF16:
                assert torch.equal(t[b, :, end - new:end].view(torch.int16), rows.contiguous().view(torch.int16))
            else:
                codes, sc = su.quantise64(rows.float().cpu())
                assert torch.equal(t[b, :, end - new:end].cpu().view(torch.uint8), codes.view(torch.uint8))
                assert torch.equal(scales[b, :, end - new:end].cpu().view(torch.int16), sc.view(torch.int16))
    if fmt == ffd.FFD_CACHE_BYTE:
        begin, count = cap - 40, 40
        out = [torch.full((B, Hkv, count, 128), 9.0, dtype=BF16, device="cuda") for _ in range(2)]
        ffd.read_cache(s, cache, lengths, begin, *out)
        for got, t, scales in ((out[0], cache.k, cache.k_scales), (out[1], cache.v, cache.v_scales)):
            want = (t[1, :, begin:L].float() * scales[1, :, begin:L, None].float()).to(BF16)
            assert torch.equal(got[1, :, :L - begin].view(torch.int16), want.view(torch.int16))
            assert (got[1, :, L - begin:] == 9.0).all() and (got[0] == 9.0).all()
    tree_q = su.randn(9, B, n, G * Hkv, 128).cuda()
    ws, got = ffd.tree_workspace(s, n), torch.zeros_like(tree_q)
    ffd.decode_tree(s, cache, tree_q, lengths, got, ws)
    assert ffd.check_device_status(ws) == 0
    for b, h in ((0, 7), (1, 0), (1, 7)):
        end = int(lengths[b])
        kk, vv = cache.k[b, h, :end].double(), cache.v[b, h, :end].double()
        top = torch.ones(end, dtype=torch.float64, device="cuda")
        if fmt == ffd.FFD_CACHE_BYTE:
            kk *= cache.k_scales[b, h, :end, None].double()
            top = cache.v_scales[b, h, :end].double()
            vv *= top[:, None]
        for i in range(n):
            at = end - n + i + 1
            for g in range(G):
                x = tree_q[b, i, h * G + g].double()
                p = torch.softmax(kk[:at] @ x / 128 ** 0.5, -1)
                want, mag = p @ vv[:at], p @ vv[:at].abs()
                # weights with 8 significant bits and the output in bf16, up to 2^-8 each;
                # fp32 sums over 2^21 tokens, a CTA's 2^14 one after another: below 2^-9
                tol = want.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + 2.0 ** -9)
                if fmt == ffd.FFD_CACHE_BYTE:  # units of 2^-16 of the largest weight times scale
                    tol = tol + float((p * top[:at]).max()) * at * 2.0 ** -17 * 448
                assert ((got[b, i, h * G + g].double() - want).abs() <= tol).all(), (b, h, i, g)
