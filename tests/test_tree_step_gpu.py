"""The multi-token operators as they run together: TreeStep (append, tree
attention, accepted nodes) and rotary positions in the stand-in layer."""
import numpy as np
import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import StandInAttentionLayer, TreeStep, ffd

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _rows(cache, b, slots):
    """Rows of the cache as values, float64 [Hkv, slots, 128] each."""
    k, v = cache.k[b, :, slots].cpu().double(), cache.v[b, :, slots].cpu().double()
    if cache.k_scales is not None:
        k *= cache.k_scales[b, :, slots].cpu().double()[..., None]
        v *= cache.v_scales[b, :, slots].cpu().double()[..., None]
    return k, v


@pytest.mark.parametrize("fmt", [ffd.FFD_CACHE_BF16, ffd.FFD_CACHE_BYTE])
@pytest.mark.parametrize("rotary", [0, 64])
def test_draft_verify_accept(fmt, rotary):
    """Two trees verified after another; between them a path is accepted.  The
    attention of each is checked against the cache that the operators left, the
    cache against the rows that were appended."""
    B, G, Hkv, cap, n = 3, 4, 2, 512, 7
    s = su.shape(B, G, Hkv, cap)
    o = su.options(rotary, "half") if rotary else None
    cache = ffd.KVCache.empty(s, fmt)
    start = [5, 200, 300]
    lengths = torch.tensor(start, dtype=torch.int32).cuda()
    k0, v0 = su.randn(1, B, 300, Hkv, 128).cuda(), su.randn(2, B, 300, Hkv, 128).cuda()
    # the prompts, right-aligned: token i of a sequence goes to slot lengths - count + i
    ffd.append_tokens(s, cache, k0, v0, lengths, rope=ffd.Rope(**o) if o else None, new_lengths=lengths)
    step = TreeStep(s, cache, lengths, n, rope=ffd.Rope(**o) if o else None)
    parents = [[-1, 0, 0, 1, 1, 2, 5], [-1, -1, 0], [-1, 0, 1, 2, 3, 4, 5]]
    paths = [[0, 2, 5], [1], [0, 1, 2, 3, 4]]
    now = list(start)
    for turn in range(2):
        mask, depth = ffd.tree_from_parents(parents)
        step.tree_mask.copy_(mask)
        step.depth.copy_(depth)
        sizes = [len(p) for p in parents]
        step.sizes.copy_(torch.tensor(sizes, dtype=torch.int32))
        q, k, v = (su.randn(10 * turn + i, B, n, h, 128) for i, h in ((3, G * Hkv), (4, Hkv), (5, Hkv)))
        step.q.copy_(q)
        step.k_new.copy_(k)
        step.v_new.copy_(v)
        got = step.step().cpu()
        kk, vv = (torch.zeros(B, Hkv, cap, 128, dtype=torch.float64) for _ in range(2))
        rotated = q.clone()
        for b in range(B):
            end = now[b] + sizes[b]
            kk[b, :, :end], vv[b, :, :end] = _rows(cache, b, torch.arange(end))
            if o:
                rotated[b] = su.rotate64(q[b], now[b] + depth[b], o).to(BF16)
        words = [[int(w) % (1 << 64) for w in row] for row in mask]
        scales = None
        if fmt == ffd.FFD_CACHE_BYTE:
            scales = torch.zeros(B, Hkv, cap, dtype=torch.float64)
            for b in range(B):
                scales[b, :, :now[b] + sizes[b]] = cache.v_scales[b, :, :now[b] + sizes[b]].cpu().double()
        want, tol = su.tree64(rotated, kk, vv, [x + m for x, m in zip(now, sizes)], sizes, words, weight_scale=scales)
        if o:
            # the kernel's rotated query may round the other way, by one step of bf16 (2^-7):
            # a score of std 1 moves by at most 2^-7 |k| |q| / sqrt(128) over few channels
            tol = tol + want.abs() * 2.0 ** -5 + 2.0 ** -6
        for b, m in enumerate(sizes):
            assert ((got[b, :m].double() - want[b, :m]).abs() <= tol[b, :m]).all(), (turn, b)
        # accept a path: the next turn's sequences end with its nodes
        width = max(len(p) for p in paths)
        nodes = torch.tensor([p + [0] * (width - len(p)) for p in paths]).cuda()
        counts = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
        step.accept(nodes, counts)
        for b, path in enumerate(paths):
            slots = torch.arange(now[b], now[b] + len(path))
            have_k, have_v = _rows(cache, b, slots)
            new_k, new_v = k[b, path], v[b, path].double()
            new_k = su.rotate64(new_k, slots, o) if o else new_k.double()
            half = 2.0 ** -8 if fmt == ffd.FFD_CACHE_BF16 else 2.0 ** -4
            for have, new in ((have_k, new_k), (have_v, new_v)):
                new = new.transpose(0, 1)
                # half a step of the format; e4m3: or half its smallest step, 2^-10 of
                # amax / 448 (and a scale of bf16 on either side of it)
                room = new.abs() * half * 1.01 + new.abs().amax(-1, keepdim=True) * (
                    2.0 ** -20 if fmt == ffd.FFD_CACHE_BF16 else 2.0 ** -18)
                assert ((have - new).abs() <= room).all(), (turn, b)
            now[b] += len(path)
        assert lengths.cpu().tolist() == now
    assert step.check() == 0


def test_no_room_for_the_nodes():
    s = su.shape(2, 2, 1, 64)
    cache = ffd.KVCache.empty(s, ffd.FFD_CACHE_BF16)
    cache.k.zero_()
    cache.v.zero_()
    lengths = torch.tensor([10, 62], dtype=torch.int32).cuda()
    step = TreeStep(s, cache, lengths, 4)
    step.v_new.fill_(1.0)
    out = step.step().cpu()
    assert (out[1] == 0).all() and (out[0] != 0).any()
    assert (cache.v[1] == 0).all()
    assert step.check() == ffd.FFD_DEVICE_FLAG_BAD_LENGTH


def test_single_node_is_the_dense_step():
    """A tree of one node after a rotated append: ffd_decode_append at delta
    infinity with the query and key rotated by ffd_rotate."""
    s = su.shape(2, 4, 2, 512)
    rope = ffd.Rope(**su.options(128, "half"))
    lengths = torch.tensor([100, 511], dtype=torch.int32).cuda()
    k, v = su.randn(1, 2, 2, 512, 128).cuda(), su.randn(2, 2, 2, 512, 128).cuda()
    cache = ffd.KVCache(k.clone(), v.clone())
    step = TreeStep(s, cache, lengths, 1, rope=rope)
    q, kn, vn = (su.randn(i, 2, 1, h, 128).cuda() for i, h in ((3, 8), (4, 2), (5, 2)))
    step.q.copy_(q)
    step.k_new.copy_(kn)
    step.v_new.copy_(vn)
    got = step.step().clone()
    q2, k2 = q[:, 0].contiguous(), kn[:, 0].contiguous()
    ffd.rotate(rope, lengths, q2, q2, k2, k2)
    bufs = ffd.DecodeBuffers(s)
    ffd.quantize_keys(s, k, lengths, 0, bufs.k_packed, bufs.k_scales)
    total = lengths + 1
    ffd.decode_append(s, q2, k2, vn[:, 0].contiguous(), k, v, bufs.k_packed, bufs.k_scales, total, float("inf"),
                      bufs.out, bufs.mask, bufs.workspace)
    for b, at in enumerate((100, 511)):
        assert torch.equal(cache.k[b, :, at], k[b, :, at]) and torch.equal(cache.v[b, :, at], v[b, :, at])
    # both round weights to 8 significant bits and the result to bf16
    mag = v[:, :, :].float().abs().amax()
    assert (got[:, 0].float() - bufs.out.float()).abs().max() <= mag * 2 * 2.0 ** -8


@pytest.mark.parametrize("layout,advance", [("half", True), ("interleaved", False)])
def test_stand_in_layer_with_rotary_positions(layout, advance):
    B, G, Hkv, cap, hidden = 2, 4, 2, 512, 256
    s = su.shape(B, G, Hkv, cap)
    o = su.options(128, layout)
    start = [300, 77]
    k, v = su.randn(1, B, Hkv, cap, 128).cuda(), su.randn(2, B, Hkv, cap, 128).cuda()
    lengths = torch.tensor(start, dtype=torch.int32).cuda()
    layer = StandInAttentionLayer(s, hidden, k, v, lengths, float("inf"), seed=3, advance=advance, rope=ffd.Rope(**o))
    rng = np.random.default_rng(1)
    for i in range(2):
        x = torch.from_numpy(rng.standard_normal((B, hidden)).astype(np.float32)).to(BF16)
        layer.host_x.copy_(x)
        layer.step()
        at = [n + i if advance else n - 1 for n in start]
        q = torch.matmul(x.cuda(), layer.w_q).view(B, G * Hkv, 128).cpu()
        kn = torch.matmul(x.cuda(), layer.w_k).view(B, Hkv, 128).cpu()
        pos = torch.tensor(at)
        want_k = su.rotate64(kn, pos, o)
        for b in range(B):
            err = (k[b, :, at[b]].cpu().double() - want_k[b]).abs()
            # a projection may round to the next bf16 in another call (2^-7), then one rounding
            bound = su.rotate_bound(kn[b:b + 1], want_k[b:b + 1], o)[0] + kn[b].double().abs().amax(-1, keepdim=True) * 2.0 ** -6
            assert (err <= bound).all()
        rq = su.rotate64(q, pos, o)
        att = torch.zeros(B, G * Hkv, 128, dtype=torch.float64)
        for b in range(B):
            for h in range(G * Hkv):
                kk, vv = (t[b, h // G, :at[b] + 1].cpu().double() for t in (k, v))
                att[b, h] = torch.softmax(kk @ rq[b, h] / 128 ** 0.5, -1) @ vv
        want = att.to(BF16).view(B, -1).double() @ layer.w_o.cpu().double()
        err = (layer.host_y.double() - want).abs().max()
        assert err <= 2e-2 * max(1.0, float(want.abs().max())), (i, float(err))
    assert layer.core.check() == 0
