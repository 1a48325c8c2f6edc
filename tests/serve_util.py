"""Plain 64-bit forms of the multi-token operators, on the CPU, and the error
bounds that follow from their roundings."""
import math

import torch

from sparse_long_context_ffd_b200 import ffd

D = 128
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4, torch.float32: 2.0 ** -24}


def randn(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * scale).to(dtype)


def frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_length=0.0, low=0.0,
                high=0.0, **_):
    out = []
    for i in range(rotary_dim // 2):
        b = base
        if scaling == "base" and rotary_dim > 2:
            b = base * factor ** (rotary_dim / (rotary_dim - 2))
        f = b ** (-2 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        if scaling == "by_parts":
            r = original_length * f / (2 * math.pi)
            g = min(1.0, max(0.0, (r - low) / (high - low)))
            f = (1 - g) * f / factor + g * f
        out.append(f)
    return out


def rotate64(x, positions, options, inverse=False):
    """x [..., heads, 128] -> float64, positions [...]."""
    y = x.double().clone()
    src = x.double()
    d = options["rotary_dim"]
    amp = options.get("amplitude", 1.0)
    for i, f in enumerate(frequencies(**options)):
        a, b = (i, i + d // 2) if options.get("layout", "half") == "half" else (2 * i, 2 * i + 1)
        angle = positions.double() * f * (-1 if inverse else 1)
        c, s = (amp * torch.cos(angle))[..., None], (amp * torch.sin(angle))[..., None]
        y[..., a] = src[..., a] * c - src[..., b] * s
        y[..., b] = src[..., b] * c + src[..., a] * s
    return y


def rotate_bound(x, want, options):
    """One rounding to bf16, and in fp32 two products, a sum and a (cos, sin)
    whose own error is a few steps: 16 half-steps of the pair's magnitude; the
    64-bit reference's own angle is off by 2^-52 of itself (far positions)."""
    amp = options.get("amplitude", 1.0)
    pair = x.double().abs().amax(-1, keepdim=True) * 2 * amp
    return want.abs() * 2.0 ** -8 + pair * (16 * 2.0 ** -24 + 2.0 ** -22)


def quantise64(x32):
    """Rows of fp32 x as (e4m3 codes, bf16 scales), with fp32 steps as the header has them."""
    amax = x32.abs().amax(-1)
    s = (amax / torch.full_like(amax, 448.0)).to(torch.bfloat16)
    w = s.float()[..., None]
    y = torch.where(w == 0, torch.zeros_like(x32), x32 / torch.where(w == 0, torch.ones_like(w), w))
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), s


def chain_words(n):
    return [(1 << (i + 1)) - 1 for i in range(n)]


def signed(words):
    return [w - (1 << 64) if w >> 63 else w for w in words]


def tree64(q, k, v, lengths, sizes, words, tile=128, weight_scale=None):
    """q [B, n, Hq, D]; k, v [B, Hkv, cap, D] float64; words[b][i].  Returns the
    output (rows past the size: zero) and a bound on the error of an output
    whose weights are rounded to 8 significant bits and which is itself
    rounded to bf16; weight_scale [B, Hkv, cap]: the V row scales of the 8-bit
    cache, whose weights have a floor as well."""
    B, n, Hq, _ = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    out = torch.zeros(B, n, Hq, D, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for b in range(B):
        L, m = int(lengths[b]), int(sizes[b])
        for i in range(m):
            slots = [t for t in range(L) if t < L - m or words[b][i] >> (t - (L - m)) & 1]
            if not slots:
                continue
            at = torch.tensor(slots)
            for h in range(Hq):
                kk, vv = k[b, h // G, at], v[b, h // G, at]
                qq = q[b, i, h].double()
                s = kk @ qq / math.sqrt(D)
                p = torch.exp(s - s.max())
                total = p.sum()
                y = (p[:, None] * vv).sum(0) / total
                mag = (p[:, None] * vv.abs()).sum(0) / total
                # scores: 128 fp32 products and sums (each step at most one part in
                # 2^23 of the magnitudes' sum), then an exponential of a score with
                # that error; sums over the tokens likewise
                ds = float((kk.abs() @ qq.abs()).max()) / math.sqrt(D) * 2.0 ** -20 + 2.0 ** -18
                out[b, i, h] = y
                tol[b, i, h] = y.abs() * 2.0 ** -8 + mag * (2.0 ** -8 + 2 * ds)
                if weight_scale is not None:
                    # weights p * v_scale are held in units of 2^-18 of a reference
                    # that is at most 4 times a tile's largest one (half a unit
                    # off each), times codes of up to 448
                    w = p * weight_scale[b, h // G, at]
                    full = torch.zeros((L + tile - 1) // tile * tile, dtype=torch.float64)
                    full[at] = w
                    tops = full.view(-1, tile).amax(1)
                    tol[b, i, h] += float(tops.sum() / total) * tile * 2.0 ** -19 * 4 * 448
    return out, tol


def options(rotary_dim=128, layout="half", scaling="none", **more):
    o = {"rotary_dim": rotary_dim, "layout": layout, "scaling": scaling, "base": 10000.0}
    if scaling != "none":
        o["factor"] = 4.0
    if scaling == "by_parts":
        o |= {"original_length": 4096.0, "low": 1.0, "high": 32.0, "amplitude": 1.1386}
    return o | more


def shape(B, G, Hkv, cap):
    return ffd.make_shape(B, G * Hkv, Hkv, cap, 64, 4)
