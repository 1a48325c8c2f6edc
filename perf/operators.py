"""Measured cases of the serving operators around the decode step.

Four operators, used together when drafted tokens are verified against a long
cache: ``rotate`` (rotary positions of queries and keys), ``append_tokens``
(rotary positions and the cache write in one, into a bf16 or an e4m3 cache),
``read_cache`` (an e4m3 cache read back to bf16) and ``decode_tree``
(attention of a tree of drafted tokens over the cache; one node is the
ordinary single-token step).

With ``own`` false, :func:`run` computes an operator from elementary torch
operations in 32 bits (angles in 64); with ``own`` true it makes the calls a
user makes.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128                # head dimension of every shape
E4M3_MAX = 448.0       # largest finite e4m3 value
SPREAD = 1.5           # standard deviation of the cache rows' magnitudes, in octaves


# ------------------------------------------------------------------ cases --

def _rotate(name, tokens, q_heads, kv_heads, rotary, layout, scaling, far, inverse=False):
    return {"name": name, "op": "rotate", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "rotary": rotary, "layout": layout, "scaling": scaling, "far": far, "inverse": inverse}


def _append(name, batch, new, q_heads, kv_heads, capacity, shortest, longest, cache, rotary, layout,
            scaling, tree, ragged=False):
    return {"name": name, "op": "append", "batch": batch, "new": new, "q_heads": q_heads,
            "kv_heads": kv_heads, "capacity": capacity, "shortest": shortest, "longest": longest,
            "cache": cache, "rotary": rotary, "layout": layout, "scaling": scaling, "tree": tree,
            "ragged": ragged}


def _read(name, batch, kv_heads, capacity, shortest, longest, begin, count):
    return {"name": name, "op": "read", "batch": batch, "kv_heads": kv_heads, "capacity": capacity,
            "shortest": shortest, "longest": longest, "begin": begin, "count": count}


def _tree(name, batch, nodes, q_heads, kv_heads, capacity, shortest, longest, cache, tree,
          ragged=False):
    return {"name": name, "op": "tree", "batch": batch, "nodes": nodes, "q_heads": q_heads,
            "kv_heads": kv_heads, "capacity": capacity, "shortest": shortest, "longest": longest,
            "cache": cache, "tree": tree, "ragged": ragged}


def listed():
    return [
        # queries and keys of one token for each of 16 sequences: every layer of every step
        _rotate("rotate_step", 16, 32, 8, 128, "half", "none", 65536),
        # an odd-sized prompt, half of each head rotated, interleaved, stretched past its trained length
        _rotate("rotate_prompt", 8191, 32, 8, 64, "interleaved", "by_parts", 1000000),
        # one token for each of 16 sequences into the 8-bit cache, query rotated in the same call
        _append("append_step_e4m3", 16, 1, 32, 8, 2048, 700, 2048, "e4m3", 128, "half", "none", False),
        # drafted trees of up to 31 tokens, ragged, into the bf16 cache
        _append("append_tree_bf16", 4, 31, 32, 8, 4096, 1500, 4000, "bf16", 128, "half", "linear", True,
                ragged=True),
        # a whole prompt of 32K tokens into the 8-bit cache
        _append("append_prompt_e4m3", 1, 32768, 32, 8, 32768, 32768, 32768, "e4m3", 128, "half", "by_parts",
                False),
        # a short odd window of three ragged sequences
        _read("read_window", 3, 8, 4096, 900, 3001, 33, 1001),
        # the whole cache of four 32K sequences, as a bf16 cache is restored from the 8-bit one
        _read("read_all", 4, 8, 32768, 32768, 32768, 0, 32768),
        # a handful of drafted tokens over a short context, one kv-head: latency
        _tree("tree_small_bf16", 1, 5, 4, 1, 4096, 4096, 4096, "bf16", "chain"),
        # 16 drafted tokens over 128K tokens of bf16 cache
        _tree("tree_128k_bf16", 1, 16, 32, 8, 131072, 131072, 131072, "bf16", "random"),
        # the largest trees (256 query rows a kv-head) over ragged contexts
        _tree("tree_wide_bf16", 3, 64, 32, 8, 16384, 5000, 16001, "bf16", "random", ragged=True),
        # single-token decode of four 32K sequences from the 8-bit cache
        _tree("step_32k_e4m3", 4, 1, 32, 8, 32768, 32768, 32768, "e4m3", "chain"),
        # 13 drafted tokens over ragged long contexts in the 8-bit cache
        _tree("tree_ragged_e4m3", 5, 13, 32, 8, 65536, 8192, 65536, "e4m3", "random"),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _heads(rng):
    group, kv = rng.choice([1, 2, 4, 4, 8]), rng.choice([1, 2, 3, 4, 8, 8])
    return group * kv, kv


def _rotary(rng):
    return rng.choice([128, 128, 64, 96, 32, 2, 80]), rng.choice(["half", "interleaved"]), \
        rng.choice(["none", "linear", "base", "by_parts"])


def draw(rng):
    op = rng.choice(["rotate", "append", "read", "tree", "tree"])
    q_heads, kv = _heads(rng)
    rotary, layout, scaling = _rotary(rng)
    cache = rng.choice(["bf16", "e4m3"])
    if op == "rotate":
        c = _rotate("", _log_uniform(rng, 1, 16384), q_heads, kv, rotary, layout, scaling,
                    _log_uniform(rng, 100, 2000000), rng.random() < 0.3)
    elif op == "append":
        batch = _log_uniform(rng, 1, 16)
        most = max(1, 32768 // batch * 8 // max(kv, q_heads // 4))
        new = min(32768, _log_uniform(rng, 1, most))
        longest = min(65536, new + _log_uniform(rng, 1, 4096))
        tree = new <= 64 and rng.random() < 0.5
        c = _append("", batch, new, q_heads, kv, -(-longest // 64) * 64, max(new, longest * 2 // 3), longest,
                    cache, rotary, layout, scaling, tree, ragged=rng.random() < 0.4)
    elif op == "read":
        batch = _log_uniform(rng, 1, 16)
        longest = _log_uniform(rng, 1, 32768 * 4 * 8 // (batch * kv) // 2)
        longest = min(longest, 65536)
        begin = rng.randrange(longest)
        c = _read("", batch, kv, -(-longest // 128) * 128, rng.randint(0, longest), longest, begin,
                  rng.randint(1, longest - begin))
    else:
        batch, nodes = _log_uniform(rng, 1, 8), _log_uniform(rng, 1, 64)
        # query rows times tokens stay below the listed cases'
        most = min(131072, 16 * 32 * 131072 // (batch * nodes * q_heads), 4 * 8 * 65536 // (batch * kv))
        longest = max(nodes, _log_uniform(rng, 1, most))
        shortest = rng.randint(nodes, longest)
        c = _tree("", batch, nodes, q_heads, kv, -(-longest // 64) * 64, shortest, longest, cache,
                  rng.choice(["chain", "random"]), ragged=rng.random() < 0.4)
    c.pop("name")
    return c


def _lengths(c):
    """Tokens of each sequence: evenly spread from the longest to the shortest."""
    b, lo, hi = c["batch"], c["shortest"], c["longest"]
    return [hi - (hi - lo) * i // max(1, b - 1) for i in range(b)]


def _counts(c):
    """New tokens (tree nodes) of each sequence."""
    n = c["new"] if c["op"] == "append" else c["nodes"]
    return [n - (i * n) // (2 * c["batch"]) if c["ragged"] else n for i in range(c["batch"])]


def work(case):
    c = case
    if c["op"] == "rotate":
        rows = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return {"bytes": rows * D * 4 + c["tokens"] * 4, "flops": rows * c["rotary"] * 3}
    if c["op"] == "append":
        tokens = sum(_counts(c))
        row_out = D * 2 if c["cache"] == "bf16" else D + 2
        rows = tokens * c["kv_heads"]
        return {"bytes": rows * 2 * (D * 2 + row_out) + tokens * c["q_heads"] * D * 4 + tokens * 4 * c["tree"],
                "flops": tokens * (c["q_heads"] + c["kv_heads"]) * c["rotary"] * 3
                + (rows * D * 4 if c["cache"] == "e4m3" else 0)}
    if c["op"] == "read":
        rows = sum(max(0, min(n - c["begin"], c["count"])) for n in _lengths(c)) * c["kv_heads"]
        return {"bytes": rows * 2 * (D + 2 + D * 2), "flops": rows * 2 * D}
    token = 2 * D * 2 if c["cache"] == "bf16" else 2 * (D + 2)
    lengths, counts = _lengths(c), _counts(c)
    return {"bytes": sum(lengths) * c["kv_heads"] * token + sum(counts) * c["q_heads"] * D * 4 + sum(counts) * 8,
            "flops": sum(x * y for x, y in zip(lengths, counts)) * c["q_heads"] * D * 4}


# ----------------------------------------------------------------- inputs --

def _random_trees(seed, counts, n):
    """Ancestor sets (bit j of node i's word: i sees j, itself among them) and depths."""
    r = random.Random(seed)
    words, depths = [], []
    for count in counts:
        w, d = [], []
        for i in range(count):
            parent = r.randint(max(-1, i - 6), i - 1)
            w.append((w[parent] if parent >= 0 else 0) | (1 << i))
            d.append(d[parent] + 1 if parent >= 0 else 0)
        words.append([x - (1 << 64) if x >> 63 else x for x in w] + [0] * (n - count))
        depths.append(d + [0] * (n - count))
    return words, depths


def _rope_options(c):
    """The rotary settings of a case, as a model's configuration gives them."""
    o = {"rotary_dim": c["rotary"], "layout": c["layout"], "base": 500000.0, "scaling": c["scaling"]}
    if c["scaling"] != "none":
        o["factor"] = 8.0
    if c["scaling"] == "by_parts":
        o |= {"original_length": 8192.0, "low": 1.0, "high": 32.0, "amplitude": 0.1 * math.log(8.0) + 1.0}
    return o


def _quantised(x):
    """Rows of x as e4m3 codes and bf16 scales, in 32 bits: scale = bf16(amax / 448), code = e4m3(x / scale)."""
    amax = x.abs().amax(-1)
    scale = (amax / torch.full_like(amax, E4M3_MAX)).to(torch.bfloat16)
    wide = scale.float().unsqueeze(-1)
    return torch.where(wide == 0, 0.0, x / wide).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)

    s = {"case": c}
    if c["op"] in ("rotate", "append"):
        s["rope"] = _rope_options(c)
    if c["op"] == "rotate":
        t = c["tokens"]
        s["q"], s["k"] = normal(t, c["q_heads"], D), normal(t, c["kv_heads"], D)
        s["positions"] = torch.randint(0, c["far"], (t,), generator=gen, device=dev, dtype=torch.int32)
        s["q_out"], s["k_out"] = torch.zeros_like(s["q"]), torch.zeros_like(s["k"])
        if own:
            from sparse_long_context_ffd_b200 import ffd
            s["plan"] = ffd.Rope(**s["rope"])
        return s
    B, H, cap = c["batch"], c["kv_heads"], c["capacity"]
    s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device=dev)
    k, v = normal(B, H, cap, D), normal(B, H, cap, D)
    if c["op"] == "read" or c["cache"] == "e4m3":
        # rows of different magnitudes, as tokens have them
        k *= torch.exp2(SPREAD * normal(B, H, cap, 1)) if c["op"] == "read" else 1
        v *= torch.exp2(SPREAD * normal(B, H, cap, 1)).clamp(max=8.0)
        s["k"], s["k_scales"] = _quantised(k.float())
        s["v"], s["v_scales"] = _quantised(v.float())
    else:
        s["k"], s["v"] = k, v
    del k, v
    if c["op"] == "append":
        n, counts = c["new"], _counts(c)
        s["q"], s["k_new"], s["v_new"] = normal(B, n, c["q_heads"], D), normal(B, n, H, D), normal(B, n, H, D)
        s["q_out"] = torch.zeros_like(s["q"])
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev) if c["ragged"] else None
        s["positions"] = None
        if c["tree"]:
            depths = torch.tensor(_random_trees(seed, counts, n)[1], dtype=torch.int32, device=dev)
            first = s["lengths"] - torch.tensor(counts, dtype=torch.int32, device=dev)
            s["positions"] = (first[:, None] + depths).to(torch.int32).contiguous()
    elif c["op"] == "read":
        s["k_out"] = torch.zeros(B, H, c["count"], D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        n, counts = c["nodes"], _counts(c)
        s["q"] = 2 * normal(B, n, c["q_heads"], D)  # logits of standard deviation 2
        s["out"] = torch.zeros_like(s["q"])
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev) if c["ragged"] else None
        s["tree_mask"] = None
        if c["tree"] == "random":
            s["tree_mask"] = torch.tensor(_random_trees(seed, counts, n)[0], dtype=torch.int64, device=dev)
    if own:
        from sparse_long_context_ffd_b200 import ffd
        s["shape"] = ffd.make_shape(B, c.get("q_heads", H), H, cap, 64, 32)
        s["cache"] = ffd.KVCache(s["k"], s["v"], s.get("k_scales"), s.get("v_scales"))
        if c["op"] == "append":
            s["plan"] = ffd.Rope(**s["rope"])
        if c["op"] == "tree":
            s["workspace"] = ffd.tree_workspace(s["shape"], n)
    return s


# ------------------------------------------------------------ plain forms --

def _frequencies(o):
    """Radians a position for each rotated pair."""
    half = o["rotary_dim"] // 2
    base = o["base"]
    if o["scaling"] == "base" and o["rotary_dim"] > 2:
        base *= o["factor"] ** (o["rotary_dim"] / (o["rotary_dim"] - 2))
    f = np.power(base, -np.arange(half, dtype=np.float64) / half)
    if o["scaling"] == "linear":
        f = f / o["factor"]
    if o["scaling"] == "by_parts":
        rotations = o["original_length"] * f / (2 * math.pi)
        keep = np.clip((rotations - o["low"]) / (o["high"] - o["low"]), 0.0, 1.0)
        f = f * keep + f / o["factor"] * (1 - keep)
    return f


def _rotated(x, positions, o, inverse=False):
    """x [..., heads, D] in 32 bits, positions [...]; the angles are reduced in 64 bits."""
    half, amplitude = o["rotary_dim"] // 2, o.get("amplitude", 1.0)
    f = torch.from_numpy(_frequencies(o)).to(x.device)
    angle = positions.double()[..., None, None] * f
    cos = (torch.cos(angle) * amplitude).float()
    sin = (torch.sin(angle) * (-amplitude if inverse else amplitude)).float()
    x = x.float()
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if o["layout"] == "half":
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _run_rotate(s):
    o, inverse = s["rope"], s["case"]["inverse"]
    s["q_out"].copy_(_rotated(s["q"], s["positions"], o, inverse))
    s["k_out"].copy_(_rotated(s["k"], s["positions"], o, inverse))
    return s["q_out"], s["k_out"]


def _run_append(s):
    c = s["case"]
    B, n, H = c["batch"], c["new"], c["kv_heads"]
    dev = s["k"].device
    i = torch.arange(n, device=dev)
    counts = s["counts"] if s["counts"] is not None else torch.full_like(s["lengths"], n)
    slot = (s["lengths"] - counts).long()[:, None] + i
    positions = s["positions"] if s["positions"] is not None else slot
    valid = i < counts[:, None]
    s["q_out"].copy_(torch.where(valid[..., None, None], _rotated(s["q"], positions, s["rope"]),
                                 s["q_out"].float()))
    k, v = _rotated(s["k_new"], positions, s["rope"]), s["v_new"].float()
    b, t = valid.nonzero(as_tuple=True)
    where = (b[:, None], torch.arange(H, device=dev)[None, :], slot[b, t][:, None])
    if c["cache"] == "bf16":
        s["k"][where], s["v"][where] = k[b, t].to(torch.bfloat16), v[b, t].to(torch.bfloat16)
        return s["q_out"], s["k"], s["v"]
    (kc, ks), (vc, vs) = _quantised(k[b, t]), _quantised(v[b, t])
    s["k"].view(torch.uint8)[where], s["v"].view(torch.uint8)[where] = kc.view(torch.uint8), vc.view(torch.uint8)
    s["k_scales"][where], s["v_scales"][where] = ks, vs
    return s["q_out"], s["k"], s["v"], s["k_scales"], s["v_scales"]


def _run_read(s):
    c = s["case"]
    a, z = c["begin"], c["begin"] + c["count"]
    valid = (torch.arange(a, z, device=s["k"].device) < s["lengths"][:, None])[:, None, :, None]
    k = s["k"][:, :, a:z].float() * s["k_scales"][:, :, a:z, None].float()
    v = s["v"][:, :, a:z].float() * s["v_scales"][:, :, a:z, None].float()
    s["k_out"].copy_(torch.where(valid, k, s["k_out"].float()))
    s["v_out"].copy_(torch.where(valid, v, s["v_out"].float()))
    return s["k_out"], s["v_out"]


def _run_tree(s):
    c = s["case"]
    B, n, H, cap = c["batch"], c["nodes"], c["kv_heads"], c["capacity"]
    G = c["q_heads"] // H
    dev = s["k"].device
    k, v = s["k"].float(), s["v"].float()
    if c["cache"] == "e4m3":
        k, v = k * s["k_scales"].float()[..., None], v * s["v_scales"].float()[..., None]
    counts = s["counts"] if s["counts"] is not None else torch.full_like(s["lengths"], n)
    i = torch.arange(n, device=dev)
    words = s["tree_mask"] if s["tree_mask"] is not None else (torch.full_like(i, -1) << i << 1).bitwise_not().expand(B, n)
    node = torch.arange(cap, device=dev) - (s["lengths"] - counts)[:, None]          # [B, cap]
    seen = ((words[:, :, None] >> node.clamp(0, 63)[:, None, :]) & 1).bool()         # [B, n, cap]
    seen = (node < 0)[:, None, :] | (seen & (node < counts[:, None])[:, None, :])
    q = s["q"].float().view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    score = (q @ k.transpose(-1, -2)) * (1 / math.sqrt(D))
    score = score.view(B, H, n, G, cap).masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, H, n * G, cap) @ v).view(B, H, n, G, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(B, n, H * G, D)
    s["out"].copy_(torch.where((i < counts[:, None])[..., None, None], o, s["out"].float()))
    return s["out"]


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"rotate": _run_rotate, "append": _run_append, "read": _run_read, "tree": _run_tree}[c["op"]](s)
    from sparse_long_context_ffd_b200 import ffd
    if c["op"] == "rotate":
        ffd.rotate(s["plan"], s["positions"], s["q"], s["q_out"], s["k"], s["k_out"], inverse=c["inverse"])
        return s["q_out"], s["k_out"]
    if c["op"] == "append":
        ffd.append_tokens(s["shape"], s["cache"], s["k_new"], s["v_new"], s["lengths"], rope=s["plan"],
                          positions=s["positions"], new_lengths=s["counts"], q=s["q"], q_out=s["q_out"])
        if c["cache"] == "bf16":
            return s["q_out"], s["k"], s["v"]
        return s["q_out"], s["k"], s["v"], s["k_scales"], s["v_scales"]
    if c["op"] == "read":
        ffd.read_cache(s["shape"], s["cache"], s["lengths"], c["begin"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    ffd.decode_tree(s["shape"], s["cache"], s["q"], s["lengths"], s["out"], s["workspace"],
                    tree_mask=s["tree_mask"], tree_sizes=s["counts"])
    return s["out"]


# ------------------------------------------------- the definition, 64 bits --

def _turn(x, position, o, inverse=False):
    """One definition at a time: every pair (a, b) becomes amplitude times its rotation by position * frequency."""
    d = o["rotary_dim"]
    m = torch.arange(d // 2, device=x.device)
    first, second = (m, m + d // 2) if o["layout"] == "half" else (2 * m, 2 * m + 1)
    theta = o["base"] * (o["factor"] ** (d / (d - 2)) if o["scaling"] == "base" and d > 2 else 1.0)
    f = torch.exp(-2.0 * m.double() / d * math.log(theta))
    if o["scaling"] == "linear":
        f = f / o["factor"]
    elif o["scaling"] == "by_parts":
        turns = f * o["original_length"] / (2 * math.pi)
        g = ((turns - o["low"]) / (o["high"] - o["low"])).clamp(0, 1)
        f = (1 - g) * f / o["factor"] + g * f
    z = torch.polar(torch.full_like(f, o.get("amplitude", 1.0)).expand(*position.shape, d // 2),
                    position.double()[..., None] * f * (-1 if inverse else 1)).unsqueeze(-2)
    y = x.double().clone()
    w = torch.complex(y[..., first], y[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rotate":
        return tuple(_turn(s[x], s["positions"], s["rope"], c["inverse"]) for x in ("q", "k"))
    lengths = _lengths(c)
    if c["op"] == "read":
        outs = s["k_out"].double(), s["v_out"].double()
        for b, length in enumerate(lengths):
            m = max(0, min(length - c["begin"], c["count"]))
            at = slice(c["begin"], c["begin"] + m)
            for o, x in zip(outs, ("k", "v")):
                o[b, :, :m] = s[x][b, :, at].double() * s[x + "_scales"][b, :, at].double()[..., None]
        return outs
    counts = _counts(c)
    if c["op"] == "append":
        q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
        scales = [s[x].double() for x in ("k_scales", "v_scales")] if c["cache"] == "e4m3" else []
        for b, (length, m) in enumerate(zip(lengths, counts)):
            at = torch.arange(length - m, length, device=q.device)
            p = s["positions"][b, :m] if s["positions"] is not None else at
            q[b, :m] = _turn(s["q"][b, :m], p, s["rope"])
            rows = [_turn(s["k_new"][b, :m], p, s["rope"]).transpose(0, 1), s["v_new"][b, :m].double().transpose(0, 1)]
            for j, cached in enumerate((k, v)):
                if scales:
                    top = rows[j].abs().amax(-1) / E4M3_MAX
                    scales[j][b][:, at] = top
                    rows[j] = rows[j] / top.float().to(torch.bfloat16).double().clamp(min=1e-300)[..., None]
                cached[b][:, at] = rows[j]
        return (q, k, v, *scales)
    out = s["out"].double()
    group = c["q_heads"] // c["kv_heads"]
    for b, (length, m) in enumerate(zip(lengths, counts)):
        visible = torch.ones(m, length, dtype=torch.bool)
        for i in range(m):
            word = (1 << i + 1) - 1 if s["tree_mask"] is None else int(s["tree_mask"][b, i])
            for j in range(m):
                visible[i, length - m + j] = bool(word >> j & 1)
        visible = visible.to(out.device)
        for h in range(c["kv_heads"]):
            k, v = s["k"][b, h, :length].double(), s["v"][b, h, :length].double()
            if c["cache"] == "e4m3":
                k, v = k * s["k_scales"][b, h, :length, None].double(), v * s["v_scales"][b, h, :length, None].double()
            for g in range(group):
                x = s["q"][b, :m, h * group + g].double() @ k.T / math.sqrt(D)
                out[b, :m, h * group + g] = torch.softmax(x.masked_fill(~visible, -math.inf), -1) @ v
    return out
