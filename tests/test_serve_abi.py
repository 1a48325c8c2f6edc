"""Host side of the multi-token operators, without a GPU: the rotary plan,
refusals before any launch, tree masks from parent lists, the plain forms."""
import ctypes
import math
import random

import pytest
import torch

import serve_util as su
from sparse_long_context_ffd_b200 import ffd

INVALID, UNSUPPORTED, WORKSPACE = ffd.FFD_ERR_INVALID_ARG, ffd.FFD_ERR_UNSUPPORTED, ffd.FFD_ERR_WORKSPACE
A = 1 << 20  # 16-byte aligned addresses, never dereferenced on these paths


def at(i):
    return A + (i << 36)  # far apart: no two of them overlap


@pytest.mark.parametrize("rotary", [2, 64, 96, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "by_parts"])
def test_rope_plan(rotary, scaling):
    o = su.options(rotary, "half", scaling)
    r = ffd.Rope(**o)
    for i, f in enumerate(su.frequencies(**o)):
        turns = f / (2 * math.pi)
        assert abs(r.turns[i] / 2.0 ** 64 - turns % 1.0) <= 2.0 ** -45 * max(turns, 2.0 ** -8)
    assert all(r.turns[i] == 0 for i in range(rotary // 2, 64))
    assert r.amplitude == ctypes.c_float(o.get("amplitude", 1.0)).value
    assert (r.rotary_dim, r.layout) == (rotary, 0)


def test_rope_plan_exact_pairs():
    """Pair 0 turns by one radian a position whatever the base."""
    for base in (1.0, 10000.0, 1e6):
        assert abs(ffd.Rope(base=base).turns[0] / 2.0 ** 64 - 1 / (2 * math.pi)) < 1e-16
    # the whole range of frequencies, by parts: untouched at the top, divided at the bottom
    a, b = ffd.Rope(base=1e4), ffd.Rope(**su.options(128, "half", "by_parts"))
    assert a.turns[0] == b.turns[0]
    assert abs(a.turns[63] / 4 - b.turns[63]) <= 1


@pytest.mark.parametrize("bad", [
    {"rotary_dim": 0}, {"rotary_dim": 3}, {"rotary_dim": 130}, {"base": 0.0}, {"base": float("nan")},
    {"amplitude": 0.0}, {"amplitude": float("inf")}, {"amplitude": 1e-60}, {"scaling": "linear", "factor": 0.0},
    {"scaling": "base", "factor": float("inf")}, {"scaling": "by_parts", "factor": 2.0},
    {"scaling": "by_parts", "factor": 2.0, "original_length": 10.0, "low": 3.0, "high": 3.0},
    {"scaling": "by_parts", "factor": 2.0, "original_length": 10.0, "low": -1.0, "high": 3.0}])
def test_rope_refusals(bad):
    with pytest.raises(ffd.FFDError) as e:
        ffd.Rope(**bad)
    assert e.value.status == INVALID


def test_rope_words():
    with pytest.raises(ValueError):
        ffd.Rope(layout="other")
    with pytest.raises(ValueError):
        ffd.Rope(scaling="other")
    lib = ffd.load_library()
    assert lib.ffd_rope_init(None, None) == INVALID


def test_rotate_refusals():
    lib, rope = ffd.load_library(), ffd.Rope()

    def call(r=rope, tokens=5, pos=at(1), inverse=0, hq=4, q=at(2), qo=at(3), hk=2, k=at(4), ko=at(5)):
        return lib.ffd_rotate(None if r is None else ctypes.byref(r), tokens, pos, inverse, hq, q, qo, hk, k, ko, None)

    size = 5 * 4 * 256
    for bad in ({"r": None}, {"tokens": -1}, {"inverse": 2}, {"hq": 0}, {"hk": 0}, {"q": None}, {"qo": None},
                {"pos": None}, {"k": None}, {"ko": None}, {"q": at(2) + 8}, {"qo": at(3) + 2}, {"k": at(4) + 4},
                {"ko": at(5) + 8}, {"pos": at(1) + 2}, {"qo": at(2) + 16}, {"ko": at(3) + size - 16}, {"k": at(3)},
                {"ko": at(2)}, {"ko": at(4) + 256}, {"pos": at(3) + 64}):
        assert call(**bad) == INVALID, bad
    for bad in ({"tokens": 1 << 31}, {"hq": 65536}, {"hk": 65536}):
        assert call(**bad) == UNSUPPORTED, bad
    broken = ffd.Rope()
    broken.rotary_dim = 130
    assert call(r=broken) == INVALID
    broken.rotary_dim, broken.layout = 128, 2
    assert call(r=broken) == INVALID
    assert call(tokens=0, q=None, qo=None, k=None, ko=None, pos=None) == ffd.FFD_OK


def _cache(fmt=0, **over):
    c = ffd._Cache(fmt, 0, at(1), at(2), at(3) if fmt else None, at(4) if fmt else None)
    for name, value in over.items():
        setattr(c, name, value)
    return c


SHAPE = ffd.make_shape(2, 16, 4, 4096, 64, 16)
BAD_CACHES = [_cache(2), _cache(-1), _cache(0, reserved=1), _cache(0, k=None), _cache(0, v=None), _cache(0, v=at(2) + 8),
              _cache(1, k_scales=None), _cache(1, v_scales=None), _cache(1, k_scales=at(3) + 2)]


def test_append_refusals():
    lib, rope = ffd.load_library(), ffd.Rope()

    def call(s=SHAPE, c=_cache(1), r=rope, n=5, q=at(5), k=at(6), v=at(7), pos=at(8), ln=at(9), nl=at(10), qo=at(11)):
        return lib.ffd_append_tokens(ctypes.byref(s), None if c is None else ctypes.byref(c),
                                     None if r is None else ctypes.byref(r), n, q, k, v, pos, ln, nl, qo, None)

    for bad in ({"c": None}, {"n": -1}, {"n": 4097}, {"q": None}, {"qo": None}, {"k": None}, {"v": None}, {"ln": None},
                {"q": at(5) + 2}, {"k": at(6) + 8}, {"v": at(7) + 2}, {"pos": at(8) + 1}, {"ln": at(9) + 2},
                {"nl": at(10) + 3}, {"qo": at(11) + 8}, {"qo": at(5) + 16}, {"qo": at(6)}, {"k": at(1) + 64},
                {"v": at(4)}, {"ln": at(2) + 4}, {"c": _cache(1, v=at(1))}, {"c": _cache(1, k_scales=at(11))},
                *({"c": c} for c in BAD_CACHES)):
        assert call(**bad) == INVALID, bad
    broken = ffd.Rope()
    broken.amplitude = 0
    assert call(r=broken) == INVALID
    assert call(s=ffd.make_shape(2, 12, 4, 4096, 64, 16)) == UNSUPPORTED
    assert call(n=0, c=None, k=None) == ffd.FFD_OK
    assert call(s=ffd.make_shape(0, 16, 4, 4096, 64, 16), c=None) == ffd.FFD_OK


def test_read_refusals():
    lib = ffd.load_library()

    def call(s=SHAPE, c=_cache(1), ln=at(5), begin=0, count=100, k=at(6), v=at(7)):
        return lib.ffd_read_cache(ctypes.byref(s), None if c is None else ctypes.byref(c), ln, begin, count, k, v, None)

    for bad in ({"c": None}, {"c": _cache(0)}, {"ln": None}, {"ln": at(5) + 2}, {"begin": -1}, {"count": -1},
                {"begin": 4097}, {"begin": 4000, "count": 97}, {"k": None, "v": None}, {"k": at(6) + 2}, {"v": at(7) + 8},
                {"k": at(1)}, {"v": at(6)}, {"k": at(3) + 16}, {"begin": 2 ** 31 - 1, "count": 2 ** 31 - 1},
                *({"c": c} for c in BAD_CACHES)):
        assert call(**bad) == INVALID, bad
    assert call(count=0, c=None) == ffd.FFD_OK


def test_tree_refusals():
    lib = ffd.load_library()
    need = lib.ffd_decode_tree_workspace_bytes(ctypes.byref(SHAPE), 9)
    assert need > 0 and need % 256 == 0

    def call(s=SHAPE, c=_cache(1), n=9, q=at(5), ln=at(6), sizes=at(7), mask=at(8), out=at(9), ws=at(10), wb=need):
        return lib.ffd_decode_tree(ctypes.byref(s), None if c is None else ctypes.byref(c), n, q, ln, sizes, mask, out,
                                   ws, wb, None)

    for bad in ({"c": None}, {"n": 0}, {"n": 65}, {"q": None}, {"ln": None}, {"out": None}, {"q": at(5) + 8},
                {"out": at(9) + 2}, {"ws": at(10) + 8}, {"ln": at(6) + 1}, {"sizes": at(7) + 2}, {"mask": at(8) + 4},
                {"out": at(5)}, {"out": at(1) + 256}, {"ws": at(2)}, {"ws": at(9)}, {"out": at(8)}, {"ws": at(5)},
                *({"c": c} for c in BAD_CACHES)):
        assert call(**bad) == INVALID, bad
    assert call(ws=None) == WORKSPACE and call(wb=need - 1) == WORKSPACE
    assert call(s=ffd.make_shape(65535, 4096, 512, 64, 64, 16), n=64, wb=1 << 60) == UNSUPPORTED
    assert call(s=ffd.make_shape(0, 16, 4, 4096, 64, 16), c=None) == ffd.FFD_OK
    assert lib.ffd_decode_tree_workspace_bytes(ctypes.byref(SHAPE), 0) == 0
    assert lib.ffd_decode_tree_workspace_bytes(ctypes.byref(SHAPE), 65) == 0
    init = lib.ffd_decode_tree_workspace_init
    assert init(ctypes.byref(SHAPE), 9, None, need, None) == WORKSPACE
    assert init(ctypes.byref(SHAPE), 9, A, need - 1, None) == WORKSPACE
    assert init(ctypes.byref(SHAPE), 9, A + 8, need, None) == INVALID
    assert init(ctypes.byref(SHAPE), 65, A, need, None) == INVALID


def test_cpu_tensors_are_refused():
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    k = torch.zeros((1, 1, 64, 128), dtype=bf)
    with pytest.raises(ValueError):
        ffd.KVCache(k, k.clone())
    with pytest.raises(ValueError):
        ffd.KVCache(k.to(f8), k.to(f8))
    q = torch.zeros((3, 2, 128), dtype=bf)
    with pytest.raises(ValueError):
        ffd.rotate(ffd.Rope(), torch.zeros(3, dtype=torch.int32), q, q)


def test_trees_from_parents():
    mask, depth = ffd.tree_from_parents([[-1, 0, 0, 1, -1], [], [-1, 0]])
    assert mask.tolist() == [[1, 3, 5, 11, 16], [0] * 5, [1, 3, 0, 0, 0]]
    assert depth.tolist() == [[0, 1, 1, 2, 0], [0] * 5, [0, 1, 0, 0, 0]]
    full, _ = ffd.tree_from_parents([list(range(-1, 63))])
    assert full[0].tolist() == su.signed(su.chain_words(64)) and full[0, 63] == -1
    for bad in ([0], [-1, 1], [-2], [-1] * 65):
        with pytest.raises(ValueError):
            ffd.tree_from_parents([bad])


def test_plain_forms():
    """The 64-bit forms the GPU tests compare with, against torch's own steps."""
    r = random.Random(1)
    q, k, v = su.randn(1, 1, 3, 4, 128), su.randn(2, 1, 2, 40, 128).double(), su.randn(3, 1, 2, 40, 128).double()
    words = [[r.getrandbits(3) | 1 << i for i in range(3)]]
    got, tol = su.tree64(q, k, v, [37], [3], words)
    seen = torch.ones(3, 37, dtype=torch.bool)
    for i in range(3):
        for j in range(3):
            seen[i, 34 + j] = bool(words[0][i] >> j & 1)
    for h in range(4):
        s = (q[0, :, h].double() @ k[0, h // 2, :37].T / 128 ** 0.5).masked_fill(~seen, -math.inf)
        assert torch.allclose(torch.softmax(s, -1) @ v[0, h // 2, :37], got[0, :, h], atol=1e-12)
    assert (tol > 0).all()
    # rotation: complex multiplication
    for layout in ("half", "interleaved"):
        o = su.options(64, layout, "base")
        x, pos = su.randn(4, 5, 2, 128), torch.tensor([0, 1, 2, 1000, 65535])
        y = su.rotate64(x, pos, o)
        z = x.double()[..., :64]
        z = torch.complex(z[..., :32], z[..., 32:]) if layout == "half" else torch.complex(z[..., 0::2], z[..., 1::2])
        f = torch.tensor(su.frequencies(**o), dtype=torch.float64)
        w = z * torch.polar(torch.ones(5, 1, 32, dtype=torch.float64), pos.double()[:, None, None] * f)
        back = torch.cat([w.real, w.imag], -1) if layout == "half" else torch.stack([w.real, w.imag], -1).flatten(-2)
        assert torch.allclose(y[..., :64], back, atol=1e-9)
        assert torch.equal(y[..., 64:], x.double()[..., 64:])
        # lengths are kept, and turning back restores
        assert torch.allclose(su.rotate64(y, pos, o, inverse=True), x.double(), atol=1e-9)
