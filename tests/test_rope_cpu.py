"""Rotary positions without a GPU: the reference's own pins, and every refusal of the calls."""
import ctypes

import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from oracle import rope_ref as rope

RNG = np.random.default_rng(7)
INTERLEAVED, INVERSE = 64, 128


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_is_a_rotation_by_the_angle(interleaved):
    """As complex numbers: (x1 + i x2) e^(i p f); norms stay, and scores depend on distances alone."""
    f = 10000.0 ** (-np.arange(4) / 4)
    tab, x = rope.table(f, 50), RNG.standard_normal((1, 1, 10))
    for p in (0, 1, 17, 49):
        y = rope.rotate(x, tab, [p], 10, interleaved=interleaved)[0, 0]
        for i in range(4):
            lo, hi = rope.pair_channels(i, 4, interleaved)
            z = (x[0, 0, lo] + 1j * x[0, 0, hi]) * np.exp(1j * p * f[i])
            assert np.allclose([y[lo], y[hi]], [z.real, z.imag], atol=1e-13)
        assert np.array_equal(y[8:], x[0, 0, 8:])  # the rest stays
    k = RNG.standard_normal((1, 1, 10))
    at = lambda a, p: rope.rotate(a, tab, [p], 10, interleaved=interleaved)[0, 0]  # noqa: E731
    assert abs(at(x, 5) @ at(k, 2) - at(x, 40) @ at(k, 37)) < 1e-12


def test_reference_turns_back_and_is_its_own_gradient():
    f = 10000.0 ** (-np.arange(8) / 8)
    tab, pos, axes = rope.table(f, 30), RNG.integers(0, 30, (3, 5)), RNG.integers(0, 3, 8)
    x, g = RNG.standard_normal((2, 5, 2, 32))
    args = dict(axes=axes, interleaved=True)
    y = rope.rotate(x, tab, pos, 16, **args)
    assert np.allclose(rope.rotate(y, tab, pos, 16, inverse=True, **args), x, atol=1e-13)
    gx = rope.rotate(g, tab, pos, 16, inverse=True, **args)
    for _ in range(10):  # differences of sum(g y)
        i = tuple(RNG.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = 1e-3
        d = np.sum(g * (rope.rotate(x + e, tab, pos, 16, **args) - rope.rotate(x - e, tab, pos, 16, **args))) / 2e-3
        assert abs(d - gx[i]) < 1e-10


def test_reference_axes_take_their_own_positions():
    f = np.array([1.0, 0.5, 0.25, 0.125])
    tab, x = rope.table(f, 9), RNG.standard_normal((1, 1, 8))
    y = rope.rotate(x, tab, [[3], [7]], 8, axes=[0, 1, 0, 1])
    for i, p in enumerate((3, 7, 3, 7)):
        assert np.allclose(y[0, 0, i], x[0, 0, i] * np.cos(p * f[i]) - x[0, 0, i + 4] * np.sin(p * f[i]))
    assert np.array_equal(rope.rotate(x, tab, [[3], [-1]], 8, axes=[0, 1, 0, 1]), x)


def test_reference_rounds_once():
    x = np.concatenate([RNG.standard_normal(4000), [0.0, 1.00390625, 1.01171875, 1 + 2.0 ** -8 + 2.0 ** -40, -2.0 ** -133 * 1.5, 2.0 ** -140,
                                                    3.4e38, np.inf, -np.inf]])
    grid = np.unique(np.arange(0, 0x7f80, dtype=np.uint16).astype(np.uint32) << 16).astype(np.uint32).view(np.float32).astype(np.float64)
    y = rope.to_bf16(x)
    for a, b in zip(np.abs(x), np.abs(y)):
        if np.isinf(a) or a > 3.39e38:
            assert np.isinf(b)
            continue
        i = np.searchsorted(grid, a)
        near = grid[max(0, i - 1):i + 1]
        best = np.min(np.abs(near - a))
        assert abs(b - a) == best
    assert list(y[4001:4004]) == [1.0, 1.015625, 1.0078125]  # ties to even; a hair above one goes up


def strides(*pairs):
    return (ctypes.c_longlong * 8)(*(v for p in pairs for v in p))


P = ctypes.c_void_p


def rope_call(**kw):
    a = dict(q=64, k=128, qo=256, ko=512, st=strides((256, 128), (128, 128), (256, 128), (128, 128)), tab=1024, pos=4, axes=None, total=4,
             hq=2, hk=1, width=128, d=128, pairs=64, n=1, top=10, flags=0, dtype=0)
    a.update(kw)
    return da.lib().diffattn_rope(P(a["q"]), P(a["k"]), P(a["qo"]), P(a["ko"]), a["st"], P(a["tab"]), P(a["pos"]), P(a["axes"]), a["total"],
                                  a["hq"], a["hk"], a["width"], a["d"], a["pairs"], a["n"], a["top"], a["flags"], a["dtype"], None)


def append_call(kv4=False, **kw):
    a = dict(q=64, k=128, v=256, qo=512, kp=1024, vp=2048, st=strides((256, 128), (128, 128), (128, 128), (256, 128)), tab=1024, pos=4,
             axes=None, slots=8, total=4, hq=2, H=1, kw=128, vw=128, d=128, pairs=64, n=1, top=10, pages=3, page=16, ke=0, ve=0, flags=0)
    a.update(kw)
    head = [P(a["q"]), P(a["k"]), P(a["v"]), P(a["qo"]), P(a["kp"])]
    mid = [a["st"], P(a["tab"]), P(a["pos"]), P(a["axes"]), P(a["slots"]), a["total"], a["hq"], a["H"], a["kw"], a["vw"]]
    if kv4:
        return da.lib().diffattn_rope_kv4_append(*head, *mid, a["pairs"], a["n"], a["top"], a["pages"], a["page"], a["ke"], a["ve"],
                                                 a["flags"], None)
    return da.lib().diffattn_rope_append(*head, P(a["vp"]), *mid, a["d"], a["pairs"], a["n"], a["top"], a["pages"], a["page"],
                                         a["flags"], None)


ARG, SHAPE, DTYPE, ALIGN = -1, -2, -3, -4
COMMON = [
    (dict(tab=None), ARG), (dict(pos=None), ARG), (dict(n=2), ARG), (dict(flags=4), ARG), (dict(q=None), ARG), (dict(k=None), ARG),
    (dict(qo=None), ARG), (dict(st=None), ARG), (dict(total=-1), SHAPE), (dict(hq=-1), SHAPE), (dict(hq=65536), SHAPE),
    (dict(total=1 << 29, hq=8), SHAPE), (dict(pairs=4), SHAPE), (dict(pairs=72), SHAPE), (dict(pairs=20), SHAPE), (dict(pairs=0), SHAPE),
    (dict(n=0), SHAPE), (dict(n=5, axes=4), SHAPE), (dict(top=0), SHAPE), (dict(tab=1028), ALIGN), (dict(pos=6), ALIGN), (dict(q=72), ALIGN),
    (dict(st=strides((252, 128), (128, 128), (256, 128), (128, 128))), ALIGN),
    (dict(st=strides((256, 0), (128, 128), (256, 128), (128, 128))), ALIGN),
    (dict(st=strides((256, 128), (128, 128), (256, 128), (-128, 128))), ALIGN)]


@pytest.mark.parametrize("change,want", COMMON + [
    (dict(dtype=2), DTYPE), (dict(ko=None), ARG), (dict(d=96), SHAPE), (dict(d=256, width=256), SHAPE), (dict(width=192), SHAPE),
    (dict(width=64), SHAPE), (dict(width=8192), SHAPE), (dict(hk=-1), SHAPE), (dict(ko=8), ALIGN)])
def test_rope_refuses(change, want):
    assert rope_call(**change) == want
    assert "diffattn_rope:" in da.lib().diffattn_last_error_string().decode()


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("change,want", COMMON + [
    (dict(v=None), ARG), (dict(kp=None), ARG), (dict(slots=None), ARG), (dict(flags=128), ARG), (dict(H=0), SHAPE), (dict(vw=192), SHAPE),
    (dict(vw=0), SHAPE), (dict(pages=0), SHAPE), (dict(page=0), SHAPE), (dict(pages=1 << 27, page=16), SHAPE), (dict(kp=1032), ALIGN),
    (dict(slots=6), ALIGN), (dict(v=264), ALIGN)])
def test_appends_refuse(kv4, change, want):
    assert append_call(kv4, **change) == want
    assert "append:" in da.lib().diffattn_last_error_string().decode()


@pytest.mark.parametrize("change,want", [
    (dict(page=24), SHAPE), (dict(kw=256), SHAPE), (dict(pairs=24), SHAPE), (dict(ke=65), ARG), (dict(ve=-65), ARG)])
def test_4_bit_append_refuses(change, want):
    assert append_call(True, **change) == want


def test_bf16_append_refuses_its_own():
    assert append_call(False, vp=None) == ARG
    assert append_call(False, vp=2050) == ALIGN
    assert append_call(False, d=96) == SHAPE


def test_table_refuses():
    call = da.lib().diffattn_rope_table
    for args, want in (((None, 16, 3, 8), ARG), ((8, None, 3, 8), ARG), ((8, 16, 0, 8), SHAPE), ((8, 16, 3, 0), SHAPE),
                       ((8, 16, 3, 5000), SHAPE), ((12, 16, 3, 8), ALIGN), ((8, 8, 3, 8), ALIGN)):
        assert call(P(args[0]), P(args[1]), args[2], args[3], None) == want


def test_binding_refuses_tensors_without_a_device():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    t, p = torch.zeros(10, 64, 2), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        da.diffattn_rope(x, x, t, p)
    with pytest.raises(ValueError):
        da.diffattn_rope_append(x, x, x, t, p, p, x, x)
    with pytest.raises(ValueError):
        da.diffattn_rope_kv4_append(x, x, x, t, p, p, x)
    with pytest.raises(ValueError):
        da.diffattn_rope_table(torch.zeros(8, dtype=torch.float64), 4)
    with pytest.raises(ValueError):
        da.diffattn_rope(None, None, t, p)
