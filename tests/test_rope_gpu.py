"""Rotary positions on the GPU against the float64 reference (oracle/rope_ref.py).

bf16 results are the exact value rounded once, over the table's fp32 numbers: they are compared bit by bit
(the products of an 8-bit and a 24-bit factor are exact in fp64, and so is their sum unless one is 2^21
times the other, whose loss of 2^-53 moves a rounding to 8 bits only on a border that the larger product
alone lies on: random tables have none).

fp32: y = x1 c - x2 s with p = fl(x2 s), f = fl(x1 c - p), e = p - x2 s (exact), fl(f + e): off by
2^-24 (|f| + |y|) <= 2^-23 |y| + 2^-24 |e|, |e| <= 2^-24 |p|. TOL = 2^-22 |y| + 2^-46 (|x1| + |x2|).

The table: fp64's sincos is good to some 2 units in its last place of an argument whose rounding is off by
2^-53 p f, and each value is then rounded to fp32: 2^-24 |v| + 2^-52 (1 + p f)."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from oracle import kv4_ref as kv4
from oracle import rope_ref as rope

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.lib()
    yield
    da.diffattn_device_status()


def dev32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32).to(DEV)


def n64(t):
    return t.detach().cpu().double().numpy()


def angles(top, pairs):
    f = 10000.0 ** (-np.arange(pairs) / pairs)
    return torch.as_tensor(rope.table(f, top)).float().to(DEV)


def rows(gen, total, heads, width, dtype=torch.bfloat16):
    x = torch.randn((total, heads, width), generator=gen)
    return (x * 2.0 ** torch.randint(-9, 4, (total, heads, width), generator=gen)).to(dtype).to(DEV)


def places(gen, n, total, top, gaps=True):
    p = torch.randint(0, top, (n, total), generator=gen)
    if gaps and total > 2:
        p[int(torch.randint(0, n, (1,), generator=gen)), ::5] = -1
    return p.to(torch.int32).to(DEV)


def check_rows(got, x, tab, pos, d, before, **kw):
    """bf16 rows bit by bit; rows of tokens left out are those of `before`."""
    want = rope.to_bf16(rope.rotate(n64(x), n64(tab), pos.cpu().numpy(), d, **kw))
    out = np.any(np.atleast_2d(pos.cpu().numpy()) < 0, axis=0)
    want[out] = n64(before)[out]
    assert np.array_equal(n64(got), want)


@pytest.mark.parametrize("top,pairs", [(1, 8), (777, 64), (70000, 24), (3, 4096)])
def test_table(top, pairs):
    f = 10000.0 ** (-np.arange(pairs) / pairs)
    t = da.diffattn_rope_table(torch.as_tensor(f).to(DEV), top)
    want = rope.table(f, top)
    off = np.abs(n64(t) - want)
    angle = np.arange(top)[:, None, None] * f[None, :, None]
    assert np.all(off <= 2.0 ** -24 * np.abs(want) + 2.0 ** -52 * (1 + angle))


def test_table_of_far_positions():
    """Every position up to 2^22, of the fastest pair: an angle formed in fp32 would be off by 0.25 there."""
    top = 1 << 22
    t = da.diffattn_rope_table(torch.tensor([1.0, 0.1], dtype=torch.float64, device=DEV), top)
    p = np.arange(top, dtype=np.float64)
    assert np.max(np.abs(n64(t[:, 0, 0]) - np.cos(p))) <= 2.0 ** -24 + 2.0 ** -29
    assert np.max(np.abs(n64(t[:, 0, 1]) - np.sin(p))) <= 2.0 ** -24 + 2.0 ** -29


CASES = [  # total, hq, hk, parts, d, pairs, axes, top
    (1, 1, 0, 1, 64, 8, 1, 1), (1, 64, 8, 1, 128, 64, 1, 32768), (5, 3, 2, 2, 64, 32, 3, 100), (33, 12, 12, 2, 128, 64, 1, 500),
    (64, 5, 1, 1, 128, 24, 2, 4096), (130, 1, 7, 3, 64, 16, 4, 9), (1000, 2, 3, 1, 128, 56, 1, 2000), (3000, 9, 1, 2, 128, 32, 3, 64),
    (7, 33, 40, 2, 128, 64, 2, 50), (2, 3, 0, 32, 128, 64, 1, 8)]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("total,hq,hk,parts,d,pairs,n,top", CASES)
def test_rope_bf16_is_the_exact_value_rounded_once(total, hq, hk, parts, d, pairs, n, top, interleaved, inverse):
    gen = torch.Generator().manual_seed(total + d)
    tab, pos = angles(top, pairs), places(gen, n, total, top)
    axes = dev32(np.arange(pairs) % n) if n > 1 else None
    q, k = rows(gen, total, hq, parts * d), rows(gen, total, hk, parts * d) if hk else None
    bq, bk = torch.full_like(q, 7.0), torch.full_like(k, -3.0) if hk else None
    got = da.diffattn_rope(q, k, tab, pos if n > 1 else pos[0], d, axes=axes, interleaved=interleaved, inverse=inverse,
                           out=(bq.clone(), bk.clone() if hk else None))
    kw = dict(axes=None if axes is None else axes.cpu().numpy(), interleaved=interleaved, inverse=inverse)
    check_rows(got[0], q, tab, pos, d, bq, **kw)
    if hk:
        check_rows(got[1], k, tab, pos, d, bk, **kw)
    else:
        assert got[1] is None


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("total,hq,hk,parts,d,pairs,n,top", CASES)
def test_rope_fp32(total, hq, hk, parts, d, pairs, n, top, interleaved):
    gen = torch.Generator().manual_seed(total + d + 1)
    tab, pos = angles(top, pairs), places(gen, n, total, top, gaps=False)
    axes = dev32(np.arange(pairs) * n // pairs) if n > 1 else None
    q, k = rows(gen, total, hq, parts * d, torch.float32), rows(gen, total, max(hk, 1), parts * d, torch.float32)
    got = da.diffattn_rope(q, k, tab, pos if n > 1 else pos[0], d, axes=axes, interleaved=interleaved)
    for x, y in ((q, got[0]), (k, got[1])):
        kw = dict(axes=None if axes is None else axes.cpu().numpy(), interleaved=interleaved)
        want = rope.rotate(n64(x), n64(tab), pos.cpu().numpy(), d, **kw)
        size = rope.rotate(np.abs(n64(x)), np.abs(n64(tab)) * [1, -1], pos.cpu().numpy(), d, **kw)
        size = np.maximum(size, np.abs(rope.rotate(np.abs(n64(x)), np.abs(n64(tab)), pos.cpu().numpy(), d, **kw)))
        assert np.all(np.abs(n64(y) - want) <= 2.0 ** -22 * np.abs(want) + 2.0 ** -45 * size)


def test_rope_near_the_borders_of_bf16():
    """Values picked so that the exact result lies on a border of bf16 or a hair beside it, among zeros, signed
    zeros, subnormal and huge values; the kernel's fp64 way decides them."""
    c = np.array([1.0, 0.5, 1 + 2.0 ** -23, 1 - 2.0 ** -24, 0.75, 2.0 ** -20, 0.0, -1.0])
    s = np.array([2.0 ** -8, 2.0 ** -9, 2.0 ** -9, -2.0 ** -8, 2.0 ** -22, 1.0, 1.0, 2.0 ** -30])
    tab = torch.as_tensor(np.stack([c, s], -1)[None]).float().to(DEV)
    vals = [0.0, -0.0, 1.0, -1.0, 1.0078125, 1.9921875, 3.0, 2.0 ** -120, 1.5 * 2.0 ** -133, 3.3e38, -3.3e38, 255.0, 1.0 / 3]
    a, b = np.meshgrid(vals, vals)
    x = torch.zeros((a.size, 1, 64))
    x[:, 0, :8] = torch.as_tensor(a.reshape(-1, 1)).expand(-1, 8)
    x[:, 0, 8:16] = torch.as_tensor(b.reshape(-1, 1)).expand(-1, 8)
    x = x.to(torch.bfloat16).to(DEV)
    pos = dev32(np.zeros(a.size))
    got = n64(da.diffattn_rope(x, None, tab, pos, 64)[0])
    want = rope.rotate(n64(x), n64(tab), pos.cpu().numpy(), 64)
    near = rope.to_bf16(want)
    # below 2^-100: half a step of bf16 (2^-8 of a value, or 2^-134) and a step of fp32's subnormals
    small = np.abs(want) < 2.0 ** -100
    assert np.array_equal(got[~small], near[~small])
    assert np.all(np.abs(got - want)[small] <= 2.0 ** -134 + 2.0 ** -8 * np.abs(want[small]) + 2.0 ** -148)


def test_rope_infinities_and_nans_stay_in_their_pairs():
    gen = torch.Generator().manual_seed(3)
    tab, pos = angles(40, 64), places(gen, 1, 6, 40, gaps=False)[0]
    q = rows(gen, 6, 2, 256)
    clean = da.diffattn_rope(q, None, tab, pos)[0]
    bad = q.clone()
    bad[1, 0, 5], bad[2, 1, 128 + 70], bad[3, 0, 130] = float("inf"), float("nan"), float("-inf")
    got = da.diffattn_rope(bad, None, tab, pos)[0]
    hit = torch.zeros_like(q, dtype=torch.bool)
    for t, h, i in ((1, 0, 5), (1, 0, 69), (2, 1, 134), (2, 1, 198), (3, 0, 130), (3, 0, 194)):
        hit[t, h, i] = True
    assert torch.equal(got[~hit], clean[~hit]) and not torch.isfinite(got[hit]).any()


def test_rope_in_place_on_views_and_streams():
    """q and k as slices of one projection, turned in place on a stream of their own, then back."""
    gen = torch.Generator().manual_seed(4)
    proj = rows(gen, 50, 9, 128)
    before = proj.clone()
    tab, pos = angles(60, 64), places(gen, 1, 50, 60)[0]
    q, k = proj[:, :4], proj[:, 4:6]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = da.diffattn_rope(q, k, tab, pos, out=(q, k), stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert got[0].data_ptr() == q.data_ptr()
    check_rows(q, before[:, :4], tab, pos, 128, before[:, :4])
    check_rows(k, before[:, 4:6], tab, pos, 128, before[:, 4:6])
    assert torch.equal(proj[:, 6:], before[:, 6:])
    big = torch.full((50, 7, 256), 2.0, dtype=torch.bfloat16, device=DEV)  # an output with other strides
    da.diffattn_rope(before[:, :4], None, tab, pos, out=(big[:, 1:5, 128:], None))
    check_rows(big[:, 1:5, 128:], before[:, :4], tab, pos, 128, torch.full_like(before[:, :4], 2.0))
    assert torch.all(big[:, :, :128] == 2) and torch.all(big[:, 5:] == 2) and torch.all(big[:, 0] == 2)


def test_rope_bad_positions_are_reported_and_left_out():
    gen = torch.Generator().manual_seed(5)
    tab, q = angles(10, 64), rows(gen, 4, 2, 128)
    out = torch.full_like(q, 9.0)
    da.diffattn_device_status()
    da.diffattn_rope(q, None, tab, dev32([3, 10, -2, 9]), out=(out, None))
    with pytest.raises(da.DiffAttnError):
        da.diffattn_device_status()
    assert torch.all(out[1:3] == 9)
    check_rows(out[[0, 3]], q[[0, 3]], tab, dev32([3, 9]), 128, out[[0, 3]])
    da.diffattn_rope(q, None, tab, dev32(np.ones((2, 4))), axes=dev32([5] + [1] * 63), out=(out, None))
    with pytest.raises(da.DiffAttnError):
        da.diffattn_device_status()
    assert torch.equal(out, da.diffattn_rope(q, None, tab, dev32([1] * 4))[0])


def test_rope_gradient_through_the_operator():
    """The gradient of a score after rotation, by autograd through plain operations and by turning back."""
    gen = torch.Generator().manual_seed(6)
    tab, pos = angles(300, 64), places(gen, 1, 90, 300, gaps=False)[0]
    x = torch.randn((90, 3, 256), generator=gen).to(DEV)
    g = torch.randn((90, 3, 256), generator=gen).to(DEV)
    xd = x.double().requires_grad_()
    c, s = (tab[pos.long()].double()[:, None, None, :, i] for i in (0, 1))
    h = xd.unflatten(-1, (2, 2, 64))
    y = torch.stack([h[..., 0, :] * c - h[..., 1, :] * s, h[..., 1, :] * c + h[..., 0, :] * s], -2).flatten(2)
    y.backward(g.double())
    gx, _ = da.diffattn_rope(g, None, tab, pos, inverse=True)
    assert torch.max((gx.double() - xd.grad).abs()) <= 2.0 ** -21 * g.abs().max()
    fx, _ = da.diffattn_rope(x, None, tab, pos)
    assert torch.max((fx.double() - y.detach()).abs()) <= 2.0 ** -21 * x.abs().max()


def test_rope_captured_and_replayed():
    gen = torch.Generator().manual_seed(8)
    tab, pos = angles(64, 64), places(gen, 1, 20, 64, gaps=False)[0]
    q = rows(gen, 20, 4, 128)
    out = torch.zeros_like(q)
    da.diffattn_rope(q, None, tab, pos, out=(out, None))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        da.diffattn_rope(q, None, tab, pos, out=(out, None))
    for seed in (1, 2):
        q.copy_(rows(torch.Generator().manual_seed(seed), 20, 4, 128))
        pos.copy_(places(torch.Generator().manual_seed(seed), 1, 20, 64, gaps=False)[0])
        g.replay()
        check_rows(out, q, tab, pos, 128, out)


APPENDS = [  # form, total, hq, H, pages, page, pairs, axes, interleaved
    ("v1", 1, 1, 1, 2, 16, 64, 1, False), ("v1", 70, 12, 12, 9, 32, 64, 1, False), ("v1", 33, 0, 3, 5, 16, 32, 3, True),
    ("v2", 64, 64, 8, 9, 48, 64, 1, False), ("v2", 500, 4, 2, 40, 16, 16, 2, False), ("v2", 17, 8, 1, 3, 16, 24, 1, True),
    ("v2", 3000, 16, 8, 60, 64, 64, 3, False)]


def append_inputs(form, total, hq, H, pages, page, pairs, n, seed):
    gen = torch.Generator().manual_seed(seed)
    w = 256 if form == "v1" else 128
    proj = rows(gen, total + 1, hq + 2 * H, w)[:total]
    pos = places(gen, n, total, 900)
    slots = torch.randperm(pages * page, generator=gen)[:total]
    slots[3::7] = -1
    axes = dev32(np.arange(pairs) % n) if n > 1 else None
    return w, proj[:, :hq], proj[:, hq:hq + H], proj[:, hq + H:], angles(900, pairs), pos if n > 1 else pos[0], slots.to(torch.int32).to(DEV), axes


@pytest.mark.parametrize("form,total,hq,H,pages,page,pairs,n,interleaved", APPENDS)
def test_append_to_bf16_pages(form, total, hq, H, pages, page, pairs, n, interleaved):
    w, q, k, v, tab, pos, slots, axes = append_inputs(form, total, hq, H, pages, page, pairs, n, 11)
    page = page - 5 if total < pages * (page - 5) else page  # a bf16 page may have any size
    slots = torch.where(slots >= pages * page, -1, slots)
    gen = torch.Generator().manual_seed(2)
    kp, vp = (rows(gen, pages * page, H, w).view(pages, page, H, w) for _ in range(2))
    k0, v0 = n64(kp).reshape(-1, H, w), n64(vp).reshape(-1, H, w)
    got = da.diffattn_rope_append(q if hq else None, k, v, tab, pos, slots, kp, vp, axes=axes, interleaved=interleaved)
    kw = dict(axes=None if axes is None else axes.cpu().numpy(), interleaved=interleaved)
    turned = rope.to_bf16(rope.rotate(n64(k), n64(tab), pos.cpu().numpy(), 128, **kw))
    s = slots.cpu().numpy()
    keep = (s >= 0) & np.all(np.atleast_2d(pos.cpu().numpy()) >= 0, axis=0)
    k0[s[keep]], v0[s[keep]] = turned[keep], n64(v)[keep]
    assert np.array_equal(n64(kp).reshape(-1, H, w), k0) and np.array_equal(n64(vp).reshape(-1, H, w), v0)
    if hq:
        live = torch.as_tensor(np.all(np.atleast_2d(pos.cpu().numpy()) >= 0, axis=0))
        assert torch.equal(got.cpu()[live], da.diffattn_rope(q, None, tab, pos, axes=axes, interleaved=interleaved)[0].cpu()[live])
    else:
        assert got is None


@pytest.mark.parametrize("k_exp,v_exp", [(0, 0), (3, -2)])
@pytest.mark.parametrize("form,total,hq,H,pages,page,pairs,n,interleaved", APPENDS)
def test_append_to_4_bit_pages(form, total, hq, H, pages, page, pairs, n, interleaved, k_exp, v_exp):
    """Byte by byte what the reference writes of the turned keys' bf16, and what the two calls give."""
    w, q, k, v, tab, pos, slots, axes = append_inputs(form, total, hq, H, pages, page, pairs, n, 13)
    kp = w // 128
    pool = torch.randint(0, 256, (pages, H, page // 16, 2 * kp * 1152), generator=torch.Generator().manual_seed(1)).to(torch.uint8).to(DEV)
    want, two = pool.cpu().numpy().copy(), pool.clone()
    got = da.diffattn_rope_kv4_append(q if hq else None, k, v, tab, pos, slots, pool, axes=axes, interleaved=interleaved, k_exp=k_exp,
                                      v_exp=v_exp)
    kw = dict(axes=None if axes is None else axes.cpu().numpy(), interleaved=interleaved)
    left_out = np.any(np.atleast_2d(pos.cpu().numpy()) < 0, axis=0)
    s = np.where(left_out, -1, slots.cpu().numpy())
    if total <= 100:
        turned = rope.to_bf16(rope.rotate(n64(k), n64(tab), pos.cpu().numpy(), 128, **kw))
        for i in np.flatnonzero(s >= 0):
            for h in range(H):
                kv4.write_row(want[s[i] // page, h, s[i] % page // 16], kp, turned[i, h], n64(v)[i, h], s[i] % 16, k_exp, v_exp)
        assert np.array_equal(pool.cpu().numpy(), want)
    kt = da.diffattn_rope(k, None, tab, pos, axes=axes, interleaved=interleaved, out=(torch.zeros_like(k), None))[0]
    da.diffattn_kv4_append(kt, v, dev32(s), two, k_exp, v_exp)
    assert torch.equal(pool, two)
    if hq:
        live = torch.as_tensor(~left_out)
        assert torch.equal(got.cpu()[live], da.diffattn_rope(q, None, tab, pos, axes=axes, interleaved=interleaved)[0].cpu()[live])


@pytest.mark.parametrize("kv4", [False, True])
def test_append_bad_slots_are_reported_and_left_out(kv4):
    w, q, k, v, tab, pos, slots, axes = append_inputs("v2", 40, 4, 2, 5, 16, 64, 1, 17)
    bad = slots.clone()
    bad[0], bad[10] = 80, -2
    fixed = slots.clone()
    fixed[0] = fixed[10] = -1
    da.diffattn_device_status()
    out = []
    for s in (bad, fixed):
        if kv4:
            pools = (torch.zeros((5, 2, 1, 2304), dtype=torch.uint8, device=DEV),)
            qo = da.diffattn_rope_kv4_append(q, k, v, tab, pos.clamp(min=0), s, *pools)
        else:
            pools = tuple(torch.zeros((5, 16, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
            qo = da.diffattn_rope_append(q, k, v, tab, pos.clamp(min=0), s, *pools)
        if s is bad:
            with pytest.raises(da.DiffAttnError):
                da.diffattn_device_status()
        out.append((qo, *pools))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    da.diffattn_device_status()


def test_binding_refuses():
    gen = torch.Generator().manual_seed(9)
    tab, pos, q = angles(20, 64), dev32([1, 2, 3]), rows(gen, 3, 2, 128)
    pools = [torch.zeros((2, 16, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    p4 = torch.zeros((2, 2, 1, 2304), dtype=torch.uint8, device=DEV)
    slots = dev32([0, 1, 2])
    for bad in (lambda: da.diffattn_rope(q.half(), None, tab, pos), lambda: da.diffattn_rope(q, q.float(), tab, pos),
                lambda: da.diffattn_rope(q, q[:2], tab, pos), lambda: da.diffattn_rope(q, None, tab.double(), pos),
                lambda: da.diffattn_rope(q, None, tab, pos.long()), lambda: da.diffattn_rope(q, None, tab, pos[:2]),
                lambda: da.diffattn_rope(q, None, tab, dev32(np.ones((2, 3)))), lambda: da.diffattn_rope(q, None, tab, pos, out=(q, q)),
                lambda: da.diffattn_rope(q.transpose(1, 2), None, tab, pos), lambda: da.diffattn_rope(q.cpu(), None, tab, pos),
                lambda: da.diffattn_rope(q, None, tab, pos.cpu()), lambda: da.diffattn_rope(q, None, tab, pos, axes=dev32([0])),
                lambda: da.diffattn_rope_append(q, q, q, tab, pos, slots[:2], *pools),
                lambda: da.diffattn_rope_append(q, q, q[:2], tab, pos, slots, *pools),
                lambda: da.diffattn_rope_append(None, q, q, tab, pos, slots, *pools, q_out=q),
                lambda: da.diffattn_rope_append(q, q, q, tab, pos, slots, pools[0][:, :, :1], pools[1]),
                lambda: da.diffattn_rope_kv4_append(q, q, q, tab, pos, slots, p4[:, :, :, :1152]),
                lambda: da.diffattn_rope_kv4_append(q, q, q, tab, pos, slots.long(), p4),
                lambda: da.diffattn_rope_table(torch.ones(4, device=DEV), 3)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(da.DiffAttnError):
        da.diffattn_rope(q, None, tab, pos, 64)  # 64 pairs of a part of 64 channels
    with pytest.raises(da.DiffAttnError):
        da.diffattn_rope(torch.zeros((3, 2, 132), dtype=torch.bfloat16, device=DEV)[:, :, 2:130], None, tab, pos)
    none = q[:0]
    a, b = da.diffattn_rope(none, none, tab, pos[:0])
    assert a.shape == (0, 2, 128) and b.shape == (0, 2, 128)
