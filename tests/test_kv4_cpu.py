"""The 4-bit cache without a GPU: the reference's own pins (its small float types against torch's,
its rounding against brute force, its byte order against the header's statement), the plan
reference's invariants, and the entry points' refusals (pure host arithmetic: pointers are never
followed)."""
import ctypes

import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from oracle import kv4_ref as kv4


@pytest.fixture(scope="module")
def L():
    da.build()
    return da.lib()


# ---- the reference ----------------------------------------------------------------------------

def test_e4m3_grid_is_torchs():
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(kv4.E4M3, want)


def test_scales_round_as_torch_rounds():
    x = torch.linspace(0, 460, 20011, dtype=torch.float32)
    want = x.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv4.nearest(np.minimum(x.double().numpy(), 448), kv4.E4M3), want)


def test_codes_are_the_nearest_values_and_ties_go_to_the_even_code():
    x = np.concatenate([np.arange(0, 8, 1 / 64), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 100.0]])
    got = kv4.nearest(x, kv4.E2M1)
    for v, c in zip(x, got):
        d = np.abs(kv4.E2M1 - v)
        best = np.flatnonzero(d == d.min())
        assert c in best and (len(best) == 1 or c % 2 == 0), (v, c)
    assert [int(c) for c in got[-8:]] == [0, 2, 2, 4, 4, 6, 6, 7]


def test_a_block_reads_back_within_its_rounding():
    """|x - c s| <= half a step of e2m1 at its place: s / 4 below 2 s, s / 2 below 4 s, s above (or
    0.4 s where s, rounded down by up to 2^-4, leaves the largest value past 6 s)."""
    x = torch.randn((200, 128), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).double().numpy()
    c, s = kv4.quantize_blocks(x)
    v, sv = kv4.values(c, s), np.repeat(kv4.E4M3[s], 16, axis=-1)
    step = np.where(np.abs(x) <= 2 * sv, 0.25, np.where(np.abs(x) <= 4 * sv, 0.5, 1.0))
    assert np.all(np.abs(x - v) <= step * sv)


def test_a_record_holds_every_value_in_a_place_of_its_own():
    at = []
    for i in range(16):
        at += [kv4.k_code_at(i, t) + n for t in range(4) for n in range(16)]
        at += [kv4.k_scale_at(i, t, u) for t in range(4) for u in range(2)]
    assert sorted(at) == list(range(1152))
    at = []
    for i in range(16):
        at += [kv4.v_code_at(i, g) + n for g in range(8) for n in range(8)]
        at += [kv4.v_scale_at(i, g) for g in range(8)]
    assert sorted(at) == list(range(1152))


def test_rows_read_back_as_written():
    g = np.random.default_rng(3)
    pool = g.integers(0, 256, (2, 3, 2, 4608)).astype(np.uint8)
    k, v = g.normal(size=(3, 256)), g.normal(size=(3, 256)) * 7
    for h in range(3):
        kv4.write_row(pool[1, h, 1], 2, k[h], v[h], 5, 1, -2)
    kk, vv = kv4.read_rows(pool, 2, [1], [21], 1, -2)
    for h in range(3):
        assert np.array_equal(kk[0, h], kv4.values(*kv4.quantize_blocks(k[h], 1), 1))
        assert np.array_equal(vv[0, h], kv4.values(*kv4.quantize_blocks(v[h], -2), -2))


def random_step(rng, B, page_size, max_pages, spare, new_top):
    """A consistent state and a step on it: (seqlens, new_tokens, table, ring, state, total)."""
    cap = max_pages * page_size
    seqlens = rng.integers(0, cap + 1, B) // rng.integers(1, 5, B)
    new = np.minimum(rng.integers(0, new_top + 1, B), cap - seqlens)
    new[rng.random(B) < 0.25] = -1
    new[rng.random(B) < 0.2] = 0
    used = -(-seqlens // page_size)
    need = (-(-(seqlens + np.maximum(new, 0)) // page_size) - used).sum()
    num_pages = int(used.sum() + max(0, need + spare)) or 1
    order = rng.permutation(num_pages)
    table = np.full((B, max_pages), -7)
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    free = order[at:]
    head = int(rng.integers(0, num_pages))
    ring = np.full(num_pages, -9)
    ring[(head + np.arange(len(free))) % num_pages] = free
    return seqlens, new, table, ring, [head, len(free)], int(np.maximum(new, 0).sum())


@pytest.mark.parametrize("seed", range(6))
def test_plan_reference_keeps_every_page_once(seed):
    """After a step each page is in exactly one place: one request's table, or the ring."""
    rng = np.random.default_rng(seed)
    s, n, table, ring, state, total = random_step(rng, 9, 4, 6, 0 if seed % 2 else 5, 9)
    p = kv4.paged_plan(s, n, table, ring, state, 4, total + 3)
    pages = [q for b in range(9) for q in p["block_table"][b, :-(-p["seqlens"][b] // 4)]]
    head, count = p["ring_state"]
    pages += [p["free_ring"][(head + i) % len(ring)] for i in range(count)]
    assert sorted(pages) == list(range(len(ring)))
    slots = p["slot_map"][:total]
    assert len(set(slots.tolist())) == total and np.all(p["slot_map"][total:] == -1)


# ---- refusals ---------------------------------------------------------------------------------

FAKE, ODD16, ODD4 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)
ARG, SHAPE, ALIGN, WORKSPACE = -1, -2, -4, -8


def test_record_bytes(L):
    assert da.diffattn_kv4_record_bytes(256, 256) == 4608 and da.diffattn_kv4_record_bytes(128, 128) == 2304
    for kw, vw in ((128, 256), (64, 64), (0, 0), (-128, -128), (384, 384)):
        assert da.diffattn_kv4_record_bytes(kw, vw) == 0


def test_plan_refusals(L):
    def plan(ptrs=(), B=4, max_pages=8, num_pages=64, page_size=16, total_max=32):
        p = [FAKE] * 11
        for i, v in ptrs:
            p[i] = v
        return L.diffattn_paged_plan(*p, B, max_pages, num_pages, page_size, total_max, None)

    for i in range(10):
        assert plan([(i, None)]) == ARG, i
        assert plan([(i, ODD4)]) == ALIGN, i
    assert plan(B=0) == SHAPE and plan(B=8193) == SHAPE
    assert plan(max_pages=0) == SHAPE and plan(num_pages=0) == SHAPE and plan(page_size=0) == SHAPE
    assert plan(total_max=-1) == SHAPE and plan(total_max=(1 << 30) + 1) == SHAPE
    assert plan(max_pages=1 << 20, page_size=2048) == SHAPE
    assert plan(num_pages=1 << 20, page_size=2048) == SHAPE


def test_append_refusals(L):
    def append(k=FAKE, v=FAKE, slots=FAKE, pool=FAKE, st=(2048, 256, 2048, 256), total=4, H=8, kw=256, vw=256,
               num_pages=10, page_size=16, ke=0, ve=0):
        s = None if st is None else (ctypes.c_longlong * 4)(*st)
        return L.diffattn_kv4_append(k, v, s, slots, pool, total, H, kw, vw, num_pages, page_size, ke, ve, None)

    assert append(k=None) == ARG and append(v=None) == ARG and append(slots=None) == ARG
    assert append(pool=None) == ARG and append(st=None) == ARG
    assert append(ke=65) == ARG and append(ve=-65) == ARG
    assert append(total=-1) == SHAPE and append(H=0) == SHAPE and append(kw=128) == SHAPE
    assert append(kw=64, vw=64) == SHAPE and append(num_pages=0) == SHAPE
    assert append(page_size=8) == SHAPE and append(page_size=24) == SHAPE and append(page_size=0) == SHAPE
    assert append(num_pages=1 << 27) == SHAPE
    assert append(st=(2048, 256, 2044, 256)) == ALIGN and append(st=(2048, -256, 2048, 256)) == ALIGN
    assert append(st=(0, 256, 2048, 256)) == ALIGN
    assert append(k=ODD16) == ALIGN and append(pool=ODD16) == ALIGN and append(slots=ODD4) == ALIGN


def test_gather_refusals(L):
    def gather(p=(), total=4, B=2, H=8, kw=128, vw=128, num_pages=10, page_size=16, max_pages=4, ke=0, ve=0):
        a = [FAKE, FAKE, FAKE, None, FAKE, FAKE]
        for i, v in p:
            a[i] = v
        return L.diffattn_kv4_gather(*a, total, B, H, kw, vw, num_pages, page_size, max_pages, ke, ve, None)

    for i in (0, 1, 2, 4, 5):
        assert gather([(i, None)]) == ARG, i
    assert gather([(0, ODD16)]) == ALIGN and gather([(4, ODD16)]) == ALIGN and gather([(3, ODD4)]) == ALIGN
    assert gather(B=0) == SHAPE and gather(B=8193) == SHAPE and gather(total=-1) == SHAPE
    assert gather(max_pages=0) == SHAPE and gather(max_pages=1 << 27) == SHAPE and gather(kw=256) == SHAPE
    assert gather(page_size=17) == SHAPE and gather(ke=100) == ARG


def test_decode_refusals(L):
    n = ctypes.c_size_t(0)
    assert L.diffattn_decode_kv4_workspace_size(4, 12, 128, 256, ctypes.byref(n)) == 0 and n.value >= 256
    need = n.value
    assert L.diffattn_decode_kv4_workspace_size(4, 12, 64, 128, ctypes.byref(n)) == SHAPE
    assert L.diffattn_decode_kv4_workspace_size(0, 12, 128, 256, ctypes.byref(n)) == SHAPE
    assert L.diffattn_decode_kv4_workspace_size(4, 12, 128, 256, None) == ARG

    def dec(p=(), eps=1e-5, B=4, H=12, d=128, dv=256, num_pages=10, page_size=16, max_pages=4, ke=0, ve=0,
            flags=6, ws=FAKE, ws_bytes=need):
        a = [FAKE] * 6
        for i, v in p:
            a[i] = v
        return L.diffattn_decode_kv4(*a, 0.5, None, eps, B, H, d, dv, num_pages, page_size, max_pages, ke, ve,
                                     flags, ws, ws_bytes, None)

    for i in range(6):
        assert dec([(i, None)]) == ARG, i
    assert dec(flags=8) == ARG and dec(eps=0.0) == ARG and dec(ke=65) == ARG
    assert dec(d=64, dv=128) == SHAPE and dec(dv=128) == SHAPE and dec(B=0) == SHAPE and dec(B=8193) == SHAPE
    assert dec(H=0) == SHAPE and dec(page_size=20) == SHAPE and dec(max_pages=0) == SHAPE
    assert dec(B=8192, H=9, max_pages=1 << 26) == SHAPE
    assert dec([(0, ODD16)]) == ALIGN and dec([(1, ODD16)]) == ALIGN and dec([(4, ODD16)]) == ALIGN
    assert dec([(2, ODD4)]) == ALIGN and dec([(3, ODD4)]) == ALIGN and dec([(5, ODD4)]) == ALIGN
    assert dec(ws=None) == WORKSPACE and dec(ws_bytes=need - 1) == WORKSPACE
    assert dec(ws=ctypes.c_void_p(0x10080)) == WORKSPACE


def test_v2_decode_refusals(L):
    n = ctypes.c_size_t(0)
    assert L.diffattn_v2_decode_kv4_workspace_size(4, 32, 8, 128, ctypes.byref(n)) == 0
    need = n.value
    for bad in ((4, 32, 8, 64), (4, 24, 8, 128), (4, 8, 8, 128), (4, 128, 8, 128), (0, 32, 8, 128), (4, 0, 0, 128)):
        assert L.diffattn_v2_decode_kv4_workspace_size(*bad, ctypes.byref(n)) == SHAPE, bad

    def dec(p=(), B=4, Hq=32, Hkv=8, d=128, num_pages=10, page_size=16, max_pages=4, ke=0, ve=0, flags=0, ws=FAKE,
            ws_bytes=need):
        a = [FAKE] * 6
        for i, v in p:
            a[i] = v
        return L.diffattn_v2_decode_kv4(*a, B, Hq, Hkv, d, num_pages, page_size, max_pages, ke, ve, flags, ws,
                                        ws_bytes, None)

    for i in range(6):
        assert dec([(i, None)]) == ARG, i
    assert dec(flags=8) == ARG and dec(flags=2) == ARG and dec(ve=-70) == ARG
    assert dec(Hq=24) == SHAPE and dec(Hkv=0) == SHAPE and dec(d=64) == SHAPE and dec(B=0) == SHAPE
    assert dec(page_size=8) == SHAPE and dec(num_pages=0) == SHAPE and dec(max_pages=1 << 27) == SHAPE
    assert dec(B=8192, Hq=36, Hkv=9, max_pages=1 << 26) == SHAPE
    assert dec([(0, ODD16)]) == ALIGN and dec([(5, ODD16)]) == ALIGN
    assert dec(ws_bytes=need - 1) == WORKSPACE


def test_binding_refusals():
    """The Python binding checks kinds and shapes before it calls (CPU tensors are refused)."""
    x = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    pool = torch.zeros((3, 4, 1, 2304), dtype=torch.uint8)
    with pytest.raises(ValueError):
        da.diffattn_kv4_append(x, x, i, pool)
    with pytest.raises(ValueError):
        da.diffattn_kv4_gather(pool, i[:, None], i, 2, 128, 128)
    with pytest.raises(ValueError):
        da.diffattn_v2_decode_kv4(x, pool, i[:, None], i, torch.zeros((2, 2)))
    with pytest.raises(ValueError):
        da.diffattn_decode_kv4(x, pool, i[:, None], i, torch.zeros(4))
    with pytest.raises(ValueError):
        da.diffattn_paged_plan(i, i, i[:, None], i, i, 16, 4)
    with pytest.raises(ValueError):
        da.diffattn_kv4_pool(4, 24, 4, 128, 128, device="cpu")
    with pytest.raises(ValueError):
        da.diffattn_kv4_pool(4, 16, 4, 128, 256, device="cpu")
    assert da.diffattn_kv4_pool(4, 32, 3, 256, 256, device="cpu").shape == (4, 3, 2, 4608)
