"""The 4-bit cache on the GPU against the float64 reference (oracle/kv4_ref.py): the page plan and
the pool's bytes exactly, rows read back exactly, and the decodes within a bound that follows from
their roundings.

The decodes' bound. out = sum_j p_j v_j / sum_j p_j. A cached value enters the products exactly, the
sums are fp32. Each p_j carries
  - its rounding to fp16, 2^-11 of it (at most two such roundings: 2^-10);
  - the error of its score s in the exponent. The query enters exactly, the products of 11-bit
    factors are exact in fp32, and 128 of them are summed: at most 2^-22 of sum |q_i k_i| / sqrt(d)
    per addition step. With |q|_2 <= 40, |k|_2 <= 40 here that is under 128 * 2^-22 * 142 = 2^-7.9
    in the very worst case, where every addition errs by its most in one direction, and about
    sqrt(128) instead of 128 times as much as that of one for errors of either sign: 2^-11.4.
    ex2.approx adds 2^-22.
Both errors move numerator and denominator alike, so twice their sum covers the quotient:
SLACK = 2 (2^-10 + 2^-11) < 2^-8.4, on sum_j p_j |v_j| (reference `bound`). Below 2^-14 fp16 has an
absolute error instead: half its smallest step 2^-24. The kernels hold p at 2^10 against a
reference m that is never above the largest score, so the largest P is at least 2^10, and the
error at most 2^-25 / 2^10 = FLOOR = 2^-35 of it, for each key. The output's own rounding to bf16 is
2^-8 relative (half a step of eps = 2^-7 is 2^-8)."""
import ctypes

import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from oracle import diffattn_ref as ref
from oracle import kv4_ref as kv4
from tests.gpu_util import assert_bf16, to64
from tests.test_kv4_cpu import random_step

pytestmark = pytest.mark.gpu

DEV = "cuda"
SLACK, FLOOR = 2.0 ** -8.4, 2.0 ** -35
BF16 = torch.finfo(torch.bfloat16).eps / 2


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


def within(got, want, bound):
    g = to64(got)
    assert g.shape == want.shape and np.all(np.isfinite(g))
    over = np.abs(g - want) - (bound + BF16 * (np.abs(want) + bound) + 1e-30)
    assert np.all(over <= 0), f"off by {np.max(np.abs(g - want)):.3e}, {np.sum(over > 0)} past the bound"


# ---- plan -------------------------------------------------------------------------------------

def run_plan(s, n, table, ring, state, page_size, total_max, in_place=False):
    S, T, R, St = dev32(s), dev32(table), dev32(ring), dev32(state)
    out = None
    if in_place:
        B = len(s)
        out = {"seqlens": S, "ring_state": St}
        for name, size in (("cu_seqlens_q", B + 1), ("cu_seqlens_k", B + 1), ("slot_map", total_max), ("positions", total_max)):
            out[name] = torch.full((size,), 77, dtype=torch.int32, device=DEV)
    p = da.diffattn_paged_plan(S, dev32(n), T, R, St, page_size, total_max, out=out)
    return {**{k: v.cpu().numpy() for k, v in p.items()}, "block_table": T.cpu().numpy(), "free_ring": R.cpu().numpy()}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page_size,max_pages,spare,new_top", [
    (1, 1, 1, 0, 1), (1, 16, 5, 0, 60), (3, 16, 9, 2, 40), (33, 7, 11, 0, 3), (64, 64, 20, 50, 1), (257, 16, 8, 1, 90),
    (1023, 32, 6, 0, 2), (1024, 16, 3, 9, 1), (1025, 1, 30, 0, 30), (3000, 16, 4, 0, 9), (8192, 16, 2, 3, 1)])
def test_plan(B, page_size, max_pages, spare, new_top, in_place):
    for seed in range(3):
        s, n, table, ring, state, total = random_step(np.random.default_rng(100 * B + seed), B, page_size, max_pages,
                                                      spare, new_top)
        want = kv4.paged_plan(s, n, table, ring, state, page_size, total + seed)
        got = run_plan(s, n, table, ring, state, page_size, total + seed, in_place)
        for name in want:
            assert np.array_equal(got[name], want[name]), name
    da.diffattn_device_status()


def test_plan_one_long_prompt_among_short_ones():
    s, n = np.array([5, 0, 100, 64]), np.array([1, 70001, -1, 1])
    table = np.full((4, 1200), -1)
    table[0, 0], table[2, :2], table[3, 0] = 7, [3, 9], 4
    ring = np.setdiff1d(np.arange(1200), [7, 3, 9, 4])
    ring = np.concatenate([ring, [-1] * 4])
    want = kv4.paged_plan(s, n, table, ring, [0, 1196], 64, 70003)
    got = run_plan(s, n, table, ring, [0, 1196], 64, 70003)
    for name in want:
        assert np.array_equal(got[name], want[name]), name


@pytest.mark.parametrize("what", ["pages", "tokens", "length", "negative", "minus_two", "capacity", "head", "count", "overfull"])
def test_plan_that_does_not_fit_changes_nothing(what):
    s, n = np.array([16, 30, 0, 5]), np.array([1, -1, 40, 0])
    table = np.arange(16).reshape(4, 4)
    ring, state, total_max = np.arange(20, 30), [3, 9], 50
    num_pages = 10
    if what == "pages":
        n[2], n[1], state = 64, 0, [3, 4]
    elif what == "tokens":
        total_max = 40
    elif what == "length":
        s[3] = 65
    elif what == "negative":
        s[0] = -1
    elif what == "minus_two":
        n[3] = -2
    elif what == "capacity":
        n[0] = 49
    elif what == "head":
        state = [num_pages, 3]
    elif what == "count":
        state = [0, num_pages + 1]
    elif what == "overfull":
        state = [0, 10]  # 2 pages come back to a ring that is full
    with pytest.raises(ValueError):
        kv4.paged_plan(s, n, table, ring, state, 16, total_max)
    got = run_plan(s, n, table, ring, state, 16, total_max)
    with pytest.raises(da.DiffAttnError) as e:
        da.diffattn_device_status()
    assert e.value.status == -9
    assert np.array_equal(got["seqlens"], s) and np.array_equal(got["ring_state"], state)
    assert np.array_equal(got["block_table"], table) and np.array_equal(got["free_ring"], ring)
    assert not got["cu_seqlens_q"].any() and not got["cu_seqlens_k"].any()
    assert np.all(got["slot_map"] == -1) and np.all(got["positions"] == -1)


def test_plan_bad_page_gets_no_slot():
    got = run_plan([16, 3], [2, 2], [[0, -1], [99, -1]], [1, -5, 2, 3], [1, 2], 16, 4)
    with pytest.raises(da.DiffAttnError) as e:
        da.diffattn_device_status()
    assert e.value.status == -9
    assert got["slot_map"].tolist() == [-1, -1, -1, -1] and got["positions"].tolist() == [16, 17, 3, 4]
    assert got["block_table"].tolist() == [[0, -5], [99, -1]]


def test_plan_without_positions_or_tokens():
    L, p = da.lib(), lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    s, n, table, ring, state = dev32([3, 20]), dev32([0, -1]), dev32([[1, -1], [2, 0]]), dev32([5, 5, 5]), dev32([1, 0])
    outs = [dev32([9] * 3) for _ in range(4)]
    rc = L.diffattn_paged_plan(p(s), p(n), p(outs[0]), p(table), p(ring), p(state), p(outs[1]), p(outs[2]), p(outs[3]),
                               None, None, 2, 2, 3, 16, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert rc == 0
    assert [o.tolist() for o in outs] == [[3, 0, 9], [1, 2, 9], [0, 0, 0], [0, 0, 0]]
    assert ring.tolist() == [5, 2, 0]
    da.diffattn_device_status()


# ---- rows in ----------------------------------------------------------------------------------

def random_rows(rng, shape, kind="normal"):
    x = rng.normal(size=shape)
    if kind == "wide":  # magnitudes over the whole of bf16, whole blocks of zeros
        x = x * 2.0 ** rng.integers(-40, 30, shape)
        x[..., :16] = 0
    if kind == "ties":  # quotients on the borders of e2m1: multiples of a quarter of a scale
        x = rng.integers(-24, 25, shape) / 4.0
        x[..., ::16] = 6.0
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


def expected_pool(pool, kp, k, v, slots, page_size, k_exp=0, v_exp=0):
    want = pool.copy()
    k, v = to64(k), to64(v)
    for row, slot in enumerate(slots):
        if slot < 0:
            continue
        for h in range(k.shape[1]):
            kv4.write_row(want[slot // page_size, h, slot % page_size // 16], kp, k[row, h], v[row, h], slot % 16, k_exp, v_exp)
    return want


@pytest.mark.parametrize("kind", ["normal", "wide", "ties"])
@pytest.mark.parametrize("kp,H,page_size,total", [(1, 1, 16, 1), (1, 8, 64, 3), (2, 3, 48, 37), (2, 12, 16, 5), (1, 5, 32, 100)])
def test_append(kp, H, page_size, total, kind):
    rng = np.random.default_rng(total * 10 + kp)
    w, pages = 128 * kp, -(-2 * total // page_size) + 2
    k, v = random_rows(rng, (total, H, w), kind), random_rows(rng, (total, H, w), kind)
    slots = rng.permutation(pages * page_size)[:total]
    slots[total // 2] = -1 if total > 1 else slots[0]
    pool = rng.integers(0, 256, (pages, H, page_size // 16, 2304 * kp)).astype(np.uint8)
    want = expected_pool(pool, kp, k, v, slots, page_size)
    got = torch.tensor(pool).to(DEV)
    da.diffattn_kv4_append(k.to(DEV), v.to(DEV), dev32(slots), got)
    assert np.array_equal(got.cpu().numpy(), want)
    da.diffattn_device_status()


@pytest.mark.parametrize("k_exp,v_exp", [(3, -5), (-40, 20), (64, -64)])
def test_append_exponents(k_exp, v_exp):
    rng = np.random.default_rng(9)
    k, v = random_rows(rng, (20, 2, 128), "wide"), random_rows(rng, (20, 2, 128), "wide")
    slots = rng.permutation(32)[:20]
    pool = np.zeros((2, 2, 1, 2304), dtype=np.uint8)
    want = expected_pool(pool, 1, k, v, slots, 16, k_exp, v_exp)
    got = torch.tensor(pool).to(DEV)
    da.diffattn_kv4_append(k.to(DEV), v.to(DEV), dev32(slots), got, k_exp, v_exp)
    assert np.array_equal(got.cpu().numpy(), want)


def test_append_views_and_layouts():
    """Views of one projection, head-major rows, and one row broadcast over the heads' stride."""
    rng = np.random.default_rng(11)
    H, total, pages, ps = 4, 21, 4, 16
    proj = random_rows(rng, (total, 3, H, 256)).to(DEV)
    head_major = random_rows(rng, (H, total, 256)).to(DEV).transpose(0, 1)
    slots = rng.permutation(pages * ps)[:total]
    for k, v in ((proj[:, 1], proj[:, 2]), (head_major, proj[:, 0])):
        pool = np.zeros((pages, H, 1, 4608), dtype=np.uint8)
        want = expected_pool(pool, 2, k, v, slots, ps)
        got = torch.tensor(pool).to(DEV)
        da.diffattn_kv4_append(k, v, dev32(slots), got)
        assert np.array_equal(got.cpu().numpy(), want)
    with pytest.raises(da.DiffAttnError):
        wide = torch.zeros((total, H, 260), dtype=torch.bfloat16, device=DEV)[..., :256]
        da.diffattn_kv4_append(wide, wide, dev32(slots), got)


def test_append_not_finite_and_extremes():
    """A block with an Inf or NaN gets the NaN scale (and reads as NaN), its neighbours do not; a
    block past the largest scale is cut to it; one below the smallest is zero."""
    x = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    x[0, 0, 3], x[0, 0, 20], x[0, 0, 40], x[0, 0, 50] = float("nan"), float("inf"), -float("inf"), 1.0
    x[0, 0, 64], x[0, 0, 65], x[0, 0, 80], x[0, 0, 96] = 30000.0, -1400.0, 2.0 ** -12, 3e38
    x[0, 0, 112], x[0, 0, 113] = 1.0, 2.0 ** -130
    pool = torch.zeros((1, 1, 1, 2304), dtype=torch.uint8, device=DEV)
    da.diffattn_kv4_append(x.to(DEV), x.to(DEV), dev32([7]), pool)
    want = expected_pool(np.zeros((1, 1, 1, 2304), dtype=np.uint8), 1, x, x, [7], 16)
    assert np.array_equal(pool.cpu().numpy(), want)
    k, v = da.diffattn_kv4_gather(pool, dev32([[0]]), dev32([0, 1]), 1, 128, 128, starts=dev32([7]))
    for row in (k[0, 0].float().cpu(), v[0, 0].float().cpu()):
        assert torch.isnan(row[:48]).all() and not torch.isnan(row[48:]).any()
        # 1 / 6 rounds to the scale 11 / 64, and 6 * 11 / 64 = 1.03125
        assert row[50] == 1.03125 and row[64] == 2688.0 and row[65] == -1344.0 and row[80] == 0 and row[96] == 2688.0
        assert row[112] == 1.03125 and row[113] == 0


def test_append_bad_slots_are_skipped_and_reported():
    rng = np.random.default_rng(13)
    k = random_rows(rng, (5, 2, 128))
    slots = [3, 32, -2, 2 ** 31 - 1, 20]
    pool = np.full((2, 2, 1, 2304), 0x5A, dtype=np.uint8)
    got = torch.tensor(pool).to(DEV)
    da.diffattn_kv4_append(k.to(DEV), k.to(DEV), dev32(slots), got)
    with pytest.raises(da.DiffAttnError) as e:
        da.diffattn_device_status()
    assert e.value.status == -9
    want = expected_pool(pool, 1, k[[0, 4]], k[[0, 4]], [3, 20], 16)
    assert np.array_equal(got.cpu().numpy(), want)


def test_append_and_gather_of_no_rows():
    pool = torch.full((1, 2, 1, 2304), 9, dtype=torch.uint8, device=DEV)
    e = torch.empty((0, 2, 128), dtype=torch.bfloat16, device=DEV)
    da.diffattn_kv4_append(e, e, dev32([]), pool)
    k, v = da.diffattn_kv4_gather(pool, dev32([[0]]), dev32([0, 0]), 0, 128, 128)
    assert k.shape == (0, 2, 128) and v.shape == (0, 2, 128) and bool((pool == 9).all())
    da.diffattn_device_status()


# ---- rows out ---------------------------------------------------------------------------------

def random_pool(rng, pages, H, R, kp, top_scale=0x48):
    """A pool of random codes with scales up to 2^2 (code 0x48), none of them NaN."""
    pool = rng.integers(0, 256, (pages, H, R, 2 * kp, 1152)).astype(np.uint8)
    pool[..., 1024:] = rng.integers(0x28, top_scale + 1, pool[..., 1024:].shape)
    return pool.reshape(pages, H, R, 2304 * kp)


def random_table(rng, lens, page_size, spare=2, width=None):
    used = [-(-n // page_size) for n in lens]
    pages = sum(used) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), width or max(1, max(used))), -1)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    return table, pages


@pytest.mark.parametrize("k_exp,v_exp", [(0, 0), (5, -3)])
@pytest.mark.parametrize("kp,H,page_size,lens", [(1, 1, 16, [1]), (2, 3, 16, [15, 16, 17, 0, 33]), (1, 8, 64, [0, 200, 0, 63]),
                                                 (2, 2, 48, [100, 1, 47, 49]), (1, 5, 128, [700, 3])])
def test_gather(kp, H, page_size, lens, k_exp, v_exp):
    rng = np.random.default_rng(sum(lens) + kp)
    table, pages = random_table(rng, lens, page_size)
    pool = random_pool(rng, pages, H, page_size // 16, kp)
    cu, total, w = np.concatenate([[0], np.cumsum(lens)]), sum(lens) + 3, 128 * kp
    out = [torch.full((total, H, w), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    got = da.diffattn_kv4_gather(torch.tensor(pool).to(DEV), dev32(table), dev32(cu), total, w, w, k_exp=k_exp, v_exp=v_exp, out=out)
    for b, n in enumerate(lens):
        want = kv4.sequence_rows(pool, kp, table, b, n, 0, k_exp, v_exp)
        for g, x in zip(got, want):
            assert np.array_equal(to64(g[cu[b]:cu[b + 1]]), x), b
    for g in got:
        assert bool((g[sum(lens):] == 7.0).all())
    da.diffattn_device_status()


def test_gather_from_the_middle_and_bad_pages():
    rng = np.random.default_rng(21)
    table, pages = random_table(rng, [90, 64, 40], 16)
    pool = random_pool(rng, pages, 2, 1, 1)
    starts, counts = [33, 0, 25], [57, 1, 15]
    cu = np.concatenate([[0], np.cumsum(counts)])
    args = (torch.tensor(pool).to(DEV), dev32(table), dev32(cu), sum(counts), 128, 128)
    got = da.diffattn_kv4_gather(*args, starts=dev32(starts))
    for b in range(3):
        for g, x in zip(got, kv4.sequence_rows(pool, 1, table, b, counts[b], starts[b])):
            assert np.array_equal(to64(g[cu[b]:cu[b + 1]]), x)
    da.diffattn_device_status()
    # a page outside the pool reads page 0, a token outside its table is left out; both are reported
    table[0, 3] = pages
    out = [torch.full((sum(counts), 2, 128), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    got = da.diffattn_kv4_gather(args[0], dev32(table), *args[2:], starts=dev32([33, 96, -2]), out=out)
    with pytest.raises(da.DiffAttnError) as e:
        da.diffattn_device_status()
    assert e.value.status == -9
    table[0, 3] = 0
    assert np.array_equal(to64(got[0][:57]), kv4.sequence_rows(pool, 1, table, 0, 57, 33)[0])
    assert bool((got[0][57] == 3.0).all()) and bool((got[0][58:60] == 3.0).all())
    assert np.array_equal(to64(got[1][60:]), kv4.sequence_rows(pool, 1, table, 2, 13, 0)[1])


# ---- decodes ----------------------------------------------------------------------------------

def real_pool(rng, pages, H, R, kp, std=1.0):
    """A pool as rows of normal values leave it."""
    pool = np.empty((pages, H, R, 2304 * kp), dtype=np.uint8)
    t = torch.tensor(pool).to(DEV)
    n = pages * R * 16
    rows = torch.tensor(rng.normal(size=(2, n, H, 128 * kp)) * std, dtype=torch.float32).to(torch.bfloat16).to(DEV)
    da.diffattn_kv4_append(rows[0], rows[1], torch.arange(n, dtype=torch.int32, device=DEV), t)
    return t.cpu().numpy()


def v1_case(rng, lens, H, page_size, std=1.0, spare=2, width=None):
    table, pages = random_table(rng, lens, page_size, spare, width)
    pool = real_pool(rng, pages, H, page_size // 16, 2, std)
    q = torch.tensor(rng.normal(size=(len(lens), H, 256)), dtype=torch.float32).to(torch.bfloat16)
    lam = torch.tensor(rng.uniform(0.2, 0.8, H), dtype=torch.float32)
    w = torch.tensor(rng.uniform(0.8, 1.2, 256), dtype=torch.float32)
    return table, pool, q, lam, w


def v2_case(rng, lens, Hkv, G, page_size, std=1.0, spare=2, width=None):
    table, pages = random_table(rng, lens, page_size, spare, width)
    pool = real_pool(rng, pages, Hkv, page_size // 16, 1, std)
    q = torch.tensor(rng.normal(size=(len(lens), Hkv * G, 128)), dtype=torch.float32).to(torch.bfloat16)
    lam = torch.tensor(rng.normal(size=(len(lens), Hkv * G // 2)), dtype=torch.float32)
    return table, pool, q, lam


def widened(table, page_size, heads, wide):
    """The table, or one of such a capacity that the decode cuts the batch into ranges for all blocks
    (few keys at most: one row for each cluster)."""
    if not wide:
        return table
    width = -(-5 * 456 * 128 // (page_size * heads * len(table))) + table.shape[1]
    return np.concatenate([table, np.full((len(table), width - table.shape[1]), -1)], axis=1)


LENS = [[1], [0], [2, 0, 15], [16, 17, 31, 32, 33], [63, 64, 65, 127, 128, 129, 0, 1], [1000, 3, 511], [4097]]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("H,page_size", [(1, 16), (3, 48), (12, 64)])
def test_v1_decode(lens, H, page_size, wide):
    rng = np.random.default_rng(sum(lens) * 7 + H)
    table, pool, q, lam, w = v1_case(rng, lens, H, page_size)
    table = widened(table, page_size, H, wide)
    got = da.diffattn_decode_kv4(q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), lam.to(DEV), 0.4,
                                 norm_weight=w.to(DEV))
    within(got, *kv4.decode(q, pool, table, lens, lam.numpy(), 0.4, w, slack=SLACK, floor=FLOOR))
    for b, n in enumerate(lens):
        assert n or not got[b].any()
    da.diffattn_device_status()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("norm,scale,weight", [(False, False, False), (False, True, False), (True, False, True), (True, True, False)])
def test_v1_decode_epilogues(norm, scale, weight, wide):
    rng = np.random.default_rng(31)
    table, pool, q, lam, w = v1_case(rng, [77, 300], 2, 32)
    table = widened(table, 32, 2, wide)
    got = da.diffattn_decode_kv4(q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32([77, 300]), lam.to(DEV), 0.4,
                                 norm_weight=w.to(DEV) if weight else None, eps=1e-3, norm=norm, scale=scale)
    within(got, *kv4.decode(q, pool, table, [77, 300], lam.numpy(), 0.4, w if weight else None, 1e-3, norm, scale, slack=SLACK, floor=FLOOR))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("Hkv,G,page_size", [(1, 2, 16), (2, 4, 48), (3, 8, 64), (8, 8, 16)])
def test_v2_decode(lens, Hkv, G, page_size, wide):
    rng = np.random.default_rng(sum(lens) * 5 + G)
    table, pool, q, lam = v2_case(rng, lens, Hkv, G, page_size)
    table = widened(table, page_size, Hkv, wide)
    got = da.diffattn_v2_decode_kv4(q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), lam.to(DEV))
    within(got, *kv4.v2_decode(q, pool, table, lens, lam.numpy(), slack=SLACK, floor=FLOOR))
    for b, n in enumerate(lens):
        assert n or not got[b].any()
    da.diffattn_device_status()


@pytest.fixture(params=["by row", "by range"])
def wide(request):
    return request.param == "by range"


def both(rng, lens, page_size, wide, std=1.0, heads=2, spare=2, width=None):
    """The two decodes as (name, call(pool, table, lens, q) -> out, reference(...), q, pool, table)."""
    t1, p1, q1, l1, w1 = v1_case(rng, lens, heads, page_size, std, spare, width)
    t2, p2, q2, l2 = v2_case(rng, lens, heads, 8, page_size, std, spare, width)
    t1, t2 = widened(t1, page_size, heads, wide), widened(t2, page_size, heads, wide)
    D1, D2, W1 = l1.to(DEV), l2.to(DEV), w1.to(DEV)
    dev = lambda x: x.to(DEV) if isinstance(x, torch.Tensor) else torch.tensor(x).to(DEV)  # noqa: E731
    v1 = lambda q, pool, table, lens, **k: da.diffattn_decode_kv4(dev(q), dev(pool), dev32(table), dev32(lens), D1, 0.4, norm_weight=W1, **k)  # noqa: E731
    v2 = lambda q, pool, table, lens, **k: da.diffattn_v2_decode_kv4(dev(q), dev(pool), dev32(table), dev32(lens), D2, **k)  # noqa: E731
    r1 = lambda q, pool, table, lens, **k: kv4.decode(q, pool, table, lens, l1.numpy(), 0.4, w1, slack=SLACK, floor=FLOOR, **k)  # noqa: E731
    r2 = lambda q, pool, table, lens, **k: kv4.v2_decode(q, pool, table, lens, l2.numpy(), slack=SLACK, floor=FLOOR, **k)  # noqa: E731
    return [("v1", v1, r1, q1, p1, t1), ("v2", v2, r2, q2, p2, t2)]


def test_decode_many_sequences(wide):
    """More (sequence, head) pairs than blocks at once, of every length up to 40, a few of 900."""
    lens = [900 if i % 97 == 5 else i % 41 for i in range(700)]
    for name, call, want, q, pool, table in both(np.random.default_rng(41), lens, 16, wide, heads=2):
        within(call(q, pool, table, lens), *want(q, pool, table, lens))


def test_decode_more_rows_than_blocks_of_mixed_lengths():
    """480 (sequence, head) rows of up to 900 keys: ranges that hold several rows and rows that lie in
    several ranges, merged by a block for each range."""
    lens = [(i * 97) % 900 for i in range(60)]
    for name, call, want, q, pool, table in both(np.random.default_rng(131), lens, 16, False, heads=8):
        within(call(q, pool, table, lens), *want(q, pool, table, lens))


def test_decode_long_sequence_beside_short_ones(wide):
    lens = [3, 20011, 0, 130]
    for name, call, want, q, pool, table in both(np.random.default_rng(43), lens, 64, wide, heads=1):
        within(call(q, pool, table, lens), *want(q, pool, table, lens))


def test_decode_exponents(wide):
    lens = [100, 37]
    for name, call, want, q, pool, table in both(np.random.default_rng(47), lens, 16, wide):
        within(call(q, pool, table, lens, k_exp=1, v_exp=-7), *want(q, pool, table, lens, k_exp=1, v_exp=-7))


@pytest.mark.parametrize("at", [0, 17, 900, 1499])
def test_decode_one_key_far_above_the_rest(at, wide):
    """A key whose score is 30 to 100 above the others takes all of the weight, wherever it stands
    (first, where it sets the reference of all others, or last, where all before it has to shrink)."""
    lens = [1500]
    for name, call, want, q, pool, table in both(np.random.default_rng(53), lens, 16, wide, heads=1):
        k, v = kv4.sequence_rows(pool, 2 if name == "v1" else 1, table, 0, 1500)
        row = np.sign(to64(q)[0, 0]) * 6.0
        kp = 2 if name == "v1" else 1
        page, off = table[0, at // 16], at % 16
        kv4.write_row(pool[page, 0, 0], kp, row[:128 * kp], v[at, 0], off)
        within(call(q, pool, table, lens), *want(q, pool, table, lens))


def test_decode_a_first_key_that_outweighs_each_but_not_all(wide):
    """A first key some 13 above the rest in the exponent: each of the others has 2^-19 of its
    weight, and 9000 of them together still count."""
    lens = [9000]
    for name, call, want, q, pool, table in both(np.random.default_rng(59), lens, 64, wide, heads=1, std=0.02):
        kp = 2 if name == "v1" else 1
        q = torch.ones_like(q) * 0.5
        row = np.full(128 * kp, 2.25)  # 128 * 0.5 * 2.25 / sqrt(128) = 12.7
        v0 = np.full(128 * kp, 3.0)
        kv4.write_row(pool[table[0, 0], 0, 0], kp, row, v0, 0)
        within(call(q, pool, table, lens), *want(q, pool, table, lens))


def test_decode_small_and_large_queries(wide):
    """Queries far from unit size: tiny ones (uniform weights), and ones whose largest channel is
    2^40 times the others (which then count for nothing), with keys of matching exponents."""
    lens = [333]
    for name, call, want, q, pool, table in both(np.random.default_rng(61), lens, 32, wide):
        tiny = (q.float() * 2.0 ** -60).to(torch.bfloat16)
        within(call(tiny, pool, table, lens), *want(tiny, pool, table, lens))
        big = (q.float() * 2.0 ** 60).to(torch.bfloat16)
        within(call(big, pool, table, lens, k_exp=-60), *want(big, pool, table, lens, k_exp=-60))
        mixed = q.clone()
        mixed[..., 1:] = (mixed[..., 1:].float() * 2.0 ** -40).to(torch.bfloat16)
        within(call(mixed, pool, table, lens), *want(mixed, pool, table, lens))
        zero = torch.zeros_like(q)
        within(call(zero, pool, table, lens), *want(zero, pool, table, lens))


def test_decode_slots_past_the_end_may_hold_anything(wide):
    """NaN scales, any codes in the rest of the last record, of the last page, and in every page of
    no sequence; table entries past a sequence's pages are never used."""
    lens = [1, 30, 64, 75]
    for name, call, want, q, pool, table in both(np.random.default_rng(67), lens, 32, wide, width=9):
        clean = call(q, pool, table, lens)
        within(clean, *want(q, pool, table, lens))
        kp, page_size = (2 if name == "v1" else 1), 32
        live = np.zeros((pool.shape[0], page_size), dtype=bool)
        for b, n in enumerate(lens):
            for j in range(n):
                live[table[b, j // page_size], j % page_size] = True
        foul = np.full_like(pool, 0xFF)
        for page, off in zip(*np.nonzero(live)):
            for h in range(pool.shape[1]):
                i = off % 16
                for p in range(2 * kp):
                    base, src, dst = p * 1152, pool[page, h, off // 16], foul[page, h, off // 16]
                    for b8 in range(8):
                        a = base + (kv4.k_code_at(i, b8 // 2) + 8 * (b8 % 2) if p < kp else kv4.v_code_at(i, b8))
                        s = base + (kv4.k_scale_at(i, b8 // 2, b8 % 2) if p < kp else kv4.v_scale_at(i, b8))
                        dst[a:a + 8], dst[s] = src[a:a + 8], src[s]
        wild = np.where(table < 0, 2 ** 31 - 1, table)
        assert torch.equal(call(q, foul, wild, lens), clean)
        da.diffattn_device_status()


def test_decode_nan_key_reaches_its_head_alone(wide):
    lens = [50, 50]
    for name, call, want, q, pool, table in both(np.random.default_rng(71), lens, 16, wide):
        clean = call(q, pool, table, lens)
        kp = 2 if name == "v1" else 1
        for plane in (0, 2 * kp - 1):  # a K plane and a V plane
            bad = pool.copy()
            bad[table[1, 2], 1, 0, plane * 1152 + 1024 + 5] = 0x7F
            got = call(q, bad, table, lens)
            per = got.shape[1] // 2
            assert torch.isnan(got[1, per:]).any()
            assert torch.equal(got[0], clean[0]) and torch.equal(got[1, :per], clean[1, :per])


def test_decode_nan_and_inf_queries(wide):
    lens = [40, 40]
    for name, call, want, q, pool, table in both(np.random.default_rng(73), lens, 16, wide):
        clean = call(q, pool, table, lens)
        for x in (float("nan"), float("inf")):
            bad = q.clone()
            bad[1, 0, 5] = x
            got = call(bad, pool, table, lens)
            assert not torch.isfinite(got[1, 0]).all()
            assert torch.equal(got[0], clean[0]) and torch.equal(got[1, -1], clean[1, -1])


def test_decode_lengths_out_of_range_are_clamped(wide):
    lens = [64, 64, 5]
    for name, call, want, q, pool, table in both(np.random.default_rng(79), lens, 32, wide):
        table = np.maximum(table, 0)  # every entry of the capacity may be used
        a = call(q, pool, table, [table.shape[1] * 32, 0, 5])
        b = call(q, pool, table, [10 ** 9, -4, 5])
        assert torch.equal(a, b)


def test_decode_bad_page_reads_page_0_and_is_reported(wide):
    lens = [40, 20]
    for name, call, want, q, pool, table in both(np.random.default_rng(83), lens, 16, wide):
        for bad in (-1, pool.shape[0], 2 ** 31 - 1):
            t, z = table.copy(), table.copy()
            t[0, 1], z[0, 1] = bad, 0
            got = call(q, pool, t, lens)
            with pytest.raises(da.DiffAttnError) as e:
                da.diffattn_device_status()
            assert e.value.status == -9
            assert torch.equal(got, call(q, pool, z, lens))
            da.diffattn_device_status()


def test_decode_repeats_bit_for_bit_whatever_the_workspace_holds(wide):
    lens = [5000, 1, 777, 0, 2048]
    for name, call, want, q, pool, table in both(np.random.default_rng(89), lens, 64, wide):
        n = (da.diffattn_decode_kv4_workspace_size(5, 2) if name == "v1" else da.diffattn_v2_decode_kv4_workspace_size(5, 16, 2))
        first = call(q, pool, table, lens)
        for fill in (0x00, 0xFF, 0x7F):
            ws = torch.full((n + 512,), fill, dtype=torch.uint8, device=DEV)
            assert torch.equal(call(q, pool, table, lens, workspace=ws[:n]), first)
            torch.cuda.synchronize()
            assert bool((ws[n:] == fill).all())


def test_decode_on_another_stream(wide):
    lens = [300, 41]
    for name, call, want, q, pool, table in both(np.random.default_rng(97), lens, 16, wide):
        clean = call(q, pool, table, lens)
        Q, P, T, S = q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens)
        fn = (lambda **k: call(Q, P, table, lens, **k))
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            got = call(Q, P, table, lens)
        torch.cuda.current_stream().wait_stream(other)
        assert torch.equal(got, clean)
        for stream in (other, other.cuda_stream):
            got = fn(stream=stream)
            other.synchronize()
            assert torch.equal(got, clean)


def decode_pair(name, q, pool, table, lens, lam, out, ws, w=None):
    if name == "v1":
        da.diffattn_decode_kv4(q, pool, table, lens, lam, 0.4, norm_weight=w, workspace=ws, out=out)
    else:
        da.diffattn_v2_decode_kv4(q, pool, table, lens, lam, workspace=ws, out=out)


@pytest.mark.parametrize("name", ["v1", "v2"])
def test_decode_captured_graphs_follow_their_inputs(name, wide):
    """A captured decode replays on new queries, lengths, tables and rows in the captured buffers."""
    rng = np.random.default_rng(101)
    lens = [200, 64, 1]
    if name == "v1":
        table, pool, q, lam, w = v1_case(rng, lens, 2, 16, width=20)
        n, shape = da.diffattn_decode_kv4_workspace_size(3, 2), (3, 2, 256)
    else:
        (table, pool, q, lam), w = v2_case(rng, lens, 2, 4, 16, width=20), None
        n, shape = da.diffattn_v2_decode_kv4_workspace_size(3, 8, 2), (3, 4, 128)
    table = widened(table, 16, 2, wide)
    Q, P, T, S, L = q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), lam.to(DEV)
    W = w.to(DEV) if w is not None else None
    out, ws = torch.zeros(shape, dtype=torch.bfloat16, device=DEV), torch.empty(n, dtype=torch.uint8, device=DEV)
    decode_pair(name, Q, P, T, S, L, out, ws, W)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode_pair(name, Q, P, T, S, L, out, ws, W)
    want = (lambda q, t, s: kv4.decode(q, pool, t, s, lam.numpy(), 0.4, w, slack=SLACK, floor=FLOOR) if name == "v1"
            else kv4.v2_decode(q, pool, t, s, lam.numpy(), slack=SLACK, floor=FLOOR))
    for step in range(3):
        q2 = torch.tensor(rng.normal(size=tuple(q.shape)), dtype=torch.float32).to(torch.bfloat16)
        s2 = [[200, 0, 1], [17, 64, 1], [1, 1, 0]][step]
        t2 = table.copy()
        t2[0, 0], t2[1, 0] = table[1, 0], table[0, 0]
        Q.copy_(q2), S.copy_(dev32(s2)), T.copy_(dev32(t2))
        ws.fill_(0xEE)
        graph.replay()
        torch.cuda.synchronize()
        within(out, *want(q2, t2, s2))


def test_two_decodes_at_once(wide):
    """Two streams, a workspace each: neither disturbs the other."""
    rng = np.random.default_rng(103)
    lens = [3000, 1, 900]
    cases = both(rng, lens, 32, wide)
    want = [c[1](c[3], c[4], c[5], lens) for c in cases]
    P = [torch.tensor(c[4]).to(DEV) for c in cases]
    Q = [c[3].to(DEV) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(10):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i].append(c[1](Q[i], P[i], c[5], lens))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


def test_decode_guards(wide):
    lens = [90, 33, 0]
    for name, call, want, q, pool, table in both(np.random.default_rng(107), lens, 16, wide):
        clean = call(q, pool, table, lens)
        buf = torch.full((clean.numel() + 8192,), 7.0, dtype=torch.bfloat16, device=DEV)
        out = buf[4096:4096 + clean.numel()].view(clean.shape)
        call(q, pool, table, lens, out=out)
        assert torch.equal(out, clean) and bool((buf[:4096] == 7).all()) and bool((buf[4096 + clean.numel():] == 7).all())


def test_decode_pool_offsets_past_32_bits():
    """A pool of more than 4 GB: the last page is where it should be."""
    page_size, H = 1024, 12
    rec = (page_size // 16) * 4608 * H
    pages = (1 << 32) // rec + 3
    pool = torch.zeros((pages, H, page_size // 16, 4608), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(109)
    rows = torch.tensor(rng.normal(size=(2, 40, H, 256)), dtype=torch.float32).to(torch.bfloat16).to(DEV)
    first = (pages - 1) * page_size + 100
    da.diffattn_kv4_append(rows[0], rows[1], torch.arange(first, first + 40, dtype=torch.int32, device=DEV), pool)
    k, v = da.diffattn_kv4_gather(pool, dev32([[pages - 1]]), dev32([0, 40]), 40, 256, 256, starts=dev32([100]))
    for got, x in ((k, rows[0]), (v, rows[1])):
        assert np.array_equal(to64(got), kv4.values(*kv4.quantize_blocks(to64(x))))
    q = torch.tensor(rng.normal(size=(1, H, 256)), dtype=torch.float32).to(torch.bfloat16)
    lam = torch.full((H,), 0.3)
    got = da.diffattn_decode_kv4(q.to(DEV), pool, dev32([[pages - 1]]), dev32([140]), lam.to(DEV), 0.2)
    small = pool[-1:].cpu().numpy()
    within(got, *kv4.decode(q, small, [[0]], [140], lam.numpy(), 0.2, slack=SLACK, floor=FLOOR))


def test_v2_decode_agrees_with_the_bf16_decode_on_the_same_values():
    """The framework's decode over bf16 pages, given the values the 4-bit pool stands for."""
    rng = np.random.default_rng(113)
    lens, ps = [300, 65], 64
    table, pool, q, lam = v2_case(rng, lens, 2, 8, ps)
    got = da.diffattn_v2_decode_kv4(q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), lam.to(DEV))
    pages = pool.shape[0]
    k, v = kv4.read_rows(pool, 1, np.repeat(np.arange(pages), ps), np.tile(np.arange(ps), pages))
    as_pool = lambda x: torch.tensor(x.reshape(pages, ps, 2, 128)).to(torch.bfloat16).to(DEV)  # noqa: E731
    wide = da.diffattn_v2_decode_paged(q.to(DEV), as_pool(k), as_pool(v), dev32(np.maximum(table, 0)), dev32(lens), lam.to(DEV))
    assert_bf16(got, wide)


# ---- together ---------------------------------------------------------------------------------

@pytest.mark.parametrize("form", ["v1", "v2"])
def test_serving_steps(form):
    """Requests that come and go over a small pool: plan, append, then prompts through the read-out
    and the packed prefill, single tokens through the decode; each step's outputs against the
    reference over the values that were cached so far (kept here as plain rows), and pages of
    ended requests used again."""
    rng = np.random.default_rng(127)
    B, H, ps, num_pages, width = 3, 2, 128, 14, 8
    kp = 2 if form == "v1" else 1
    w, Hq = 128 * kp, H if form == "v1" else 4 * H
    pool = da.diffattn_kv4_pool(num_pages, ps, H, w, w)
    state = {"seqlens": dev32([0] * B), "ring_state": dev32([0, num_pages])}
    table, ring = dev32(np.full((B, width), -1)), dev32(rng.permutation(num_pages))
    lam = torch.tensor(rng.uniform(0.2, 0.8, H), dtype=torch.float32)
    cached = [(np.zeros((0, H, w)), np.zeros((0, H, w))) for _ in range(B)]
    steps = [[150, 0, 3], [1, 260, 1], [1, 1, -1], [130, 1, 500], [-1, 1, 1], [700, -1, 1], [1, 90, 1]]
    for new in steps:
        total = sum(max(n, 0) for n in new)
        plan = da.diffattn_paged_plan(state["seqlens"], dev32(new), table, ring, state["ring_state"], ps, total)
        state = plan
        rows = torch.tensor(rng.normal(size=(2, total, H, w)), dtype=torch.float32).to(torch.bfloat16)
        q = torch.tensor(rng.normal(size=(total, Hq, w)) * 0.5, dtype=torch.float32).to(torch.bfloat16)
        lg = torch.tensor(rng.normal(size=(total, Hq // 2)), dtype=torch.float32)
        da.diffattn_kv4_append(rows[0].to(DEV), rows[1].to(DEV), plan["slot_map"], pool)
        at = 0
        for b, n in enumerate(new):
            if n < 0:
                cached[b] = tuple(x[:0] for x in cached[b])
            if n > 0:
                piece = [kv4.values(*kv4.quantize_blocks(to64(r[at:at + n]))) for r in rows]
                cached[b] = tuple(np.concatenate([x, y]) for x, y in zip(cached[b], piece))
                at += n
        cu_q = np.concatenate([[0], np.cumsum(np.maximum(new, 0))])
        lens_k = [len(c[0]) if n > 0 else 0 for c, n in zip(cached, new)]
        total_k = sum(lens_k)
        assert plan["cu_seqlens_k"].tolist() == [0, *np.cumsum(lens_k)]
        k, v = da.diffattn_kv4_gather(pool, table, plan["cu_seqlens_k"], total_k, w, w)
        if form == "v1":
            got = da.diffattn_fwd_varlen_qk(q.to(DEV), k, v, plan["cu_seqlens_q"], plan["cu_seqlens_k"], lam.to(DEV), 0.3)
        else:
            got = da.diffattn_v2_fwd_varlen(q.to(DEV), k, v, lg.to(DEV), plan["cu_seqlens_q"], plan["cu_seqlens_k"])
        want_k = np.concatenate([c[0] for c, n in zip(cached, new) if n > 0])
        want_v = np.concatenate([c[1] for c, n in zip(cached, new) if n > 0])
        assert np.array_equal(to64(k), want_k) and np.array_equal(to64(v), want_v)
        cu_k = np.concatenate([[0], np.cumsum(lens_k)])
        if form == "v1":
            want = ref.diffattn_fwd_varlen_qk(q, want_k, want_v, cu_q, cu_k, lam.numpy(), 0.3)
        else:
            want = ref.diffattn_v2_fwd_varlen(q, want_k, want_v, lg, cu_q, cu_k)
        assert_bf16(got, want)
        # the last token of each request, through the decode over the same pages
        last = [cu_q[b + 1] - 1 if n > 0 else 0 for b, n in enumerate(new)]
        if form == "v1":
            one = da.diffattn_decode_kv4(q[last].to(DEV), pool, table, plan["seqlens"], lam.to(DEV), 0.3)
        else:
            one = da.diffattn_v2_decode_kv4(q[last].to(DEV), pool, table, plan["seqlens"], lg[last].to(DEV))
        for b, n in enumerate(new):
            if n > 0:
                assert_bf16(one[b:b + 1], want[last[b]:last[b] + 1])
            elif len(cached[b][0]) == 0:
                assert not one[b].any()
    da.diffattn_device_status()


@pytest.mark.parametrize("form", ["v1", "v2"])
def test_captured_decode_step_replays(form):
    """A whole decoding step (plan in place, append, decode) captured once and replayed: every replay
    goes on from the lengths, tables and ring that the last one left; requests grow over page ends, and
    an ended one's pages are taken again."""
    rng = np.random.default_rng(137)
    B, H, ps, num_pages, width = 3, 2, 16, 12, 8
    kp = 2 if form == "v1" else 1
    w, Hq = 128 * kp, H if form == "v1" else 4 * H
    pool = da.diffattn_kv4_pool(num_pages, ps, H, w, w)
    lens, new, state = dev32([14, 31, 0]), dev32([1, 1, 1]), dev32([0, num_pages])
    table, ring = dev32(np.full((B, width), -1)), dev32(rng.permutation(num_pages))
    lam = torch.tensor(rng.uniform(0.2, 0.8, H), dtype=torch.float32)
    lg = torch.tensor(rng.normal(size=(B, Hq // 2)), dtype=torch.float32)
    L, LG = lam.to(DEV), lg.to(DEV)
    # the first rows, by a step of their own
    first = [14, 31, 0]
    out = da.diffattn_paged_plan(dev32([0, 0, 0]), dev32(first), table, ring, state, ps, 45)
    rows = torch.tensor(rng.normal(size=(2, 45, H, w)), dtype=torch.float32).to(torch.bfloat16)
    da.diffattn_kv4_append(rows[0].to(DEV), rows[1].to(DEV), out["slot_map"], pool)
    state.copy_(out["ring_state"])
    at, cached = 0, []
    for n in first:
        cached.append([kv4.values(*kv4.quantize_blocks(to64(r[at:at + n]))) for r in rows])
        at += n
    # the step, in place; rows of requests without a new token are padding
    step = {"seqlens": lens, "ring_state": state}
    for name, n in (("cu_seqlens_q", B + 1), ("cu_seqlens_k", B + 1), ("slot_map", B), ("positions", B)):
        step[name] = torch.zeros(n, dtype=torch.int32, device=DEV)
    k, v = (torch.zeros((B, H, w), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q = torch.zeros((B, Hq, w), dtype=torch.bfloat16, device=DEV)

    def run():
        da.diffattn_paged_plan(lens, new, table, ring, state, ps, B, out=step)
        da.diffattn_kv4_append(k, v, step["slot_map"], pool)
        if form == "v1":
            return da.diffattn_decode_kv4(q, pool, table, lens, L, 0.3)
        return da.diffattn_v2_decode_kv4(q, pool, table, lens, LG)

    keep = [t.clone() for t in (lens, state, table, ring, pool)]
    run()  # (once outside, then everything as it was)
    for t, was in zip((lens, state, table, ring, pool), keep):
        t.copy_(was)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i in range(24):
        n = [1, -1 if i == 9 else 1 if i < 9 or i > 12 else 0, 1 if i % 3 else 0]
        rows = torch.tensor(rng.normal(size=(2, B, H, w)), dtype=torch.float32).to(torch.bfloat16)
        qs = torch.tensor(rng.normal(size=(B, Hq, w)), dtype=torch.float32).to(torch.bfloat16)
        order = [b for b in range(B) if n[b] > 0]
        for x, r in ((k, rows[0]), (v, rows[1])):
            x[:len(order)].copy_(r[order])
        q.copy_(qs), new.copy_(dev32(n))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            if n[b] < 0:
                cached[b] = [x[:0] for x in cached[b]]
            if n[b] > 0:
                cached[b] = [np.concatenate([x, kv4.values(*kv4.quantize_blocks(to64(r[b:b + 1])))]) for x, r in zip(cached[b], rows)]
        assert lens.tolist() == [len(c[0]) for c in cached]
        for b in range(B):
            N = len(cached[b][0])
            if N == 0:
                assert not got[b].any()
                continue
            kc, vc = (x[None] for x in cached[b])
            if form == "v1":
                want = ref.diffattn_decode(qs[b:b + 1], kc, vc, [N], lam.numpy(), 0.3)
            else:
                want = ref.diffattn_v2_decode(qs[b:b + 1], kc, vc, [N], lg[b:b + 1])
            assert_bf16(got[b:b + 1], want)
    da.diffattn_device_status()


def test_rows_and_plan_on_another_stream():
    """Plan, append and gather on a stream of their own, given by the caller."""
    rng = np.random.default_rng(139)
    other = torch.cuda.Stream()
    s, n, table, ring, state, total = random_step(rng, 40, 16, 6, 3, 30)
    want = kv4.paged_plan(s, n, table, ring, state, 16, total)
    T, R = dev32(table), dev32(ring)
    rows = random_rows(rng, (total, 2, 128)).to(DEV)
    pool = torch.zeros((len(ring), 2, 1, 2304), dtype=torch.uint8, device=DEV)
    S, N, St = dev32(s), dev32(n), dev32(state)
    torch.cuda.synchronize()
    p = da.diffattn_paged_plan(S, N, T, R, St, 16, total, stream=other)
    da.diffattn_kv4_append(rows, rows, p["slot_map"], pool, stream=other)
    new = torch.tensor(np.maximum(n, 0), dtype=torch.int32)
    k, v = da.diffattn_kv4_gather(pool, T, p["cu_seqlens_q"], total, 128, 128, starts=S, stream=other.cuda_stream)
    other.synchronize()
    for name in ("slot_map", "seqlens", "cu_seqlens_q"):
        assert np.array_equal(p[name].cpu().numpy(), want[name]), name
    assert int(new.sum()) == total
    x = kv4.values(*kv4.quantize_blocks(to64(rows)))
    assert np.array_equal(to64(k), x) and np.array_equal(to64(v), x)
    da.diffattn_device_status(other)


def test_gather_and_append_of_many_sequences_and_heads():
    """Sizes at which a warp of the read-out takes several heads, with odd head counts and ragged rows."""
    rng = np.random.default_rng(149)
    for H, lens, ps in ((13, [(i * 53) % 700 for i in range(40)], 32), (3, [5000, 1, 8191, 0, 77] * 4, 80)):
        table, pages = random_table(rng, lens, ps)
        total = sum(lens)
        cu = np.concatenate([[0], np.cumsum(lens)])
        k, v = (torch.randn((total, H, 128), device=DEV).to(torch.bfloat16) for _ in range(2))
        pos = np.concatenate([np.arange(n) for n in lens])
        seq = np.repeat(np.arange(len(lens)), lens)
        slots = table[seq, pos // ps] * ps + pos % ps
        pool = torch.zeros((pages, H, ps // 16, 2304), dtype=torch.uint8, device=DEV)
        da.diffattn_kv4_append(k, v, dev32(slots), pool)
        got = da.diffattn_kv4_gather(pool, dev32(table), dev32(cu), total, 128, 128)
        for x, g in zip((k, v), got):
            assert np.array_equal(to64(g), kv4.values(*kv4.quantize_blocks(to64(x))))
    da.diffattn_device_status()


def test_binding_names_the_operand_that_does_not_fit():
    """Of a fitting call, each operand in turn with another type, a size too many, strides of its own or
    on the host: a ValueError that names it, or the shapes that go together."""
    z = lambda shape, dtype=torch.int32: torch.zeros(shape, dtype=dtype, device=DEV)  # noqa: E731
    bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
    calls = {
        "plan": (lambda **o: da.diffattn_paged_plan(**o, page_size=16, total_max=4),
                 dict(seqlens=z(3), new_tokens=z(3), block_table=z((3, 5)), free_ring=z(9), ring_state=z(2))),
        "append": (da.diffattn_kv4_append,
                   dict(k=z((4, 2, 128), bf16), v=z((4, 2, 128), bf16), slot_map=z(4), pool=z((9, 2, 1, 2304), u8))),
        "gather": (lambda **o: da.diffattn_kv4_gather(**o, total=4, kw=128, vw=128),
                   dict(pool=z((9, 2, 1, 2304), u8), block_table=z((3, 5)), cu_seqlens=z(4), starts=z(3))),
        "v1": (da.diffattn_decode_kv4,
               dict(q=z((3, 2, 256), bf16), pool=z((9, 2, 1, 4608), u8), block_table=z((3, 5)), seqlens=z(3), lam=z(2, f32),
                    norm_weight=z(256, f32), out=z((3, 2, 256), bf16))),
        "v2": (da.diffattn_v2_decode_kv4,
               dict(q=z((3, 4, 128), bf16), pool=z((9, 2, 1, 2304), u8), block_table=z((3, 5)), seqlens=z(3),
                    lam_logit=z((3, 2), f32), out=z((3, 2, 128), bf16))),
    }
    for name, (call, good) in calls.items():
        call(**good)
        for key, t in good.items():
            longer = torch.cat([t, t[:1]])
            spread = torch.stack([t, t], -1)[..., 0]
            for bad in (t.double(), longer, spread, t.cpu(), None):
                if bad is None and key in ("starts", "norm_weight", "out"):
                    continue
                if bad is longer and (name, key) in (("plan", "free_ring"), ("append", "pool"), ("gather", "pool"), ("v1", "pool"), ("v2", "pool")):
                    continue  # one more page
                if bad is spread and (name, key) in (("append", "k"), ("append", "v")):
                    with pytest.raises(ValueError, match="contiguous"):
                        call(**{**good, key: bad})
                    continue
                with pytest.raises(ValueError):
                    call(**{**good, key: bad})
    da.diffattn_device_status()


def unwritten(name, B, H):
    """A workspace of NaN."""
    n = (da.diffattn_decode_kv4_workspace_size(B, H) if name == "v1" else da.diffattn_v2_decode_kv4_workspace_size(B, 8 * H, H))
    return torch.full((n,), 255, dtype=torch.uint8, device=DEV)


@pytest.mark.parametrize("seed", range(16))
def test_decode_random_batches(seed):
    """Batches of few long, many short and mixed sequences, cut into ranges: every piece that is read was
    written in the same call."""
    rng = np.random.default_rng(500 + seed)
    B, top, heads = int(rng.choice([1, 2, 5, 40, 300, 600])), int(rng.choice([3, 40, 300, 3000])), int(rng.integers(1, 4))
    top = min(top, 120000 // (B * heads))
    lens = [int(n) if rng.random() < 0.9 else 0 for n in np.exp(rng.uniform(0, np.log(top + 1), B))]
    lens[int(rng.integers(B))] = top
    for name, call, want, q, pool, table in both(rng, lens, 16, True, heads=heads):
        within(call(q, pool, table, lens, workspace=unwritten(name, B, heads)), *want(q, pool, table, lens))
    da.diffattn_device_status()


def test_decode_of_the_largest_batch():
    """8192 sequences, most of a few keys and some of none, a few of 700 at the ends and in the middle."""
    lens = [700 if i in (0, 4000, 4001, 8191) else i % 7 for i in range(8192)]
    for name, call, want, q, pool, table in both(np.random.default_rng(8), lens, 16, False, heads=1):
        within(call(q, pool, table, lens, workspace=unwritten(name, 8192, 1)), *want(q, pool, table, lens))
    da.diffattn_device_status()


def test_decode_one_row_in_as_many_pieces_as_there_are_blocks():
    """One (sequence, head) over every block, and two of them."""
    for lens in ([70000], [61000, 52001]):
        for name, call, want, q, pool, table in both(np.random.default_rng(9), lens, 64, True, heads=1):
            within(call(q, pool, table, lens, workspace=unwritten(name, len(lens), 1)), *want(q, pool, table, lens))


def test_captured_behind_two_streams_that_join(wide):
    """A graph in which rows are appended on one stream while another copies the lengths and forms the
    lambdas: decodes behind the join, replayed with other inputs."""
    lens = [900, 33, 0, 417]
    for name, call, want, q, pool, table in both(np.random.default_rng(71), lens, 32, wide):
        H, w = pool.shape[1], pool.shape[3] // 18
        Q, P, T, given, seq = q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), dev32([0] * 4)
        rows = torch.zeros((1, H, w), dtype=torch.bfloat16, device=DEV)
        slot = dev32([int(table[3][0]) * 32])
        raw = torch.full((H,) if name == "v1" else (4, 4 * H), 0.25, device=DEV)

        def step(side):
            main = torch.cuda.current_stream()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                lam = raw * 2.0
                seq.copy_(given)
            da.diffattn_kv4_append(rows, rows, slot, P)
            main.wait_stream(side)
            if name == "v1":
                return da.diffattn_decode_kv4(Q, P, T, seq, lam, 0.4)
            return da.diffattn_v2_decode_kv4(Q, P, T, seq, lam)

        side = torch.cuda.Stream()
        step(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(side)
        for n, scale in (([5, 33, 0, 400], 0.1), ([900, 0, 0, 417], 0.4)):  # (none past its pages)
            given.copy_(dev32(n))
            raw.fill_(scale)
            rows.normal_()
            for _ in range(3):
                g.replay()
            got = out.clone()
            assert torch.equal(got, step(torch.cuda.Stream()))
    da.diffattn_device_status()
