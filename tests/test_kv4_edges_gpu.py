"""The 4-bit cache's calls at the far ends of what their header allows: exponents, weights that are not
finite, streams of other libraries, joins of every piece. Bounds as in test_kv4_gpu.py."""
import ctypes
import gc

import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from oracle import kv4_ref as kv4
from tests import kv4_pieces as pieces
from tests.test_kv4_gpu import (DEV, FLOOR, SLACK, both, dev32, expected_pool, random_rows, random_table, to64, v1_case, widened,
                                within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.lib()
    yield
    da.diffattn_device_status()


# how a V1 row's end is reached: (lens, heads, by ranges)
ROW_ENDS = {"cluster": ([100, 37], 2, False), "whole": ([100] * 350, 2, True), "pieces of few rows": ([3000, 900], 2, True),
            "pieces of many rows": ([900] * 80, 4, True)}


@pytest.mark.parametrize("end", list(ROW_ENDS))
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("v_exp,eps", [(64, 1e-5), (48, 1e-5), (-64, 1e-5), (-64, 1e-30), (33, 1e-12)])
def test_v1_decode_norm_at_far_exponents(v_exp, eps, norm, end):
    """The norm's sum of squares stays in fp32's range whatever power of two the values carry."""
    lens, H, wide = ROW_ENDS[end]
    table, pool, q, lam, w = v1_case(np.random.default_rng(211), lens, H, 16)
    table = widened(table, 16, H, wide)
    got = da.diffattn_decode_kv4(q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), lam.to(DEV), 0.4,
                                 norm_weight=w.to(DEV), eps=eps, norm=norm, v_exp=v_exp)
    within(got, *kv4.decode(q, pool, table, lens, lam.numpy(), 0.4, w, eps, norm, v_exp=v_exp, slack=SLACK, floor=FLOOR))
    da.diffattn_device_status()


@pytest.mark.parametrize("wide", [False, True])
def test_v1_decode_of_no_keys_gives_zeros_whatever_the_norm_holds(wide):
    """An empty place in the batch is zeros also where the norm's weight is not finite or the scale is."""
    lens = [0, 70, 0]
    table, pool, q, lam, w = v1_case(np.random.default_rng(223), lens, 2, 16)
    table = widened(table, 16, 2, wide)
    w[3], w[200] = float("nan"), float("inf")
    for lambda_init in (0.4, float("nan")):
        got = da.diffattn_decode_kv4(q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), lam.to(DEV), lambda_init,
                                     norm_weight=w.to(DEV))
        assert not got[0].any() and not got[2].any()
        assert torch.isnan(got[1, :, 3]).all()
    da.diffattn_device_status()


class ForeignStream:
    """A stream that torch did not make."""

    def __init__(self):
        self.cudart = torch.cuda.cudart()
        handle = ctypes.c_uint64(0)
        assert int(self.cudart.cudaStreamCreate(ctypes.addressof(handle))) == 0
        self.handle = handle.value

    def close(self):
        assert int(self.cudart.cudaStreamDestroy(self.handle)) == 0


def test_decode_keeps_nothing_for_foreign_streams():
    """A handle of another library may be destroyed and its value come back: scratch is not kept by it."""
    lens = [300, 41]
    table, pool, q, lam, w = v1_case(np.random.default_rng(227), lens, 2, 16)
    Q, P, T, S, L = q.to(DEV), torch.tensor(pool).to(DEV), dev32(widened(table, 16, 2, True)), dev32(lens), lam.to(DEV)
    want = da.diffattn_decode_kv4(Q, P, T, S, L)
    out = [torch.empty_like(want) for _ in range(12)]
    torch.cuda.synchronize()

    def use(o):
        s = ForeignStream()
        da.diffattn_decode_kv4(Q, P, T, S, L, out=o, stream=s.handle)
        with torch.cuda.stream(torch.cuda.ExternalStream(s.handle)):
            da.diffattn_decode_kv4(Q, P, T, S, L, out=o)
        return s

    open_ = [use(out[0])]
    gc.collect()
    held = torch.cuda.memory_allocated()
    open_ += [use(o) for o in out[1:]]
    assert torch.cuda.memory_allocated() <= held
    torch.cuda.synchronize()
    for s in open_:
        s.close()
    assert all(torch.equal(o, want) for o in out)
    da.diffattn_device_status()


def test_decodes_on_two_foreign_streams_do_not_share_scratch_in_time():
    lens = [5000, 41, 900]
    streams, calls = [ForeignStream(), ForeignStream()], []
    for i, s in enumerate(streams):
        table, pool, q, lam, w = v1_case(np.random.default_rng(229 + i), lens, 2, 16)
        calls.append((q.to(DEV), torch.tensor(pool).to(DEV), dev32(widened(table, 16, 2, True)), dev32(lens), lam.to(DEV)))
    want = [da.diffattn_decode_kv4(*c) for c in calls]
    out = [[torch.empty_like(want[0]) for _ in range(20)] for _ in streams]
    torch.cuda.synchronize()
    for k in range(20):
        for s, c, o in zip(streams, calls, out):
            da.diffattn_decode_kv4(*c, out=o[k], stream=s.handle)
    torch.cuda.synchronize()
    for s, o, x in zip(streams, out, want):
        s.close()
        assert all(torch.equal(y, x) for y in o)
    da.diffattn_device_status()


def test_plan_reports_what_it_is():
    """A step that does not fit is not reported as a bad page, and a bad page not as such a step."""
    def plan(s, n, table, ring, state, total_max):
        da.diffattn_paged_plan(dev32(s), dev32(n), dev32(table), dev32(ring), dev32(state), 16, total_max)
        with pytest.raises(da.DiffAttnError) as e:
            da.diffattn_device_status()
        assert e.value.status == -9
        return str(e.value)

    fit = "does not fit"
    assert fit in plan([16], [1], [[0, -1]], [1, 2], [0, 0], 1)      # no free page
    assert fit in plan([0], [3], [[-1, -1]], [1, 2], [0, 2], 2)      # more tokens than total_max
    assert fit in plan([33], [0], [[0, -1]], [1, 2], [0, 1], 2)      # a length past the table
    bad = plan([16], [1], [[0, -1]], [7, 2], [0, 2], 1)              # page 7 of 2
    assert fit not in bad and "page" in bad


@pytest.mark.parametrize("wide", [False, True])
def test_decode_of_queries_whose_loud_channel_meets_zero_keys(wide):
    """The scores come from the other channels alone: exact down to 2^-31 of the loud one (here 2^40 at
    its side, by exponents), and zeros from 2^-40 on."""
    lens = [333]
    for name, call, want, q, pool, table in both(np.random.default_rng(239), lens, 32, wide):
        kp, pool = (2 if name == "v1" else 1), pool.copy()
        for i in range(16):  # channel 16 of every K plane: code 0 in the low nibble of its block's first byte
            for p in range(kp):
                pool[..., p * kv4.PLANE + kv4.k_code_at(i, 0) + 8] &= 0xF0
        k = kv4.sequence_rows(pool, kp, table, 0, 333)[0]
        assert not k[..., 16::128].any() and k[..., 17::128].any()

        def loud(x, exponent):
            """Channels of random sign and 8 significant bits, all of one exponent, beside the loud one."""
            y = torch.sign(x.float()) * (1.0 + torch.frac(x.float().abs() * 1000.0 / 128.0).mul(128).floor() / 128.0)
            y = y * 2.0 ** exponent
            y[..., 16::128] = 2.0 ** 40
            return y.to(torch.bfloat16)

        near = loud(q, 40 - 31)
        within(call(near, pool, table, lens, k_exp=-9), *want(near, pool, table, lens, k_exp=-9))
        far, none = loud(q, 40 - 41), torch.zeros_like(q)
        none[..., 16::128] = 2.0 ** 40
        assert torch.equal(call(far, pool, table, lens), call(none, pool, table, lens))
        within(call(far, pool, table, lens), *want(none, pool, table, lens))
    da.diffattn_device_status()


def test_plan_of_more_keys_than_32_bits_count_does_not_fit():
    """Two requests of 2^30 keys: their sum has no place in cu_seqlens_k; with one key less it has."""
    page, cap = 1 << 28, 1 << 30
    for last, fits in ((cap - 2, True), (cap - 1, False)):
        s = [cap - 1, last]
        p = da.diffattn_paged_plan(dev32(s), dev32([1, 1]), dev32([[0, 1, 2, 3]] * 2), dev32([4, 5, 6, 0, 1, 2, 3]), dev32([0, 3]), page, 4)
        if fits:
            da.diffattn_device_status()
            assert p["seqlens"].tolist() == [cap, cap - 1] and p["cu_seqlens_k"].tolist() == [0, cap, 2 * cap - 1]
            assert p["slot_map"].tolist() == [cap - 1, cap - 2, -1, -1]
        else:
            with pytest.raises(da.DiffAttnError, match="does not fit"):
                da.diffattn_device_status()
            assert p["seqlens"].tolist() == s and not p["cu_seqlens_k"].any() and (p["slot_map"] == -1).all()


def test_append_of_two_rows_to_one_slot_touches_no_other():
    rng = np.random.default_rng(241)
    k, v = random_rows(rng, (40, 3, 256)), random_rows(rng, (40, 3, 256))
    slots = np.concatenate([np.arange(10, 40), [20] * 10])
    pool = rng.integers(0, 256, (4, 3, 1, 4608)).astype(np.uint8)
    want = expected_pool(pool, 2, k[:30], v[:30], slots[:30], 16)
    got = torch.tensor(pool).to(DEV)
    da.diffattn_kv4_append(k.to(DEV), v.to(DEV), dev32(slots), got)
    got = got.cpu().numpy()
    for x in (got, want):  # (that slot itself: a row of zeros in both)
        for h in range(3):
            kv4.write_row(x[1, h, 0], 2, np.zeros(256), np.zeros(256), 4)
    assert np.array_equal(got, want)
    da.diffattn_device_status()


@pytest.mark.parametrize("batch", pieces.FEW + pieces.MANY + pieces.CLUSTER, ids=lambda b: f"{b.form}-{len(b.lens)}x{b.heads}-{max(b.lens)}")
def test_decode_takes_every_piece_once(batch):
    """Values by which each piece of each row shows (test_kv4_edges_cpu.py shows that it does), over rows cut
    for all blocks, batches cut inside most rows, and rows over a cluster. The scratch holds NaN."""
    B, cols = len(batch.lens), batch.columns // 2
    Q = torch.tensor(pieces.queries(batch), dtype=torch.bfloat16, device=DEV)
    args = Q, torch.tensor(pieces.pool(batch)).to(DEV), dev32(batch.table()), dev32(batch.lens)
    size = (da.diffattn_decode_kv4_workspace_size(B, batch.heads) if batch.form == "v1"
            else da.diffattn_v2_decode_kv4_workspace_size(B, batch.heads * batch.group, batch.heads))
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    if batch.form == "v1":
        got = da.diffattn_decode_kv4(*args, torch.full((batch.heads,), pieces.LAMBDA, device=DEV), norm=False, scale=False, workspace=ws)
    else:
        logit = float(np.log(pieces.SIGMA / (1 - pieces.SIGMA)))
        got = da.diffattn_v2_decode_kv4(*args, torch.full((B, batch.heads * cols), logit, device=DEV), workspace=ws)
    want, bound = np.zeros((B, batch.heads * cols, batch.channels)), np.zeros((B, batch.heads * cols, batch.channels))
    for b in range(B):
        for h in range(batch.heads if batch.lens[b] else 0):
            at = slice(cols * h, cols * (h + 1))
            want[b, at], bound[b, at] = batch.outputs(b, h)
    within(got, want, SLACK * bound)
    da.diffattn_device_status()


def test_v1_rows_of_many_sequences_in_and_out():
    """Four planes a record: appended by views of one projection, read back whole, over many sequences."""
    rng = np.random.default_rng(251)
    for H, lens, ps in ((13, [(i * 53) % 500 for i in range(30)], 32), (3, [3000, 1, 4095, 0, 77] * 2, 80)):
        table, pages = random_table(rng, lens, ps)
        total, cu = sum(lens), np.concatenate([[0], np.cumsum(lens)])
        proj = torch.randn((total, 3, H, 256), device=DEV).to(torch.bfloat16)
        pos, seq = np.concatenate([np.arange(n) for n in lens]), np.repeat(np.arange(len(lens)), lens)
        pool = torch.zeros((pages, H, ps // 16, 4608), dtype=torch.uint8, device=DEV)
        da.diffattn_kv4_append(proj[:, 1], proj[:, 2], dev32(table[seq, pos // ps] * ps + pos % ps), pool)
        got = da.diffattn_kv4_gather(pool, dev32(table), dev32(cu), total, 256, 256)
        for i, g in enumerate(got):
            assert np.array_equal(to64(g), kv4.values(*kv4.quantize_blocks(to64(proj[:, 1 + i]))))
    da.diffattn_device_status()


def test_append_refuses_rows_that_heads_share():
    """A stride of 0 between heads (one row for all of them) or tokens, and a last dimension with steps."""
    pool = torch.full((2, 4, 1, 2304), 9, dtype=torch.uint8, device=DEV)
    rows, slots = torch.zeros((3, 4, 128), dtype=torch.bfloat16, device=DEV), dev32([0, 1, 2])
    for bad in (rows[:, :1].expand(3, 4, 128), rows[:1].expand(3, 4, 128)):
        for k, v in ((bad, rows), (rows, bad)):
            with pytest.raises(da.DiffAttnError) as e:
                da.diffattn_kv4_append(k, v, slots, pool)
            assert e.value.status == -4
    with pytest.raises(ValueError, match="contiguous"):
        da.diffattn_kv4_append(torch.zeros((3, 4, 256), dtype=torch.bfloat16, device=DEV)[..., ::2], rows, slots, pool)
    torch.cuda.synchronize()
    assert bool((pool == 9).all())


def test_decode_takes_the_scalars_that_the_other_calls_take():
    """lambda_init and eps as numpy scalars or tensors of one value."""
    lens = [70]
    table, pool, q, lam, w = v1_case(np.random.default_rng(233), lens, 2, 16)
    args = q.to(DEV), torch.tensor(pool).to(DEV), dev32(table), dev32(lens), lam.to(DEV)
    want = da.diffattn_decode_kv4(*args, 0.5, eps=2.0 ** -10)
    for kind in (np.float32, np.float64, torch.tensor):
        assert torch.equal(da.diffattn_decode_kv4(*args, kind(0.5), eps=kind(2.0 ** -10)), want)
