"""Chunks over the 4-bit cache on the GPU against the float64 reference (oracle/kv4_ref.py), within the bound that
tests/test_kv4_gpu.py derives for the decode: each probability carries its rounding to fp16 and its score's error,
SLACK of itself. What P is held at differs: 2^6 times its value against a reference m that is at most 6 (in log2,
rounded up) below the largest score where it was set, and no more than 9 + 6 below any score later, so that the
largest P is at least 2^6 and an fp16 subnormal's error (2^-25) at most FLOOR = 2^-31 of it, for each key. Pieces
are joined in fp32. The query enters exactly (its channels here lie within 2^20 of the largest)."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from oracle import kv4_ref as kv4
from oracle import rope_ref as rope
from tests.gpu_util import assert_bf16, to64
from tests.test_kv4_gpu import SLACK, dev32, random_table, real_pool

pytestmark = pytest.mark.gpu
DEV = "cuda"
FLOOR = 2.0 ** -31
BF16 = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.lib()
    yield
    da.diffattn_device_status()


class Case:
    """A batch of chunks: `news` new tokens of `lens` cached ones, `behind` rows behind the last sequence."""

    def __init__(self, form, news, lens, heads, page_size, G=8, seed=0, std=1.0, behind=2, causal=True, k_exp=0, v_exp=0, **kw):
        rng = np.random.default_rng(seed + 7 * len(news) + sum(lens))
        self.rng, self.form, self.news, self.lens, self.causal, self.kw = rng, form, list(news), list(lens), causal, kw
        self.kp, self.H, self.G, self.page_size, self.k_exp, self.v_exp = (2 if form == "v1" else 1), heads, G, page_size, k_exp, v_exp
        self.table, pages = random_table(rng, lens, page_size)
        self.pool = real_pool(rng, pages, heads, page_size // 16, self.kp, std)
        self.cu = np.concatenate([[0], np.cumsum(news)])
        self.total = int(self.cu[-1]) + behind
        bf = lambda *shape: torch.tensor(rng.normal(size=shape), dtype=torch.float32).to(torch.bfloat16)  # noqa: E731
        if form == "v1":
            self.q = bf(self.total, heads, 256)
            self.lam = torch.tensor(rng.uniform(0.2, 0.8, heads), dtype=torch.float32)
            self.w = torch.tensor(rng.uniform(0.8, 1.2, 256), dtype=torch.float32)
        else:
            self.q = bf(self.total, heads * G, 128)
            self.lam = torch.tensor(rng.normal(size=(self.total, heads * G // 2)), dtype=torch.float32)

    def args(self):
        return (self.q.to(DEV), torch.tensor(self.pool).to(DEV), dev32(self.table), dev32(self.cu), dev32(self.lens), self.lam.to(DEV))

    def run(self, args=None, out=None, **kw):
        args = args or self.args()
        out = torch.full((self.total, self.q.shape[1] // (1 if self.form == "v1" else 2), 128 * self.kp), 5.0, dtype=torch.bfloat16,
                         device=DEV) if out is None else out
        kw = {"causal": self.causal, "k_exp": self.k_exp, "v_exp": self.v_exp, "max_seqlen_q": max(self.news), **kw, "out": out}
        if self.form == "v1":
            return da.diffattn_fwd_kv4(*args, 0.3, norm_weight=self.w.to(DEV), **{**self.kw, **kw})
        return da.diffattn_v2_fwd_kv4(*args, **kw)

    def want(self, **kw):
        kw = {"causal": self.causal, "k_exp": self.k_exp, "v_exp": self.v_exp, "slack": SLACK, "floor": FLOOR, **kw}
        if self.form == "v1":
            flags = {"norm": self.kw.get("norm", True), "apply_scale": self.kw.get("scale", True)}
            return kv4.fwd(self.q, self.pool, self.table, self.cu, self.lens, self.lam.numpy(), 0.3, self.w.numpy(), **flags, **kw)
        return kv4.v2_fwd(self.q, self.pool, self.table, self.cu, self.lens, self.lam.numpy(), **kw)

    def check(self, got=None, **kw):
        g, (want, bound) = to64(self.run() if got is None else got), self.want(**kw)
        rows = ~np.isnan(want).all(axis=(1, 2))
        assert np.all(g[~rows] == 5.0), "rows of no sequence were written"
        g, want, bound = g[rows], want[rows], bound[rows]
        assert np.all(np.isfinite(g))
        over = np.abs(g - want) - (bound + BF16 * (np.abs(want) + bound) + 1e-30)
        assert np.all(over <= 0), f"off by {np.max(np.abs(g - want)):.3e}, {np.sum(over > 0)} past the bound"


FORMS = ["v1", "v2"]
SHAPES = [  # new, cached
    ([1], [1]), ([1], [129]), ([3], [3]), ([5], [777]), ([16], [128]), ([17], [127]), ([64], [64]), ([65], [200]), ([130], [130]),
    ([1, 1, 1], [40, 0, 300]), ([7, 0, 2, 0], [7, 50, 600, 0]), ([33, 1, 128], [1000, 4, 129]), ([9, 9, 9, 9, 9], [16, 17, 250, 33, 64]),
    ([300], [1500]), ([12], [5000])]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("news,lens", SHAPES)
@pytest.mark.parametrize("form", FORMS)
def test_chunks(form, news, lens, causal):
    Case(form, news, lens, 2, 16, causal=causal).check()
    da.diffattn_device_status()


@pytest.mark.parametrize("hint", [0, 1, 8, 100000, None])
@pytest.mark.parametrize("form", FORMS)
def test_any_hint_gives_the_result(form, hint):
    c = Case(form, [6, 40, 1], [200, 130, 999], 3, 48)
    c.check(c.run(max_seqlen_q=hint))


@pytest.mark.parametrize("G,heads,page_size", [(2, 1, 16), (2, 5, 128), (4, 3, 48), (8, 8, 64), (4, 1, 1024)])
def test_v2_groups_and_pages(G, heads, page_size):
    for new in (1, 4, 37, 70):
        Case("v2", [new, 2], [400, 90], heads, page_size, G=G).check()


@pytest.mark.parametrize("heads,page_size", [(1, 16), (12, 64), (5, 112)])
def test_v1_heads_and_pages(heads, page_size):
    for new in (2, 31, 70):
        Case("v1", [new, 2], [400, 90], heads, page_size).check()


@pytest.mark.parametrize("norm,scale", [(False, False), (False, True), (True, False)])
def test_v1_epilogues(norm, scale):
    for new in (3, 100):
        Case("v1", [new], [300], 2, 16, norm=norm, scale=scale).check()
    c = Case("v1", [40], [1000], 2, 16)
    c.w = torch.ones(256)
    c.check(da.diffattn_fwd_kv4(*c.args(), 0.3, out=torch.full((42, 2, 256), 5.0, dtype=torch.bfloat16, device=DEV)))


@pytest.mark.parametrize("form", FORMS)
def test_exponents(form):
    for new in (2, 90):
        Case(form, [new], [260], 2, 16, k_exp=-2, v_exp=3).check()
        c = Case(form, [new], [260], 2, 16, k_exp=0, v_exp=-40)
        c.kw["eps"] = 1e-30
        if form == "v2":
            c.check()
        else:
            assert torch.isfinite(c.run().float()).all()


@pytest.mark.parametrize("form", FORMS)
def test_rows_that_see_no_key_are_zeros(form):
    """More new tokens than cached ones: the first see nothing. And a sequence of no keys at all."""
    for news, lens in (([9], [4]), ([200, 3], [70, 0]), ([64], [1]), ([130], [2])):
        c = Case(form, news, lens, 2, 16)
        if form == "v1":
            c.w[:] = float("inf")  # (zeros whatever the weight holds)
            g = to64(c.run())
            for b, (n, L) in enumerate(zip(news, lens)):
                assert np.all(g[c.cu[b]:c.cu[b] + max(0, n - L)] == 0)
        else:
            c.check()
    Case(form, [9], [4], 2, 16, causal=False).check()


@pytest.mark.parametrize("form", FORMS)
def test_references_move(form):
    """Scores that grow along the keys by far more than P's range, again and again, and one key far above the rest."""
    for new, n in ((2, 900), (100, 1200)):
        c = Case(form, [new], [n], 1, 16, G=2)
        # keys k_j = j / 8 e_0 (times the maps' first channels), queries 40 e_0 +- noise
        rows = np.zeros((n, 1, 128 * c.kp))
        rows[:, :, 0::128] = (np.arange(n) / 8)[:, None, None]
        t = torch.tensor(c.pool).to(DEV)
        slots = np.array([c.table[0, j // 16] * 16 + j % 16 for j in range(n)])
        v = torch.tensor(c.rng.normal(size=rows.shape), dtype=torch.float32).to(torch.bfloat16).to(DEV)
        da.diffattn_kv4_append(torch.tensor(rows, dtype=torch.float32).to(torch.bfloat16).to(DEV), v, dev32(slots), t)
        c.pool = t.cpu().numpy()
        q = np.zeros(c.q.shape)
        q[..., 0::128] = 40 * c.rng.uniform(0.2, 1.0, q[..., 0::128].shape)
        c.q = torch.tensor(q, dtype=torch.float32).to(torch.bfloat16)
        c.check()
        rows[:] = c.rng.normal(size=rows.shape) * 0.1
        rows[n // 2, :, 0::128] = 60.0
        da.diffattn_kv4_append(torch.tensor(rows, dtype=torch.float32).to(torch.bfloat16).to(DEV), v, dev32(slots), t)
        c.pool = t.cpu().numpy()
        c.check()


@pytest.mark.parametrize("form", FORMS)
def test_small_and_large_queries_side_by_side(form):
    """Queries of all sizes in one chunk: each row has its own power of two."""
    for new in (4, 80):
        c = Case(form, [new], [500], 2, 16, std=0.3)
        size = 2.0 ** c.rng.integers(-40, 6, (c.total, 1, 1))
        c.q = (c.q.double() * torch.tensor(size)).to(torch.bfloat16)
        c.q[1] = 0
        c.check()


@pytest.mark.parametrize("form", FORMS)
def test_slots_past_the_end_may_hold_anything(form):
    for new, n in ((3, 130), (70, 333)):
        c = Case(form, [new, 1], [n, 5], 2, 32)
        args = list(c.args())
        clean = c.run(args)
        pool = c.pool.copy()
        used = np.zeros(pool.shape[0] * 32, dtype=bool)
        for b, L in enumerate(c.lens):
            for j in range(L):
                used[c.table[b, j // 32] * 32 + j % 32] = True
        rows = np.full((int((~used).sum()), 2, 128 * c.kp), np.nan)
        t = torch.tensor(pool).to(DEV)
        da.diffattn_kv4_append(*(torch.tensor(rows).to(torch.bfloat16).to(DEV) for _ in range(2)), dev32(np.flatnonzero(~used)), t)
        args[1] = t
        assert torch.equal(c.run(args), clean)
        table = np.where(c.table < 0, 12345, c.table)  # nor do the table's entries past the pages
        args[2] = dev32(table)
        assert torch.equal(c.run(args), clean)
    da.diffattn_device_status()


def poison(c, token, what):
    """The pool with K's or V's row of `token` of sequence 0 and head 1 NaN (V: channels 32 .. 47 alone)."""
    k, v = kv4.sequence_rows(c.pool, c.kp, c.table, 0, c.lens[0])
    k, v = k[token:token + 1].copy(), v[token:token + 1].copy()
    if what == "k":
        k[:, 1] = np.nan
    else:
        v[:, 1, 32:48] = np.nan
    t = torch.tensor(c.pool).to(DEV)
    slot = c.table[0, token // c.page_size] * c.page_size + token % c.page_size
    da.diffattn_kv4_append(*(torch.tensor(x).to(torch.bfloat16).to(DEV) for x in (k, v)), dev32([slot]), t)
    return t


@pytest.mark.parametrize("form", FORMS)
def test_a_nan_key_or_value_reaches_the_rows_that_see_it_alone(form):
    for new, n in ((5, 140), (100, 300), (20, 3000)):
        c = Case(form, [new, 4], [n, 50], 2, 16, G=4)
        args = list(c.args())
        clean = c.run(args)
        for token in (0, n - new, n - new // 2 - 1, n - 1):
            for what in ("k", "v"):
                args[1] = poison(c, token, what)
                got = c.run(args)
                hit = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
                first = max(0, token - (n - new))
                heads = slice(1, 2) if form == "v1" else slice(2, 4)
                hit[first:new, heads, slice(None) if what == "k" or form == "v1" else slice(32, 48)] = True
                assert torch.isnan(got[hit]).all(), (new, token, what)
                assert torch.equal(got[~hit], clean[~hit]), (new, token, what)


@pytest.mark.parametrize("form", FORMS)
def test_nan_and_inf_queries_stay_in_their_rows(form):
    for new in (6, 90):
        c = Case(form, [new], [300], 2, 16, G=4)
        args = list(c.args())
        clean = c.run(args)
        for value in (float("nan"), float("inf")):
            q = args[0].clone()
            q[2, 1, 7] = value
            got = c.run([q] + args[1:])
            hit = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
            hit[2, 1 if form == "v1" else 0] = True
            assert torch.equal(got[~hit], clean[~hit]) and not torch.isfinite(got[hit]).any()


@pytest.mark.parametrize("form", FORMS)
def test_lengths_out_of_range_are_clamped_and_bad_offsets_reported(form):
    c = Case(form, [4, 6, 3], [32, 64, 48], 2, 16)
    args = list(c.args())
    assert c.table.shape[1] == 4
    clean = c.run(args)
    got = c.run(args[:4] + [dev32([32, 1000, 48])] + args[5:])
    assert torch.equal(got, clean)
    assert torch.all(c.run(args[:4] + [dev32([-5, 64, 48])] + args[5:])[:4] == 0)
    da.diffattn_device_status()
    for cu in ([0, 4, 2, 13], [0, -1, 10, 13], [0, 4, 10, 99]):
        got = c.run(args[:3] + [dev32(cu)] + args[4:])
        with pytest.raises(da.DiffAttnError):
            da.diffattn_device_status()
        taken = [set(range(cu[b], cu[b + 1])) if 0 <= cu[b] <= cu[b + 1] <= c.total else set() for b in range(3)]
        for b in range(3):  # a sequence where it was is right, but for rows that another one claims as well
            if taken[b] and cu[b:b + 2] == list(c.cu[b:b + 2]):
                own = sorted(taken[b].difference(*(taken[o] for o in range(3) if o != b)))
                assert len(own) >= 2 and torch.equal(got[own], clean[own])
    assert torch.all(got[13:] == 5)


@pytest.mark.parametrize("form", FORMS)
def test_bad_page_reads_page_0_and_is_reported(form):
    for new in (3, 80):
        c = Case(form, [new], [200], 2, 16)
        for bad in (-1, c.pool.shape[0], 1 << 30):
            table = c.table.copy()
            table[0, 5] = 0
            args = list(c.args())
            args[2] = dev32(table)
            want = c.run(args)
            table[0, 5] = bad
            args[2] = dev32(table)
            da.diffattn_device_status()
            got = c.run(args)
            with pytest.raises(da.DiffAttnError):
                da.diffattn_device_status()
            assert torch.equal(got, want)


@pytest.mark.parametrize("form", FORMS)
def test_repeats_bit_for_bit_whatever_the_workspace_holds(form):
    for news, lens in (([5, 1], [3000, 20]), ([90, 200], [1000, 200])):
        c = Case(form, news, lens, 2, 64)
        args = c.args()
        size = (da.diffattn_fwd_kv4_workspace_size(max(news)) if form == "v1"
                else da.diffattn_v2_fwd_kv4_workspace_size(max(news), 16, 2))
        want = c.run(args)
        for fill in (0, 255, 127):
            ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
            for _ in range(5):
                assert torch.equal(c.run(args, workspace=ws), want)
        c.check(want)


@pytest.mark.parametrize("form", FORMS)
def test_captured_and_replayed_and_on_another_stream(form):
    c = Case(form, [7, 50], [400, 90], 2, 16)
    args = list(c.args())
    want, out = c.run(args), torch.full_like(c.run(args), 5.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c.run(args, out=out, stream=st)
    torch.cuda.current_stream().wait_stream(st)
    assert torch.equal(out, want)
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    out2 = torch.full_like(out, 5.0)
    c.w = c.w.to(DEV) if form == "v1" else None
    with torch.cuda.graph(g):
        c.run(args, out=out)
    with torch.cuda.graph(h):
        c.run(args, out=out2)
    for n in (400, 57, 399):
        args[4].copy_(dev32([n, 90]))
        fresh = c.run(args)
        out.fill_(5.0), out2.fill_(5.0)
        a, b = torch.cuda.Stream(), torch.cuda.Stream()
        for s, graph in ((a, g), (b, h)):  # two graphs at once share no scratch
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.current_stream().wait_stream(a)
        torch.cuda.current_stream().wait_stream(b)
        assert torch.equal(out, fresh) and torch.equal(out2, fresh)


@pytest.mark.parametrize("form", FORMS)
def test_guards(form):
    c = Case(form, [5, 66], [300, 70], 2, 16)
    args = c.args()
    clean = c.run(args)
    buf = torch.full((clean.numel() + 8192,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[4096:4096 + clean.numel()].view(clean.shape)
    c.run(args, out=out)
    assert torch.equal(out[:-2], clean[:-2]) and bool((out[-2:] == 7).all())
    assert bool((buf[:4096] == 7).all()) and bool((buf[4096 + clean.numel():] == 7).all())


@pytest.mark.parametrize("form", FORMS)
def test_a_chunk_of_one_token_agrees_with_the_decode(form):
    c = Case(form, [1] * 4, [300, 0, 65, 4000], 2, 16, behind=0)
    q, pool, table, cu, lens, lam = c.args()
    got = c.run()
    dec = (da.diffattn_decode_kv4(q, pool, table, lens, lam, 0.3, norm_weight=c.w.to(DEV)) if form == "v1"
           else da.diffattn_v2_decode_kv4(q, pool, table, lens, lam))
    assert_bf16(got, dec)


def test_a_long_prompt_agrees_with_the_packed_prefill_over_the_read_out():
    """The same values through diffattn_kv4_gather and the tensor-core prefills."""
    for form in FORMS:
        c = Case(form, [700, 130], [2000, 1130], 4, 64, G=4, behind=0)
        q, pool, table, cu, lens, lam = c.args()
        cu_k = dev32([0, 2000, 3130])
        k, v = da.diffattn_kv4_gather(pool, table.clamp(min=0), cu_k, 3130, 128 * c.kp, 128 * c.kp)
        got = c.run()
        wide = (da.diffattn_fwd_varlen_qk(q, k, v, cu, cu_k, lam, 0.3, norm_weight=c.w.to(DEV)) if form == "v1"
                else da.diffattn_v2_fwd_varlen(q, k, v, lam, cu, cu_seqlens_k=cu_k))
        assert_bf16(got, wide)


@pytest.mark.parametrize("seed", range(12))
def test_random_batches(seed):
    rng = np.random.default_rng(900 + seed)
    form, B = FORMS[seed % 2], int(rng.integers(1, 12))
    news = [int(n) for n in np.exp(rng.uniform(0, np.log(120 if seed % 3 else 9), B))]
    lens = [0 if rng.random() < 0.1 else n + int(np.exp(rng.uniform(0, np.log(1500)))) - 1 for n in news]
    news = [0 if rng.random() < 0.1 else n for n in news]
    if max(news) == 0:
        news[0] = 3
    Case(form, news, lens, int(rng.integers(1, 5)), 16 * int(rng.integers(1, 6)), G=int(rng.choice([2, 4, 8])), seed=seed,
         causal=bool(rng.random() < 0.8)).check()


def test_the_largest_batch_and_more_units_than_blocks():
    for form in FORMS:
        B = 8192 if form == "v2" else 700
        rng = np.random.default_rng(5)
        news, lens = [1] * B, [int(n) for n in rng.integers(0, 3, B)]
        Case(form, news, lens, 1, 16, G=2).check()


def test_pool_offsets_past_32_bits():
    """A pool of more than 4 GB: the last page is where it should be."""
    page_size, H = 1024, 12
    rec = (page_size // 16) * 4608 * H
    pages = (1 << 32) // rec + 3
    pool = torch.zeros((pages, H, page_size // 16, 4608), dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(109)
    rows = torch.tensor(rng.normal(size=(2, 140, H, 256)), dtype=torch.float32).to(torch.bfloat16).to(DEV)
    first = (pages - 1) * page_size
    da.diffattn_kv4_append(rows[0], rows[1], torch.arange(first, first + 140, dtype=torch.int32, device=DEV), pool)
    lam = torch.full((H,), 0.3)
    for n in (3, 70):
        q = torch.tensor(rng.normal(size=(n, H, 256)), dtype=torch.float32).to(torch.bfloat16)
        got = to64(da.diffattn_fwd_kv4(q.to(DEV), pool, dev32([[pages - 1]]), dev32([0, n]), dev32([140]), lam.to(DEV), 0.2, max_seqlen_q=n))
        want, bound = kv4.fwd(q, pool[-1:].cpu().numpy(), [[0]], [0, n], [140], lam.numpy(), 0.2, slack=SLACK, floor=FLOOR)
        assert np.all(np.abs(got - want) <= bound + BF16 * (np.abs(want) + bound))


@pytest.mark.parametrize("form", FORMS)
def test_steps_that_extend_sequences(form):
    """What a server does: plan, turn and append, attend, chunk after chunk over one small pool; the pool's rows
    and every chunk's outputs against the reference, and all chunks against one of the whole prompt."""
    rng = np.random.default_rng(31)
    B, H, G, page, kp = 3, 2, 4, 16, 2 if form == "v1" else 1
    hq, w = (H, 256) if form == "v1" else (H * G, 128)
    steps = [[40, 7, 130], [1, 1, 1], [5, 0, 3], [64, 1, 2], [1, 90, 1]]
    tab = torch.as_tensor(rope.table(10000.0 ** (-np.arange(64) / 64), 400)).float().to(DEV)
    pool, i32 = da.diffattn_kv4_pool(80, page, H, w, w), dict(dtype=torch.int32, device=DEV)
    seqlens, table = torch.zeros(B, **i32), torch.zeros((B, 20), **i32)
    ring, state = torch.as_tensor(rng.permutation(80)).to(**i32), torch.tensor([17, 80], **i32)
    lam1 = torch.tensor(rng.uniform(0.2, 0.8, H), dtype=torch.float32)
    host = np.zeros((80, H, 1, 2304 * kp), dtype=np.uint8)
    for new in steps:
        total = sum(new) + 3
        plan = da.diffattn_paged_plan(seqlens, dev32(new), table, ring, state, page, total)
        seqlens, state = plan["seqlens"], plan["ring_state"]
        proj = torch.tensor(rng.normal(size=(total, hq + 2 * H, w)), dtype=torch.float32).to(torch.bfloat16).to(DEV)
        q, k, v = proj[:, :hq], proj[:, hq:hq + H], proj[:, hq + H:]
        turned = da.diffattn_rope_kv4_append(q, k, v, tab, plan["positions"], plan["slot_map"], pool, q_out=torch.zeros_like(q).contiguous())
        lam = torch.tensor(rng.normal(size=(total, hq // 2)), dtype=torch.float32)
        if form == "v1":
            out = da.diffattn_fwd_kv4(turned, pool, table, plan["cu_seqlens_q"], seqlens, lam1.to(DEV), 0.3, max_seqlen_q=max(new))
        else:
            out = da.diffattn_v2_fwd_kv4(turned, pool, table, plan["cu_seqlens_q"], seqlens, lam.to(DEV), max_seqlen_q=max(new))
        da.diffattn_device_status()
        # the reference: rows turned, rounded and written one by one, then attention over them
        pos, slots, n = plan["positions"].cpu().numpy(), plan["slot_map"].cpu().numpy(), sum(new)
        t64 = tab.cpu().double().numpy()
        kt = rope.to_bf16(rope.rotate(to64(k), t64, pos, 128))
        qt = rope.to_bf16(rope.rotate(to64(q), t64, pos, 128))
        for i in range(n):
            for h in range(H):
                kv4.write_row(host[slots[i] // page, h, 0], kp, kt[i, h], to64(v)[i, h], slots[i] % page)
        assert np.array_equal(pool.cpu().numpy(), host)
        assert np.array_equal(to64(turned)[:n], qt[:n])
        cu = np.concatenate([[0], np.cumsum(new)])
        if form == "v1":
            want, bound = kv4.fwd(qt, host, table.cpu().numpy(), cu, seqlens.cpu().numpy(), lam1.numpy(), 0.3, slack=SLACK, floor=FLOOR)
        else:
            want, bound = kv4.v2_fwd(qt, host, table.cpu().numpy(), cu, seqlens.cpu().numpy(), lam.numpy(), slack=SLACK, floor=FLOOR)
        g = to64(out)[:n]
        assert np.all(np.abs(g - want[:n]) <= bound[:n] + BF16 * (np.abs(want[:n]) + bound[:n]) + 1e-30)


def test_binding_names_the_operand_that_does_not_fit():
    for form in FORMS:
        c = Case(form, [4, 2], [40, 9], 2, 16)
        good = list(c.args())
        names = ["q", "pool", "block_table", "cu_seqlens_q", "seqlens", "lam" if form == "v1" else "lam_logit"]
        for i, name in enumerate(names):
            for bad in (good[i].double() if good[i].dtype != torch.uint8 else good[i].int(), good[i].cpu(), None, good[i][..., None]):
                with pytest.raises(ValueError):
                    c.run(good[:i] + [bad] + good[i + 1:])
        with pytest.raises(ValueError):
            c.run(good, workspace=torch.zeros(4096))
        with pytest.raises(da.DiffAttnError):
            c.run(good, workspace=torch.zeros(4096, device=DEV))
        with pytest.raises(ValueError):
            c.run(good, out=torch.zeros(3, device=DEV))
    q = torch.zeros((0, 4, 128), dtype=torch.bfloat16, device=DEV)
    out = da.diffattn_v2_fwd_kv4(q, da.diffattn_kv4_pool(1, 16, 2, 128, 128), dev32([[0]]), dev32([0, 0]), dev32([5]), torch.zeros((0, 2), device=DEV))
    assert out.shape == (0, 2, 128)
