"""Rotary positions at the values where a rounding or an infinity decides: against the formula in
float64, which holds the products of two 24-bit factors exactly."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
def test_infinities_are_the_formulas(dtype, inverse, interleaved):
    """An infinite member of a pair gives the infinities (or, where they cancel or meet a 0, the NaN) of the formula."""
    gen = torch.Generator().manual_seed(21)
    top, total = 7, 63
    tab = torch.as_tensor(rope.table(10000.0 ** (-np.arange(8) / 8), top)).float().to(DEV)
    pos = np.arange(total) % top  # position 0: sines of 0
    x = torch.randn((total, 2, 64), generator=gen)
    inf = float("inf")
    first, second = (0, 1) if interleaved else (3, 11)  # a pair's channels
    for t in range(total):
        a, b = [(inf, None), (-inf, None), (None, inf), (None, -inf), (inf, inf), (inf, -inf), (-inf, inf), (float("nan"), None),
                (None, float("nan"))][t // top]
        if a is not None:
            x[t, 1, first] = a
        if b is not None:
            x[t, 1, second] = b
    x = x.to(dtype).to(DEV)
    got = n64(da.diffattn_rope(x, None, tab, dev32(pos), 64, interleaved=interleaved, inverse=inverse)[0])
    with np.errstate(invalid="ignore"):
        want = rope.rotate(n64(x), n64(tab), pos, 64, interleaved=interleaved, inverse=inverse)
    wild = ~np.isfinite(want)
    assert np.isinf(want).sum() > total and np.array_equal(np.isnan(got), np.isnan(want))
    inf_at = np.isinf(want)
    assert np.array_equal(got[inf_at], want[inf_at])
    assert np.all(np.abs(got[~wild] - want[~wild]) <= 2.0 ** -8 * np.abs(want[~wild]) + 2.0 ** -40)


@pytest.mark.parametrize("interleaved", [False, True])
def test_fp32_where_the_products_all_but_cancel(interleaved):
    """The published bound, 2^-22 of the value and 2^-46 of the products, where the value is some 2^-24 of them: one
    fused product of a rounded other one would be off by 2^-25 of the products."""
    rng = np.random.default_rng(22)
    top, pairs = 4000, 8
    turn = rng.uniform(0.2, 1.3, (top, pairs))
    tab = np.stack([np.cos(turn), np.sin(turn)], -1).astype(np.float32)
    c, s = tab[..., 0].astype(np.float64), tab[..., 1].astype(np.float64)
    x1, x2 = np.zeros((top, pairs), np.float32), np.zeros((top, pairs), np.float32)
    half = np.arange(top) % 2 == 0
    x2[half] = rng.normal(size=(half.sum(), pairs))
    x1[half] = x2[half] * s[half] / c[half]          # x1 c - x2 s cancels
    x1[~half] = rng.normal(size=((~half).sum(), pairs))
    x2[~half] = -x1[~half] * s[~half] / c[~half]     # x2 c + x1 s cancels
    x = np.zeros((top, 1, 64), np.float32)
    lo, hi = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    x[:, 0, lo], x[:, 0, hi] = x1, x2
    got = n64(da.diffattn_rope(torch.as_tensor(x).to(DEV), None, torch.as_tensor(tab).to(DEV), dev32(np.arange(top)), 64,
                               interleaved=interleaved)[0])[:, 0]
    x1, x2 = x1.astype(np.float64), x2.astype(np.float64)
    for y, a, b in ((got[:, lo], x1 * c, -x2 * s), (got[:, hi], x2 * c, x1 * s)):
        want, size = a + b, np.abs(a) + np.abs(b)
        assert np.all(np.abs(y - want) <= 2.0 ** -22 * np.abs(want) + 2.0 ** -46 * size)
    small = np.abs(x1 * c - x2 * s)[half]
    assert np.median(small / np.abs(x1 * c)[half]) < 2.0 ** -22  # (they do cancel)
