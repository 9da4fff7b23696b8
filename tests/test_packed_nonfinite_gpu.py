"""Packed training steps in which rows of no sequence, or all rows of one sequence, hold NaN or Inf: the gradients of
the other sequences are those of the clean step. Tiles of 128 rows reach past a sequence's end on both sides of every
product, so that a masked weight of 0 meets those rows (0 times NaN is NaN).

Every gradient here is a sum in a fixed order or of two terms (dQ: of two tiles of keys; a noise head's dK: of two
signal heads), and so has equal bits, but for a noise head's dQ: four terms, two heads by two tiles, are added in fp32
in any order. Two orders differ by at most 6 * 2^-24 of the terms' magnitudes, which are taken to be at most 4 * 16 times
the largest gradient (2^-15 of it), and each is then rounded to bf16, half a step off."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = torch.finfo(torch.bfloat16).eps  # two roundings of half a step


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.lib()
    yield
    da.diffattn_device_status()


class Step:
    """A training step over sequences of `lens` rows, with `behind` rows of no sequence."""

    def __init__(self, lens, behind, grouped, norm, causal):
        gen = torch.Generator().manual_seed(sum(lens) + behind)
        self.grouped, self.kw = grouped, {"norm": norm, "causal": causal}
        self.ends = np.concatenate([[0], np.cumsum(lens)])
        total, self.H, noise = int(self.ends[-1]) + behind, 2, 1
        heads, width = (self.H + noise, 128) if grouped else (self.H, 256)
        bf = lambda *shape: torch.randn(shape, generator=gen).to(torch.bfloat16).to(DEV)  # noqa: E731
        self.clean = {"q": bf(total, heads, width) / 4, "k": bf(total, heads, width) / 4, "v": bf(total, self.H, 256),
                      "dy": bf(total, self.H, 256)}
        self.cu = torch.tensor(self.ends, dtype=torch.int32, device=DEV)
        self.lam = torch.tensor([0.4, 0.7], device=DEV)

    def run(self, x):
        if self.grouped:
            out, o_pre, stats = da.diffattn_gda_fwd_train_varlen(x["q"], x["k"], x["v"], self.cu, self.lam, self.H, 0.3, **self.kw)
            g = da.diffattn_gda_bwd_varlen(x["q"], x["k"], x["v"], o_pre, stats, x["dy"], self.cu, self.lam, self.H, 0.3, **self.kw)
        else:
            out, o_pre, stats = da.diffattn_fwd_train_varlen(x["q"], x["k"], x["v"], self.cu, self.lam, 0.3, **self.kw)
            g = da.diffattn_bwd_varlen(x["q"], x["k"], x["v"], o_pre, stats, x["dy"], self.cu, self.lam, 0.3, **self.kw)
        return {"out": out, **g}

    def same(self, got, want, rows, what):
        for name in ("out", "dq", "dk", "dv"):
            a, b = got[name][rows].float(), want[name][rows].float()
            assert torch.isfinite(a).all(), (what, name)
            if name == "dq" and self.grouped:
                top = b.abs().max()
                assert torch.all((a[:, self.H:] - b[:, self.H:]).abs() <= STEP * b[:, self.H:].abs() + 2.0 ** -15 * top), (what, name)
                a, b = a[:, :self.H], b[:, :self.H]
            assert torch.equal(a, b), (what, name)


CASES = [(grouped, norm, causal) for grouped in (False, True) for norm in (False, True) for causal in (False, True)]


@pytest.mark.parametrize("lens,behind", [([200, 1, 77], 300), ([5], 3), ([256, 129], 130)])
@pytest.mark.parametrize("grouped,norm,causal", CASES)
def test_rows_of_no_sequence_may_hold_anything(grouped, norm, causal, lens, behind):
    s = Step(lens, behind, grouped, norm, causal)
    want, rows = s.run(s.clean), slice(0, sum(lens))
    for value in (float("nan"), float("inf")):
        for names in (("q",), ("k",), ("v",), ("dy",), ("q", "k", "v", "dy")):
            x = dict(s.clean)
            for name in names:
                x[name] = x[name].clone()
                x[name][sum(lens):] = value
            got = s.run(x)
            s.same(got, want, rows, (names, value))
            assert torch.equal(got["dlam"], want["dlam"]), names
            for name in ("dq", "dk", "dv"):
                assert torch.all(got[name][sum(lens):] == 0), names  # as the call returns them


@pytest.mark.parametrize("lens", [[200, 77, 130], [1, 5, 1], [130, 256, 60]])
@pytest.mark.parametrize("grouped,norm,causal", CASES)
def test_a_sequence_of_nans_reaches_no_other(grouped, norm, causal, lens):
    s = Step(lens, 2, grouped, norm, causal)
    want, mine = s.run(s.clean), slice(int(s.ends[1]), int(s.ends[2]))
    for names in (("q",), ("k",), ("v",), ("dy",), ("q", "k", "v", "dy")):
        x = dict(s.clean)
        for name in names:
            x[name] = x[name].clone()
            x[name][mine] = float("nan")
        got = s.run(x)
        assert torch.isnan(got["dq"][mine].float()).any() or torch.isnan(got["dv"][mine].float()).any()
        for b in (0, 2):
            s.same(got, want, slice(int(s.ends[b]), int(s.ends[b + 1])), (names, b))


@pytest.mark.parametrize("grouped,norm,causal", CASES)
def test_long_sequences_with_ragged_ends(grouped, norm, causal):
    """Rings that went round several times before the last tile. dQ has up to 16 terms here (8 tiles by two heads): 30
    additions of 2^-24 of at most 16 * 16 times the largest gradient, 2^-11 of it."""
    lens = [700, 1000, 385]
    s = Step(lens, 40, grouped, norm, causal)
    want = s.run(s.clean)
    x = {name: t.clone() for name, t in s.clean.items()}
    for t in x.values():
        t[int(s.ends[1]):int(s.ends[2])] = float("nan")
        t[int(s.ends[3]):] = float("nan")
    got = s.run(x)
    for b in (0, 2):
        rows = slice(int(s.ends[b]), int(s.ends[b + 1]))
        for name in ("out", "dq", "dk", "dv"):
            a, w = got[name][rows].float(), want[name][rows].float()
            assert torch.isfinite(a).all(), (b, name)
            if name == "dq":
                assert torch.all((a - w).abs() <= STEP * w.abs() + 2.0 ** -11 * w.abs().max()), (b, name)
            else:
                assert torch.equal(a, w), (b, name)
