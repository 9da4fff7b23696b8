"""What the 4-bit cache's calls refuse or promise, as far as it shows without a GPU."""
import types

import numpy as np
import pytest

import differential_attention_gb300 as da
from oracle import kv4_ref as kv4
from tests import kv4_pieces as pieces

SLACK, BF16 = 2.0 ** -8.4, 2.0 ** -8  # (as in test_kv4_gpu.py)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """A call would run on its operands' device, on that device's current stream and not on the one given."""
    class Stream:
        def __init__(self, index):
            self.device_index = index

    class Tensor:
        is_cuda, device = True, "cuda:0"

        def get_device(self):
            return 0

    cuda = types.SimpleNamespace(Stream=Stream, stream=lambda s: ("in", s))
    monkeypatch.setattr(da, "torch", types.SimpleNamespace(Tensor=Tensor, cuda=cuda))
    own = Stream(0)
    assert da._current(own, Tensor()) == ("in", own)
    for call in (da._current, lambda s, t: da.diffattn_paged_plan(t, t, t, t, t, 16, 4, stream=s),
                 lambda s, t: da.diffattn_kv4_append(t, t, t, t, stream=s),
                 lambda s, t: da.diffattn_kv4_gather(t, t, t, 4, 128, 128, stream=s),
                 lambda s, t: da.diffattn_decode_kv4(t, t, t, t, t, stream=s),
                 lambda s, t: da.diffattn_v2_decode_kv4(t, t, t, t, t, stream=s)):
        with pytest.raises(ValueError, match="stream is of cuda:1"):
            call(Stream(1), Tensor())


# ---- the batches of tests/kv4_pieces.py ---------------------------------------------------------

@pytest.mark.parametrize("batch", pieces.CLUSTER[1:3], ids=str)
def test_pieces_outputs_are_the_oracles(batch):
    pool, q, B, cols = pieces.pool(batch), pieces.queries(batch), len(batch.lens), batch.columns // 2
    if batch.form == "v1":
        want, _ = kv4.decode(q, pool, batch.table(), batch.lens, np.full(batch.heads, pieces.LAMBDA), 0.0, norm=False, apply_scale=False)
    else:
        logit = np.log(pieces.SIGMA / (1 - pieces.SIGMA))
        want, _ = kv4.v2_decode(q, pool, batch.table(), batch.lens, np.full((B, cols * batch.heads), logit))
    for b in range(B):
        for h in range(batch.heads if batch.lens[b] else 0):
            assert np.allclose(batch.outputs(b, h)[0], want[b, cols * h:cols * (h + 1)], rtol=1e-12, atol=1e-15)


def test_pieces_fill_the_grid():
    """One row over all blocks (V1's first range holds the row's fixed cost alone), and rows in several pieces."""
    n, rows = pieces.FEW[0].ranges()
    assert n == 456 and len(rows[0, 0]) - 1 == 456
    n, rows = pieces.FEW[3].ranges()
    assert n == 304 and len(rows[0, 0]) - 1 == 303
    for batch in pieces.MANY:
        n, rows = batch.ranges()
        assert n == pieces.RANGES[batch.form][0] and max(len(r) for r in rows.values()) > 3


@pytest.mark.parametrize("batch", pieces.FEW + pieces.MANY, ids=lambda b: f"{b.form}-{len(b.lens)}x{b.heads}-{max(b.lens)}")
def test_pieces_show_when_one_is_lost_or_taken_twice(batch):
    """Twice past the bound that test_decode_takes_every_piece_once allows, whichever piece it is."""
    rows = [(row, cuts) for row, cuts in batch.ranges()[1].items() if len(cuts) > 2]
    for (b, h), cuts in rows[:: max(1, len(rows) // 8)]:
        want, plus = batch.outputs(b, h)
        allowed = SLACK * plus + BF16 * (np.abs(want) + SLACK * plus)
        for first, end in list(zip(cuts, cuts[1:]))[:: max(1, len(cuts) // 60)]:
            for times in (0.0, 2.0):
                taken = np.ones(batch.lens[b])
                taken[first:end] = times
                off = np.abs(batch.outputs(b, h, taken)[0] - want)
                assert np.any(off > 2 * allowed), (b, h, first, end, times)
