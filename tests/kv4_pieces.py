"""Batches in which every tile of keys shows in the output, for the joins of the 4-bit decodes.

Page p's values are 6 in channel p of V and 0 elsewhere, and the tables go through the pages in turn: an
output's channel c is the share that the pages of channel c have of the softmax. All terms have one
sign, so that an output's bound is relative to it, and a piece that is lost or taken twice changes some
output by far more than that bound. Keys are one value in all channels of a page, so that scores differ from
page to page."""
import functools
from dataclasses import dataclass

import numpy as np

from oracle import kv4_ref as kv4

# what the kernels cut a batch by: blocks, keys of a tile, tiles that a row costs besides its own, smallest range
RANGES = {"v1": (304, 128, 2, 2), "v2": (456, 128, 2, 3)}
LEVELS = np.array([0.0, 0.5, -1.0, 1.5, -0.5, 2.0, 1.0])  # of the keys, as they are cached:
LEVELS = kv4.values(*kv4.quantize_blocks(np.repeat(LEVELS, 16)))[::16]
Q = 0.125
SIGMA = 0.2      # V2's sigmoid(lambda)
LAMBDA = 0.25    # V1's


@dataclass(frozen=True)
class Batch:
    form: str
    lens: tuple
    heads: int
    group: int = 0
    page: int = 128

    @property
    def channels(self):
        return 256 if self.form == "v1" else 128

    @property
    def columns(self):
        return 2 if self.form == "v1" else self.group

    def factor(self, column):
        """What a query head's channels are, over Q: another one for each column."""
        return (1.0, -1.0, 0.0, 2.0, 0.5, 1.0, -2.0, 0.0)[column]

    def table(self):
        width = -(-max(self.lens) // self.page)
        return (np.arange(width)[None] + 5 * np.arange(len(self.lens))[:, None]) % self.channels

    def channel_of_keys(self, b, h):
        """The channel of each key of a row."""
        return (np.arange(self.lens[b]) // self.page + 5 * b + 7 * h) % self.channels

    def weights(self, b, h, column):
        """e^score of each key."""
        return np.exp(self.factor(column) * Q * LEVELS[self.channel_of_keys(b, h) % len(LEVELS)] * np.sqrt(128.0))

    def shares(self, b, h, column, times=None):
        """6 times each channel's share; `times`: how often each key is taken."""
        w = self.weights(b, h, column) * (1.0 if times is None else times)
        return 6.0 * np.bincount(self.channel_of_keys(b, h), w, self.channels) / w.sum()

    def outputs(self, b, h, times=None):
        """(outputs, the same with a plus for the minus) [pairs, channels] of a row."""
        second = LAMBDA if self.form == "v1" else SIGMA
        s = [self.shares(b, h, c, times) for c in range(self.columns)]
        return tuple(np.stack([s[2 * p] + sign * second * s[2 * p + 1] for p in range(self.columns // 2)]) for sign in (-1, 1))

    def ranges(self):
        """(ranges of the whole batch, for each row the pieces' first keys and the end)."""
        grid, tile, extra, least = RANGES[self.form]
        tiles = [-(-n // tile) for n in self.lens]
        total = sum(t + extra for t in tiles if t) * self.heads
        n = max(1, min(total // least, grid))
        starts = np.arange(n + 1) * total // n
        rows, at = {}, 0
        for b, t in enumerate(tiles):
            for h in range(self.heads if t else 0):
                first = at + extra
                cuts = starts[(starts > first) & (starts < first + t)] - first
                rows[b, h] = np.array([0, *(cuts * tile), self.lens[b]])
                at = first + t
        return n, rows


FEW = [Batch("v2", (192077,), 1, 8), Batch("v2", (100001, 95003), 1, 2), Batch("v2", (60000, 0, 1), 3, 4),
       Batch("v1", (80001,), 1), Batch("v1", (61000, 52001), 1), Batch("v1", (30000, 1, 0, 129), 2)]
MANY = [Batch("v2", tuple(3000 + i * 997 % 5000 for i in range(40)), 3, 8), Batch("v2", tuple(i * 613 % 4000 for i in range(300)), 2, 2),
        Batch("v1", tuple(2000 + i * 997 % 3000 for i in range(77)), 4), Batch("v1", tuple(i * 613 % 3000 for i in range(200)), 2)]
CLUSTER = [Batch("v2", (1024,), 1, 8, 16), Batch("v2", (777, 0, 300), 8, 4, 16), Batch("v1", (1500, 700, 1), 3, page=16), Batch("v1", (2047,), 1, page=16)]


@functools.lru_cache(maxsize=None)
def _records(form):
    """The record of each page: 16 rows alike."""
    W, kp = (256, 2) if form == "v1" else (128, 1)
    rec = np.zeros((W, 2304 * kp), dtype=np.uint8)
    for p in range(W):
        k, v = np.full(W, LEVELS[p % len(LEVELS)]), np.zeros(W)
        v[p] = 6.0
        for i in range(16):
            kv4.write_row(rec[p], kp, k, v, i)
    return rec


def pool(batch):
    rec, W = _records(batch.form), batch.channels
    heads = (np.arange(W)[:, None] + 7 * np.arange(batch.heads)[None]) % W
    return np.repeat(rec[heads][:, :, None], batch.page // 16, axis=2)


def queries(batch):
    cols = np.array([Q * batch.factor(c) for c in range(batch.columns)])
    per_head = np.repeat(cols, 128).reshape(batch.columns, 128)
    q = np.tile(per_head, (len(batch.lens), batch.heads, 1))
    return q.reshape(len(batch.lens), batch.heads, 256) if batch.form == "v1" else q
