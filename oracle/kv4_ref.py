"""Float64 / whole-number reference of the 4-bit key/value cache and of the page plan, written from
their definitions (include/diffattn.h): the rounding to e2m1 codes with one e4m3 scale per 16
channels, the records' byte order, the plan's bookkeeping request by request, and the decodes over
the values that a pool's bytes stand for (the attention itself is diffattn_ref's). Test
infrastructure: the library never calls it."""
from __future__ import annotations

import numpy as np

from . import diffattn_ref as ref

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])  # code 127 is NaN
PLANE = 1152


def nearest(x, grid):
    """Index of the value of the ascending `grid` nearest to each x >= 0; of two as near, the even
    index (its code ends in 0); past the last, the last."""
    x = np.asarray(x, dtype=np.float64)
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return np.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)


def quantize_blocks(x, exp: int = 0):
    """x [..., 16 n] to (codes 0..15 of the same shape, scale bytes [..., n])."""
    x = np.asarray(x, dtype=np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16) * 2.0 ** -exp
    odd = ~np.all(np.isfinite(b), axis=-1)
    safe = np.where(odd[..., None], 0.0, b)
    s = nearest(np.max(np.abs(safe), axis=-1) / 6, E4M3)
    sv = E4M3[s][..., None]
    y = np.divide(np.abs(safe), sv, out=np.zeros_like(safe), where=sv > 0)
    c = nearest(y, E2M1) + 8 * (np.signbit(safe) & (sv > 0))
    return c.reshape(x.shape).astype(np.uint8), np.where(odd, 127, s).astype(np.uint8)


def values(codes, scales, exp: int = 0):
    """What codes [..., 16 n] with scale bytes [..., n] stand for."""
    v = E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.append(E4M3, np.nan)[scales & 127]
    return v * np.repeat(s, 16, axis=-1) * 2.0 ** exp


def k_code_at(i, t):
    return 512 * (i // 2 % 2) + 128 * (i // 4) + 64 * (i % 2) + 16 * t


def k_scale_at(i, t, u):
    return 1024 + 32 * (i // 4) + 16 * (i % 2) + 4 * t + 2 * (i // 2 % 2) + u


def v_code_at(i, g):
    return 512 * (i // 2 % 2) + 64 * g + 16 * (i // 4) + 8 * (i % 2)


def v_scale_at(i, g):
    return 1024 + 16 * g + 4 * (i // 4) + i % 4


def write_row(record, kp: int, k, v, i: int, k_exp: int = 0, v_exp: int = 0):
    """Rows k [128 kp], v as token i of a record (uint8, written in place)."""
    for rows, first, exp, is_k in ((k, 0, k_exp, True), (v, kp, v_exp, False)):
        codes, scales = quantize_blocks(rows, exp)
        packed = codes[0::2] | (codes[1::2] << 4)
        for blk in range(len(scales)):
            base, b8 = (first + blk // 8) * PLANE, blk % 8
            at = base + (k_code_at(i, b8 // 2) + 8 * (b8 % 2) if is_k else v_code_at(i, b8))
            record[at:at + 8] = packed[8 * blk:8 * blk + 8]
            record[base + (k_scale_at(i, b8 // 2, b8 % 2) if is_k else v_scale_at(i, b8))] = scales[blk]


def read_rows(pool, kp: int, page, token, k_exp: int = 0, v_exp: int = 0):
    """K [n, H, 128 kp] and V of tokens `token` of pages `page` (arrays of n) of a pool
    [num_pages, H, R, record]."""
    pool = np.asarray(pool)
    page, token = np.asarray(page), np.asarray(token)
    rec, i = pool[page, :, token // 16], (token % 16)[:, None]  # [n, H, record]
    vp = pool.shape[-1] // PLANE - kp
    c = np.arange(128)

    def plane(p, code_at, scale_at):
        byte = np.take_along_axis(rec, np.broadcast_to((p * PLANE + code_at)[:, None], (*rec.shape[:2], 128)), -1)
        codes = np.where(c % 2 == 0, byte & 15, byte >> 4)
        s = np.take_along_axis(rec, np.broadcast_to((p * PLANE + scale_at)[:, None], (*rec.shape[:2], 128)), -1)
        return E2M1[codes & 7] * np.where(codes & 8, -1.0, 1.0) * np.append(E4M3, np.nan)[s & 127]

    k = [plane(p, k_code_at(i, c // 32) + c % 32 // 2, k_scale_at(i, c // 32, c % 32 // 16)) for p in range(kp)]
    v = [plane(kp + p, v_code_at(i, c // 16) + c % 16 // 2, v_scale_at(i, c // 16)) for p in range(vp)]
    return np.concatenate(k, -1) * 2.0 ** k_exp, np.concatenate(v, -1) * 2.0 ** v_exp


def sequence_rows(pool, kp, block_table, b, n, start=0, k_exp=0, v_exp=0):
    page_size = pool.shape[2] * 16
    pos = np.arange(start, start + n)
    return read_rows(pool, kp, np.asarray(block_table)[b, pos // page_size], pos % page_size, k_exp, v_exp)


def paged_plan(seqlens, new_tokens, block_table, ring, state, page_size: int, total_max: int) -> dict:
    """The plan, request by request. Raises ValueError where the step does not fit."""
    table, ring = np.array(block_table), np.array(ring)
    num_pages = len(ring)
    head, count = int(state[0]), int(state[1])
    if not (0 <= head < num_pages and 0 <= count <= num_pages):
        raise ValueError("ring state")
    out, queue = [int(s) for s in seqlens], [ring[(head + i) % num_pages] for i in range(count)]
    up = lambda n: -(-n // page_size)  # noqa: E731
    cap = table.shape[1] * page_size
    for b, (s, n) in enumerate(zip(seqlens, new_tokens)):
        if not 0 <= s <= cap or n < -1 or s + max(n, 0) > cap:
            raise ValueError("length")
        if n < 0:
            queue += [table[b, i] for i in range(up(s))]
            out[b] = 0
    if len(queue) > num_pages:
        raise ValueError("more pages than the pool has")
    for i in range(count, len(queue)):
        ring[(head + i) % num_pages] = queue[i]
    taken, slots, pos, cu_q, cu_k = 0, [], [], [0], [0]
    for b, (s, n) in enumerate(zip(seqlens, new_tokens)):
        n = max(int(n), 0)
        for i in range(up(s), up(s + n)):
            if taken == len(queue):
                raise ValueError("out of pages")
            table[b, i] = queue[taken]
            taken += 1
        if n:
            out[b] = s + n
        for j in range(s, s + n):
            page = table[b, j // page_size]
            slots.append(page * page_size + j % page_size if 0 <= page < num_pages else -1)
            pos.append(j)
        cu_q.append(cu_q[-1] + n)
        cu_k.append(cu_k[-1] + (s + n if n else 0))
    if len(slots) > total_max:
        raise ValueError("more tokens than total_max")
    fill = [-1] * (total_max - len(slots))
    return {"seqlens": np.array(out), "ring_state": np.array([(head + taken) % num_pages, len(queue) - taken]),
            "cu_seqlens_q": np.array(cu_q), "cu_seqlens_k": np.array(cu_k), "slot_map": np.array(slots + fill),
            "positions": np.array(pos + fill), "block_table": table, "free_ring": ring}


def _weights(q, k):
    s = (k @ q) / np.sqrt(q.shape[0])
    return ref.softmax_rows(s[None])[0]


def _off(a, v, slack, floor):
    """How far a @ v may be off where each weight errs by slack of itself and floor of the largest."""
    return slack * (a @ np.abs(v)) + floor * a.max() * np.abs(v).sum(axis=0)


def decode(q, pool, block_table, seqlens, lam, lam_init, norm_weight=None, eps=1e-5, norm=True,
           apply_scale=True, k_exp=0, v_exp=0, slack=0.0, floor=0.0):
    """V1 decode over a pool: q [B, H, 256]. Returns (out, bound) [B, H, 256]: `bound` is how far an
    output may be off where every product p * v of both maps carries a relative error of `slack` and
    every p an absolute one of `floor` times the map's largest (propagated through the norm), before
    the output's own rounding."""
    q = ref._f64(q)
    B, H, _ = q.shape
    out, bound = np.zeros((B, H, 256)), np.zeros((B, H, 256))
    for b in range(B):
        if seqlens[b] == 0:
            continue
        k, v = sequence_rows(pool, 2, block_table, b, int(seqlens[b]), 0, k_exp, v_exp)
        for h in range(H):
            a1, a2 = _weights(q[b, h, :128], k[:, h, :128]), _weights(q[b, h, 128:], k[:, h, 128:])
            o = a1 @ v[:, h] - lam[h] * (a2 @ v[:, h])
            e = _off(a1, v[:, h], slack, floor) + abs(lam[h]) * _off(a2, v[:, h], slack, floor)
            y = ref.head_epilogue(o[None], norm_weight, eps, lam_init, norm, apply_scale)[0]
            g = np.ones(256) if norm_weight is None or not norm else np.abs(ref._f64(norm_weight))
            g = g * (abs(1 - lam_init) if apply_scale else 1.0)
            if norm:  # y = g o / rms(o): its change is at most g (e + |o| |e| / |o|_2) / rms, to first order
                rms = np.sqrt(np.mean(o * o) + eps)
                e = (e + np.abs(o) * np.linalg.norm(e) / (np.sqrt(256) * rms)) / rms * 1.05
            out[b, h], bound[b, h] = y, g * e
    return out, bound


def v2_decode(q, pool, block_table, seqlens, lam_logit, k_exp=0, v_exp=0, slack=0.0, floor=0.0):
    """V2 decode over a pool: q [B, Hq, 128]. Returns (out, bound) [B, Hq/2, 128] as above."""
    q = ref._f64(q)
    B, Hq, _ = q.shape
    G = Hq // pool.shape[1]
    sig = ref.sigmoid(lam_logit)
    out, bound = np.zeros((B, Hq // 2, 128)), np.zeros((B, Hq // 2, 128))
    for b in range(B):
        if seqlens[b] == 0:
            continue
        k, v = sequence_rows(pool, 1, block_table, b, int(seqlens[b]), 0, k_exp, v_exp)
        for p in range(Hq // 2):
            h = 2 * p // G
            a = [_weights(q[b, 2 * p + r], k[:, h]) for r in (0, 1)]
            out[b, p] = a[0] @ v[:, h] - sig[b, p] * (a[1] @ v[:, h])
            off = [_off(x, v[:, h], slack, floor) for x in a]
            bound[b, p] = off[0] + sig[b, p] * off[1]
    return out, bound


def _chunk_weights(q, k, n, length, causal):
    """softmax weights [n, length] of the last n of `length` positions; rows that see no key are zeros."""
    s = (q @ k.T) / np.sqrt(q.shape[1])
    if causal:
        s = np.where(np.arange(length)[None] <= length - n + np.arange(n)[:, None], s, -np.inf)
    top = s.max(axis=1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    total = p.sum(axis=1, keepdims=True)
    return np.divide(p, total, out=np.zeros_like(p), where=total > 0)


def _off_rows(a, v, slack, floor):
    """_off of every row of a, over the keys that the row sees."""
    seen = (a > 0).astype(np.float64)
    return slack * (a @ np.abs(v)) + floor * a.max(axis=1, initial=0.0)[:, None] * (seen @ np.abs(v))


def fwd(q, pool, block_table, cu, seqlens, lam, lam_init, norm_weight=None, eps=1e-5, causal=True, norm=True, apply_scale=True,
        k_exp=0, v_exp=0, slack=0.0, floor=0.0):
    """V1 chunks over a pool: q [total, H, 256], sequence b's rows cu[b] .. cu[b + 1] - 1 being the last of its
    seqlens[b] positions. Returns (out, bound) [total, H, 256] as `decode` does; rows in no sequence are NaN."""
    q = ref._f64(q)
    total, H, _ = q.shape
    out, bound = np.full((total, H, 256), np.nan), np.zeros((total, H, 256))
    for b, length in enumerate(int(n) for n in seqlens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        n = rows.stop - rows.start
        if n == 0:
            continue
        if length == 0:
            out[rows] = 0.0
            continue
        k, v = sequence_rows(pool, 2, block_table, b, length, 0, k_exp, v_exp)
        for h in range(H):
            a = [_chunk_weights(q[rows, h, 128 * m:128 * m + 128], k[:, h, 128 * m:128 * m + 128], n, length, causal) for m in (0, 1)]
            o = a[0] @ v[:, h] - lam[h] * (a[1] @ v[:, h])
            e = _off_rows(a[0], v[:, h], slack, floor) + abs(lam[h]) * _off_rows(a[1], v[:, h], slack, floor)
            y = ref.head_epilogue(o, norm_weight, eps, lam_init, norm, apply_scale)
            g = np.ones(256) if norm_weight is None or not norm else np.abs(ref._f64(norm_weight))
            g = g * (abs(1 - lam_init) if apply_scale else 1.0)
            if norm:
                rms = np.sqrt(np.mean(o * o, axis=1, keepdims=True) + eps)
                e = (e + np.abs(o) * np.linalg.norm(e, axis=1, keepdims=True) / (np.sqrt(256) * rms)) / rms * 1.05
            out[rows, h], bound[rows, h] = y, g * e
    return out, bound


def v2_fwd(q, pool, block_table, cu, seqlens, lam_logit, causal=True, k_exp=0, v_exp=0, slack=0.0, floor=0.0):
    """V2 chunks over a pool: q [total, Hq, 128]. Returns (out, bound) [total, Hq/2, 128] as above."""
    q = ref._f64(q)
    total, Hq, _ = q.shape
    G = Hq // pool.shape[1]
    sig = ref.sigmoid(lam_logit)
    out, bound = np.full((total, Hq // 2, 128), np.nan), np.zeros((total, Hq // 2, 128))
    for b, length in enumerate(int(n) for n in seqlens):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        n = rows.stop - rows.start
        if n == 0:
            continue
        if length == 0:
            out[rows] = 0.0
            continue
        k, v = sequence_rows(pool, 1, block_table, b, length, 0, k_exp, v_exp)
        for p in range(Hq // 2):
            h = 2 * p // G
            a = [_chunk_weights(q[rows, 2 * p + r], k[:, h], n, length, causal) for r in (0, 1)]
            g = sig[rows, p][:, None]
            out[rows, p] = a[0] @ v[:, h] - g * (a[1] @ v[:, h])
            off = [_off_rows(x, v[:, h], slack, floor) for x in a]
            bound[rows, p] = off[0] + g * off[1]
    return out, bound
