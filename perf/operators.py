"""What is measured of the 4-bit cache: its operators' cases, inputs, plain forms and exact values.

The operators are those of one serving step over a key/value cache held in 4 bits: the plan that turns
request lengths into block tables and slot maps, the write of new rows into the pages, the read of
cached rows back into packed bf16, and the decode attentions (V1 and V2) over the pages.

The cache's format: 16 channels of one row share an e4m3 scale s and hold e2m1 codes c, and stand for
c * s. The pool is uint8 [num_pages, heads, page_size / 16, record]; a record holds 16 tokens of one
head as planes of 128 channels, the K planes first (V1: K1, K2, V's two halves; V2: K, V), each plane
1024 bytes of codes and 128 bytes of scales. Inside a plane the bytes are ordered
    K codes  [2 h][4 a][2 r][4 t][16 n]   key 4a + 2h + r, channels 32t + 2n (low nibble), + 1 (high)
    K scales [4 a][2 r][4 t][2 h][2 u]    the same key, channels 32t + 16u ..
    V codes  [2 i][8 g][4 t][2 j][8 n]    key 4t + 2i + j, channels 16g + 2n (low nibble), + 1 (high)
    V scales [8 g][4 t][4 i]              key 4t + i, channels 16g ..
"""
import math
import random

import torch

own = False

EPS = 1e-5
LAMBDA_INIT = 0.5


def _da():
    import differential_attention_gb300 as da
    return da


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a full server: every request gets one token, a few have ended
        {"name": "plan_step", "op": "plan", "B": 256, "ended": 8, "cached": 32768, "new": 1, "page": 64},
        # a prefill step: many prompts of all lengths enter at once, small pages
        {"name": "plan_prompts", "op": "plan", "B": 48, "ended": 3, "cached": 700, "new": 9000, "page": 16},
        # the rows of one decoding step written (and read back): one token of each of 64 requests
        {"name": "write_step_v2", "op": "write", "form": "v2", "B": 64, "H": 8, "new": 1, "cached": 5000, "page": 64},
        # prompts written from views of one fused q, k, v projection, and read back for their attention
        {"name": "write_prompts_v1", "op": "write", "form": "v1", "B": 8, "H": 12, "new": 2048, "cached": 37, "page": 32},
        # the cached keys of a few long chats, read for the next chunk of their prompts
        {"name": "read_chats_v2", "op": "read", "form": "v2", "B": 6, "H": 8, "L": 8190, "page": 64},
        # four prompts of 4096 tokens read back whole
        {"name": "read_prompts_v1", "op": "read", "form": "v1", "B": 4, "H": 12, "L": 4096, "page": 128},
        # one short chat: latency counts
        {"name": "v2_one_short", "op": "v2", "B": 1, "Hkv": 8, "G": 8, "L": 777, "ragged": False, "page": 16},
        # a mixed batch: lengths from one token to 16K, some slots of the batch empty
        {"name": "v2_mixed", "op": "v2", "B": 96, "Hkv": 8, "G": 4, "L": 16384, "ragged": True, "page": 48},
        # the long-context decode of the benchmark's V2 shape
        {"name": "v2_32k", "op": "v2", "B": 64, "Hkv": 8, "G": 8, "L": 32768, "ragged": False, "page": 64},
        # a small batch of short chats, V1
        {"name": "v1_few_short", "op": "v1", "B": 4, "H": 12, "L": 1500, "ragged": False, "page": 16},
        # a mixed batch, V1
        {"name": "v1_mixed", "op": "v1", "B": 48, "H": 12, "L": 9001, "ragged": True, "page": 64},
        # the benchmark's V1 heads over 32K tokens
        {"name": "v1_32k", "op": "v1", "B": 24, "H": 12, "L": 32768, "ragged": False, "page": 128},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["plan", "write", "read", "v2", "v2", "v1", "v1"])
    page = 16 * rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op == "plan":
        B = _log(rng, 1, 512)
        return {"op": op, "B": B, "ended": rng.randint(0, B // 3), "cached": _log(rng, 1, 32768),
                "new": _log(rng, 1, max(1, min(4096, 32768 // B))), "page": page}
    if op in ("write", "read"):
        form = rng.choice(["v1", "v2"])
        H = rng.randint(1, 16) if form == "v1" else rng.choice([1, 2, 3, 4, 5, 8])
        cap = 16384 * 12 // H // (1 if form == "v1" else 2)  # tokens: no more than write_prompts_v1
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(1, min(8192, cap // B)))
        if op == "write":
            return {"op": op, "form": form, "B": B, "H": H, "new": n, "cached": rng.randint(0, 3000), "page": page}
        return {"op": op, "form": form, "B": B, "H": H, "L": n, "page": page}
    if op == "v2":
        Hkv, G = rng.choice([1, 2, 3, 4, 8]), rng.choice([2, 4, 8])
        B = _log(rng, 1, 128)
        L = _log(rng, 1, max(1, min(65536, 64 * 8 * 32768 // (Hkv * B))))
        return {"op": op, "B": B, "Hkv": Hkv, "G": G, "L": L, "ragged": rng.random() < 0.5, "page": page}
    H, B = rng.randint(1, 16), _log(rng, 1, 128)
    L = _log(rng, 1, max(1, min(65536, 24 * 12 * 32768 // (H * B))))
    return {"op": op, "B": B, "H": H, "L": L, "ragged": rng.random() < 0.5, "page": page}


def _planes(form):
    return (2, 2) if form == "v1" else (1, 1)


def _spread(case, top, count, key):
    """`count` lengths from 1 to `top`, spread over their logarithm; they go by the case alone."""
    rng = random.Random("%s %d %d" % (key, top, count))
    return [_log(rng, 1, top) for _ in range(count)]


def _lens(case):
    """Cached tokens of each sequence of a decode or a read. Of a ragged batch the first is the
    longest, and one slot in sixteen is empty."""
    B, L = case["B"], case["L"]
    if case["op"] == "read":
        return [max(1, L - 13 * i) for i in range(B)]
    if not case["ragged"]:
        return [L] * B
    return [L] + [0 if i % 16 == 15 else n for i, n in enumerate(_spread(case, L, B, "len")) if i]


def _plan_lengths(case):
    """(cached tokens, new tokens or -1 where the request has ended) of each request."""
    B = case["B"]
    old = _spread(case, case["cached"], B, "old")
    new = [1] * B if case["new"] == 1 else [(n * 2) // 3 + 1 for n in _spread(case, 2 * case["new"], B, "new")]
    out = {(i * 7919 + 3) % B for i in range(case["ended"])}
    return old, [-1 if i in out else n for i, n in enumerate(new)]


def _write_lengths(case):
    """(cached tokens, new tokens) of each sequence of a write."""
    B, n = case["B"], case["new"]
    return [(case["cached"] * (i + 1)) // B for i in range(B)], [max(1, n - 5 * (i % 7)) if n > 1 else 1 for i in range(B)]


# ---------------------------------------------------------------------------------------------
# the format, in elementary operations
# ---------------------------------------------------------------------------------------------
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x):
    """Rows x [..., 16 * n] to (code bytes uint8 [..., 8 * n], e4m3 scales [..., n]): s = amax / 6
    rounded to e4m3 (448 at most), c = x / s rounded to e2m1, ties to the even code. A bf16 has 8
    significant bits, s has 4 and a border of e2m1 has 3, so a quotient off a border is off by far
    more than 32 bits round: every decision is the exact one."""
    x = x.float().unflatten(-1, (-1, 16))
    top = x.abs().amax(-1)
    s = (top / torch.full_like(top, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)  # a true division, no product with 1/6
    f = s.float()[..., None]
    y = torch.where(f > 0, x.abs() / f, torch.zeros_like(x))
    c = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    c = c + 8 * (x < 0)
    c = c.to(torch.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(-2), s


def _value_table(device):
    pos = torch.tensor(E2M1, dtype=torch.float32, device=device)
    one = torch.cat([pos, -pos])
    return torch.stack([one.repeat(16), one.repeat_interleave(16)], dim=-1)  # [256, 2]: low, high nibble


def _unpack(rec, kp, vp):
    """Records uint8 [..., bytes] to K [..., 16, 128 kp] and V [..., 16, 128 vp] in fp32."""
    lead, n = rec.shape[:-1], rec.dim() - 1
    at = lambda *dims: tuple(range(n)) + tuple(n + d for d in dims)  # noqa: E731
    table = _value_table(rec.device)
    planes = rec.unflatten(-1, (kp + vp, 1152))
    codes, scales = planes[..., :1024], planes[..., 1024:].contiguous().view(torch.float8_e4m3fn).float()
    # each permuted to key (a h r / t i j), plane, block of 16, values of the block
    k = table[codes[..., :kp, :].unflatten(-1, (2, 4, 2, 4, 2, 8)).int()]         # p h a r t u n 2
    k = k.permute(at(2, 1, 3, 0, 4, 5, 6, 7)).reshape(*lead, 16, kp * 8, 16)
    ks = scales[..., :kp, :].unflatten(-1, (4, 2, 4, 2, 2))                       # p a r t h u
    ks = ks.permute(at(1, 4, 2, 0, 3, 5)).reshape(*lead, 16, kp * 8, 1)
    v = table[codes[..., kp:, :].unflatten(-1, (2, 8, 4, 2, 8)).int()]            # p i g t j n 2
    v = v.permute(at(3, 1, 4, 0, 2, 5, 6)).reshape(*lead, 16, vp * 8, 16)
    vs = scales[..., kp:, :].unflatten(-1, (8, 4, 4))                             # p g t i
    vs = vs.permute(at(2, 3, 0, 1)).reshape(*lead, 16, vp * 8, 1)
    return (k * ks).flatten(-2), (v * vs).flatten(-2)


def _pack(k, v, kp, vp):
    """K [..., 16, 128 kp] and V [..., 16, 128 vp] to records (the inverse of _unpack)."""
    lead, n = k.shape[:-2], k.dim() - 2
    at = lambda *dims: tuple(range(n)) + tuple(n + d for d in dims)  # noqa: E731
    c, s = _quantize(k)
    c = c.reshape(*lead, 4, 2, 2, kp, 64).permute(at(3, 1, 0, 2, 4)).reshape(*lead, kp, 1024)
    s = s.view(torch.uint8).reshape(*lead, 4, 2, 2, kp, 4, 2).permute(at(3, 0, 2, 4, 1, 5)).reshape(*lead, kp, 128)
    kb = torch.cat([c, s], dim=-1).flatten(-2)
    c, s = _quantize(v)
    c = c.reshape(*lead, 4, 2, 2, vp, 8, 8).permute(at(3, 1, 4, 0, 2, 5)).reshape(*lead, vp, 1024)
    s = s.view(torch.uint8).reshape(*lead, 4, 4, vp, 8).permute(at(2, 3, 0, 1)).reshape(*lead, vp, 128)
    return torch.cat([kb, torch.cat([c, s], dim=-1).flatten(-2)], dim=-1)


def _keys(pool, table, kp, vp):
    """K [B, H, L, 128 kp] and V of every page of `table` [B, pages], in order."""
    rec = pool[table.long()]                                                    # B pages H R bytes
    B, pages, H, R, n = rec.shape
    k, v = _unpack(rec.permute(0, 2, 1, 3, 4).reshape(B, H, pages * R, n), kp, vp)
    return k.flatten(2, 3), v.flatten(2, 3)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _rows(shape, gen, dev):
    """Rows as projections give them: normal values, some channels several times as large."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
    loud = 1.0 + 3.0 * (torch.rand(shape[-1], generator=gen, device=dev) < 0.06)
    return x * loud.to(torch.bfloat16)


def _tables(lens, page, spare, gen, dev):
    """Block tables [B, max_pages] over a shuffled pool with `spare` pages in no sequence."""
    used = [-(-n // page) for n in lens]
    width = max(1, max(used))
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=dev)
    starts = torch.tensor([sum(used[:i]) for i in range(len(lens))], device=dev)
    at = starts[:, None] + torch.arange(width, device=dev)[None]
    mine = torch.arange(width, device=dev)[None] < torch.tensor(used, device=dev)[:, None]
    table[mine] = order[at[mine]]
    return table, pages


def _offsets(counts, dev):
    return torch.tensor([sum(counts[:i]) for i in range(len(counts) + 1)], dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"op": op, "page": case["page"]}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if op == "plan":
        old, new = _plan_lengths(case)
        page = case["page"]
        used = [-(-n // page) for n in old]
        after = [0 if m < 0 else n + m for n, m in zip(old, new)]
        total = sum(m for m in new if m > 0)
        # the ring holds more free pages than the step needs; its head is anywhere
        spare = sum(-(-n // page) for n in after) + 100
        table, pages = _tables(old, page, spare, gen, dev)
        width = max(max(-(-n // page) for n in after), table.shape[1]) + 4
        wide = torch.full((len(old), width), -1, dtype=torch.int32, device=dev)
        wide[:, :table.shape[1]] = table
        taken = torch.zeros(pages, dtype=torch.bool, device=dev)
        live = torch.arange(table.shape[1], device=dev)[None] < torch.tensor(used, device=dev)[:, None]
        taken[table[live].long()] = True
        free = torch.nonzero(~taken).flatten().to(torch.int32)
        free = free[torch.randperm(free.numel(), generator=gen, device=dev)]
        head = int(torch.randint(0, pages, (1,), generator=gen, device=dev).item())
        ring = torch.zeros(pages, dtype=torch.int32, device=dev)
        ring[(head + torch.arange(free.numel(), device=dev)) % pages] = free
        s.update(seqlens=ints(old), new=ints(new), table=wide, ring=ring,
                 state=ints([head, free.numel()]), total_max=total + 7)
        return s
    form = case.get("form", op)
    kp, vp = _planes(form)
    H = case["Hkv"] if op == "v2" else case["H"]
    s.update(form=form, kp=kp, vp=vp)
    if op == "write":
        old, new = _write_lengths(case)
        both = [a + b for a, b in zip(old, new)]
        table, pages = _tables(both, case["page"], 5, gen, dev)
        total = sum(new)
        # the rows are views of one projection [token, (q, k, v), head, width], two padding rows behind
        proj = _rows((total + 2, 3, H, 128 * kp), gen, dev)
        seq = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev))
        cu = _offsets(new, dev)
        pos = torch.arange(total, device=dev) - cu[seq].long() + torch.tensor(old, device=dev)[seq]
        slots = table[seq, pos // case["page"]].long() * case["page"] + pos % case["page"]
        slots = torch.cat([slots, torch.full((2,), -1, device=dev)]).to(torch.int32)
        pool = torch.zeros((pages, H, case["page"] // 16, 1152 * (kp + vp)), dtype=torch.uint8, device=dev)
        s.update(k=proj[:, 1], v=proj[:, 2], slots=slots, pool=pool, table=table, cu=cu, starts=ints(old),
                 total=total, width=128 * kp)
        return s
    lens = _lens(case)
    table, pages = _tables(lens, case["page"], 3, gen, dev)
    R = case["page"] // 16
    pool = torch.empty((pages, H, R, 1152 * (kp + vp)), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 19) // (H * case["page"]))
    for at in range(0, pages, step):  # rounded rows in every page, a few pages at a time
        n = min(step, pages - at)
        v = torch.randn((n, H, R, 16, 128 * vp), generator=gen, device=dev, dtype=torch.bfloat16)
        pool[at:at + n] = _pack(_rows((n, H, R, 16, 128 * kp), gen, dev), v, kp, vp)
    s.update(pool=pool, table=table, seqlens=ints(lens))
    if op == "read":
        s.update(cu=_offsets(lens, dev), total=sum(lens), width=128 * kp)
        return s
    B = case["B"]
    norm = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    if op == "v2":
        s["q"] = norm(B, H * case["G"], 128).to(torch.bfloat16)
        s["lam"] = norm(B, H * case["G"] // 2)
        s["G"] = case["G"]
    else:
        s["q"] = norm(B, H, 256).to(torch.bfloat16)
        s["lam"] = 0.2 + 0.6 * torch.rand(H, generator=gen, device=dev)
        s["weight"] = 1.0 + 0.1 * norm(256)
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        da = _da()
        if op == "plan":
            p = da.diffattn_paged_plan(s["seqlens"], s["new"], s["table"], s["ring"], s["state"], s["page"], s["total_max"])
            return {**p, "block_table": s["table"], "free_ring": s["ring"]}
        if op == "write":
            da.diffattn_kv4_append(s["k"], s["v"], s["slots"], s["pool"])
            return da.diffattn_kv4_gather(s["pool"], s["table"], s["cu"], s["total"], s["width"], s["width"], starts=s["starts"])
        if op == "read":
            return da.diffattn_kv4_gather(s["pool"], s["table"], s["cu"], s["total"], s["width"], s["width"])
        if op == "v2":
            return da.diffattn_v2_decode_kv4(s["q"], s["pool"], s["table"], s["seqlens"], s["lam"])
        return da.diffattn_decode_kv4(s["q"], s["pool"], s["table"], s["seqlens"], s["lam"], LAMBDA_INIT,
                                      norm_weight=s["weight"], eps=EPS)
    if op == "plan":
        return _plain_plan(s)
    if op == "write":
        _plain_append(s)
        return _plain_gather(s, s["starts"].long())
    if op == "read":
        return _plain_gather(s, torch.zeros_like(s["seqlens"]).long())
    return _plain_v2(s) if op == "v2" else _plain_v1(s)


def _plain_plan(s):
    page, ring, table = s["page"], s["ring"], s["table"]
    old, n = s["seqlens"].long(), s["new"].long()
    head, count = s["state"].long()
    dev, B = old.device, old.numel()
    ended = n < 0
    new = n.clamp(min=0)
    after = torch.where(ended, torch.zeros_like(old), old + new)
    have = (old + page - 1) // page
    need = torch.where(ended, torch.zeros_like(old), (after + page - 1) // page - have)
    freed = torch.where(ended, have, torch.zeros_like(old))
    ids, zero = torch.arange(B, device=dev), old.new_zeros(1)
    before = lambda v: torch.cat([zero, v.cumsum(0)])  # noqa: E731
    # pages of ended requests go behind the free ones, in order
    who = torch.repeat_interleave(ids, freed)
    back = table[who, torch.arange(who.numel(), device=dev) - before(freed)[who]]
    ring[(head + count + torch.arange(back.numel(), device=dev)) % ring.numel()] = back
    # the pages that requests grow into come from the front
    who = torch.repeat_interleave(ids, need)
    nth = torch.arange(who.numel(), device=dev)
    table[who, have[who] + nth - before(need)[who]] = ring[(head + nth) % ring.numel()]
    # slots and positions of the new tokens, and -1 behind the last
    cu = before(new)
    who = torch.repeat_interleave(ids, new)
    pos = old[who] + torch.arange(who.numel(), device=dev) - cu[who]
    fill = torch.full((s["total_max"] - who.numel(),), -1, device=dev)
    slots = table[who, pos // page].long() * page + pos % page
    state = torch.stack([(head + need.sum()) % ring.numel(), count + freed.sum() - need.sum()])
    keys = torch.where(new > 0, after, torch.zeros_like(after))
    out = {"seqlens": after, "ring_state": state, "cu_seqlens_q": cu, "cu_seqlens_k": before(keys),
           "slot_map": torch.cat([slots, fill]), "positions": torch.cat([pos, fill])}
    return {**{k: v.to(torch.int32) for k, v in out.items()}, "block_table": table, "free_ring": ring}


def _plain_append(s):
    """Each row's codes and scales to their places in the records of its slot."""
    kp, vp, pool = s["kp"], s["vp"], s["pool"]
    R = pool.shape[2]
    keep = s["slots"] >= 0
    slot = s["slots"][keep].long()
    page, rec, key = slot // (16 * R), slot % (16 * R) // 16, slot % 16
    a, h, r = key // 4, key % 4 // 2, key % 2
    planes = pool.unflatten(-1, (kp + vp, 1152))
    codes, scales = planes[..., :1024], planes[..., 1024:]
    c, sc = _quantize(s["k"][keep])                                              # token H bytes
    codes[..., :kp, :].unflatten(-1, (2, 4, 2, 64)).movedim(-5, -2)[page, :, rec, h, a, r] = c.unflatten(-1, (kp, 64))
    to = scales[..., :kp, :].unflatten(-1, (4, 2, 4, 2, 2)).movedim(-6, -4).movedim(-2, -5)  # P H R a h r p t u
    to[page, :, rec, a, h, r] = sc.view(torch.uint8).unflatten(-1, (kp, 4, 2))
    c, sc = _quantize(s["v"][keep])
    to = codes[..., kp:, :].unflatten(-1, (2, 8, 4, 2, 8)).movedim((-6, -4), (-3, -2))       # P H R i t j p g n
    to[page, :, rec, h, a, r] = c.unflatten(-1, (vp, 8, 8))
    to = scales[..., kp:, :].unflatten(-1, (8, 4, 4)).movedim((-4, -3), (-2, -1))             # P H R t i p g
    to[page, :, rec, a, key % 4] = sc.view(torch.uint8).unflatten(-1, (vp, 8))


def _plain_gather(s, starts):
    """Rows starts[b] .. of each sequence b, one behind the other: (K [total, H, .], V)."""
    cu, R = s["cu"].long(), s["pool"].shape[2]
    who = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=cu.device), cu[1:] - cu[:-1])
    pos = starts[who] + torch.arange(who.numel(), device=cu.device) - cu[who]
    page, rec, key = s["table"][who, pos // (16 * R)].long(), pos % (16 * R) // 16, pos % 16
    # each record that holds a wanted row once
    at, row = torch.unique(page * R + rec, return_inverse=True)
    k, v = _unpack(s["pool"][at // R, :, at % R], s["kp"], s["vp"])              # n H 16 width
    return k[row, :, key].to(torch.bfloat16), v[row, :, key].to(torch.bfloat16)


def _softmax_v(score, v, lens):
    """softmax over the first lens[b] keys of score [B, H, rows, L], times v [B, H, L, w]; 0 for no keys."""
    seen = (torch.arange(score.shape[-1], device=v.device)[None] < lens[:, None])[:, None, None]
    top = torch.where(seen, score, torch.full_like(score, -1e30)).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - top), torch.zeros_like(score))
    return (p @ v) / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_v2(s):
    k, v = _keys(s["pool"], s["table"], 1, 1)
    B, Hkv, G = k.shape[0], k.shape[1], s["G"]
    q = s["q"].float().view(B, Hkv, G, 128) / math.sqrt(128)
    o = _softmax_v(q @ k.transpose(-1, -2), v, s["seqlens"]).reshape(B, Hkv * G // 2, 2, 128)
    return (o[:, :, 0] - torch.sigmoid(s["lam"])[..., None] * o[:, :, 1]).to(torch.bfloat16)


def _plain_v1(s):
    k, v = _keys(s["pool"], s["table"], 2, 2)
    q = s["q"].float() / math.sqrt(128)
    B, H = q.shape[:2]
    score = (k.unflatten(-1, (2, 128)) * q.view(B, H, 1, 2, 128)).sum(-1).transpose(-1, -2)  # B H 2 L
    o = _softmax_v(score, v, s["seqlens"])
    o = o[:, :, 0] - s["lam"][None, :, None] * o[:, :, 1]
    o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"]
    return (o * (1.0 - LAMBDA_INIT)).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "plan":
        old, new = _plan_lengths(case)
        page, total, B = case["page"], sum(m for m in new if m > 0), case["B"]
        up = lambda n: -(-n // page)  # noqa: E731
        taken = sum(up(n + m) - up(n) for n, m in zip(old, new) if m > 0)
        back = sum(up(n) for n, m in zip(old, new) if m < 0)
        # lengths in; lengths, offsets, slots and positions out; each page that moves read and written
        return {"bytes": 8 * B + 12 * B + 8 * (total + 7) + 8 * (taken + back) + 24, "flops": 0}
    form = case.get("form", op)
    wide = sum(_planes(form)) * 128
    if op == "write":  # rows read, codes written and read, rows written
        n = sum(_write_lengths(case)[1]) * case["H"]
        return {"bytes": n * wide * (2 + 0.5625 + 0.5625 + 2), "flops": 0}
    if op == "read":
        n = sum(_lens(case)) * case["H"]
        return {"bytes": n * wide * (0.5625 + 2), "flops": 0}
    keys = sum(_lens(case))
    if op == "v2":
        n, rows = keys * case["Hkv"], case["B"] * case["Hkv"] * case["G"]
        return {"bytes": n * 144 + rows * (256 + 128 + 2), "flops": n * 4 * 128 * case["G"]}
    n, rows = keys * case["H"], case["B"] * case["H"]
    return {"bytes": n * 288 + rows * 1024, "flops": n * (4 * 128 + 4 * 256)}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits, written apart from the above
# ---------------------------------------------------------------------------------------------
def _grid(bits, man, bias, dev):
    """The non-negative values of a small float type, in the order of their codes."""
    parts = [(c >> man, (c & ((1 << man) - 1)) / (1 << man)) for c in range(1 << bits)]
    return torch.tensor([m * 2.0 ** (1 - bias) if e == 0 else (1 + m) * 2.0 ** (e - bias) for e, m in parts],
                        dtype=torch.float64, device=dev)


def _nearest(x, grid):
    """The index of the grid's value nearest to x >= 0; of two as near, the even index."""
    i = torch.searchsorted(grid, x).clamp(1, grid.numel() - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    return torch.where((lo < hi) | ((lo == hi) & (i % 2 == 1)), i - 1, i)


def _round64(x):
    """What 16 channels of x stand for once they are held in 4 bits."""
    x = x.double().unflatten(-1, (-1, 16))
    scales = _grid(7, 3, 7, x.device)[:127]
    top = x.abs().amax(-1)
    s = scales[_nearest(top / torch.full_like(top, 6.0), scales)][..., None]
    codes = _grid(3, 1, 1, x.device)
    c = codes[_nearest(x.abs() / torch.where(s > 0, s, torch.ones_like(s)), codes)]
    return (torch.sign(x) * c * s).flatten(-2)


def _read64(records, kp, vp, key):
    """K and V of row `key` of each record [n, bytes], in 64 bits, byte by byte."""
    dev = records.device
    two = _grid(3, 1, 1, dev)
    two = torch.cat([two, -two])
    eight = _grid(7, 3, 7, dev)
    ch = torch.arange(128, device=dev)

    def plane(p, code_at, scale_at):
        byte = torch.gather(records, 1, 1152 * p + code_at).int()
        c = two[torch.where(ch % 2 == 0, byte & 15, byte >> 4)]
        return c * eight[torch.gather(records, 1, 1152 * p + 1024 + scale_at).int()]

    key = key[:, None]
    a, h, r = key // 4, key % 4 // 2, key % 2
    t, n = ch // 32, ch % 32 // 2
    k = [plane(p, h * 512 + a * 128 + r * 64 + t * 16 + n, a * 32 + r * 16 + t * 4 + h * 2 + ch % 32 // 16) for p in range(kp)]
    g, n = ch // 16, ch % 16 // 2
    v = [plane(kp + p, h * 512 + g * 64 + a * 16 + r * 8 + n, g * 16 + a * 4 + key % 4) for p in range(vp)]
    return torch.cat(k, -1), torch.cat(v, -1)


def _keys64(s, b, heads, lo, hi):
    """Keys lo .. hi - 1 of one sequence, [heads, hi - lo, width]."""
    pos = torch.arange(lo, hi, device=s["pool"].device)
    page, off = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    rec = s["pool"][page, :, off // 16]                                          # n H bytes
    n = rec.shape[0]
    k, v = _read64(rec.transpose(0, 1).reshape(heads * n, -1), s["kp"], s["vp"], (off % 16).repeat(heads))
    return k.view(heads, n, -1), v.view(heads, n, -1)


def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None  # whole numbers
    s = prepare(case, seed)
    if op == "write":
        rows = s["total"]
        return _round64(s["k"][:rows]), _round64(s["v"][:rows])
    lens = _lens(case)
    H = s["pool"].shape[1]
    if op == "read":
        parts = [_keys64(s, b, H, 0, n) for b, n in enumerate(lens)]
        return tuple(torch.cat([p[i].transpose(0, 1) for p in parts]) for i in (0, 1))
    out = []
    for b, n in enumerate(lens):
        q = s["q"][b].double()
        if op == "v2":
            q = q.view(H, case["G"], 128)
        else:  # two maps, each over its half of the keys' channels
            q = torch.stack([torch.cat([q[:, :128], 0 * q[:, :128]], -1), torch.cat([0 * q[:, 128:], q[:, 128:]], -1)], 1)
        if n == 0:
            o = q.new_zeros((H, q.shape[1], 128 * s["vp"]))
        else:
            # a softmax over pieces of the keys: exponents against a bound on the scores, then one division
            k, v = zip(*[_keys64(s, b, H, lo, min(n, lo + 8192)) for lo in range(0, n, 8192)])
            score = torch.cat([torch.einsum("hgd,hnd->hgn", q, x) for x in k], -1) * 128 ** -0.5
            p = torch.softmax(score, -1).split([x.shape[1] for x in k], -1)
            o = sum(torch.einsum("hgn,hnd->hgd", x, y) for x, y in zip(p, v))
        if op == "v2":
            o = o.view(H * case["G"] // 2, 2, 128)
            out.append(o[:, 0] - torch.sigmoid(s["lam"][b].double())[:, None] * o[:, 1])
        else:
            o = o[:, 0] - s["lam"].double()[:, None] * o[:, 1]
            o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
            out.append((1 - LAMBDA_INIT) * o)
    return torch.stack(out)
