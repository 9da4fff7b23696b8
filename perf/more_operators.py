"""What is measured of rotary positions and of chunks over the 4-bit cache: cases, inputs, plain forms, exact values.

The operators are those of a step that extends sequences: the rotation of queries and keys by positions of one
or several axes (and its backward pass, the rotation back), the write of rotated keys and of values into pages,
in bf16 or in 4 bits, and the attention (V1 and V2) of each sequence's new tokens over its 4-bit pages.

Rotation. A row of a head is made of parts of d channels (V1: the two halves of a query or key; V2: one part);
the first 2 P channels of a part are P pairs, channels i and i + P, or 2 i and 2 i + 1 (interleaved). Pair i of a
token is turned by the angle whose cosine and sine are table[position, i], the position being the token's on axis
axes[i] (time, height, width):
    y1 = x1 cos - x2 sin,   y2 = x2 cos + x1 sin      (backward: sin negated).
A bf16 result is the exact value rounded once. A token at position -1 is left out.

Pages. Row t of k and v goes to slot slots[t] = page * page_size + offset; -1 is left out. In 4 bits, the rotated
key is rounded to bf16 first, then as the cache's format says: 16 channels share an e4m3 scale s = e4m3(amax / 6)
and hold e2m1 codes c = e2m1(x / s), and stand for c * s. The pool is uint8 [num_pages, heads, page_size / 16,
record]; a record holds 16 tokens of one head as planes of 128 channels, the K planes first (V1: K1, K2, V's two
halves; V2: K, V), each plane 1024 bytes of codes and 128 bytes of scales:
    K codes  [2 h][4 a][2 r][4 t][16 n]   key 4a + 2h + r, channels 32t + 2n (low nibble), + 1 (high)
    K scales [4 a][2 r][4 t][2 h][2 u]    the same key, channels 32t + 16u ..
    V codes  [2 i][8 g][4 t][2 j][8 n]    key 4t + 2i + j, channels 16g + 2n (low nibble), + 1 (high)
    V scales [8 g][4 t][4 i]              key 4t + i, channels 16g ..

Attention of a chunk. Sequence b has lens[b] cached tokens, of which its queries are the last new[b]: query i sees
keys 0 .. lens[b] - new[b] + i (causal), or all. V1: norm(softmax(Q1 K1) V - lambda softmax(Q2 K2) V) (1 - l0);
V2: softmax(Q_2p K) V - sigmoid(lam_p) softmax(Q_2p+1 K) V. Rows behind the last sequence stay as they were.
"""
import math
import random

import torch

own = False

EPS = 1e-5
LAMBDA_INIT = 0.5
FREE = 3  # rows behind the last sequence


def _da():
    import differential_attention_gb300 as da
    return da


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # the queries and keys of one decoding step of 64 requests, V2 heads
        {"name": "rope_step", "op": "rope", "total": 64, "hq": 64, "hk": 8, "parts": 1, "d": 128, "rot": 128, "axes": 1,
         "inter": False, "back": False, "fp32": False, "top": 32768},
        # the gradients of a training step's queries and keys rotated back: four sequences of 4096, V1 heads
        {"name": "rope_train_backward", "op": "rope", "total": 16384, "hq": 12, "hk": 12, "parts": 2, "d": 128, "rot": 128,
         "axes": 1, "inter": False, "back": True, "fp32": False, "top": 4096},
        # frames of a video with places in time, height and width, in fp32, neighbouring channels paired
        {"name": "rope_video_fp32", "op": "rope", "total": 3333, "hq": 8, "hk": 4, "parts": 1, "d": 64, "rot": 48, "axes": 3,
         "inter": True, "back": False, "fp32": True, "top": 1000},
        # the rows of one decoding step into bf16 pages, V1
        {"name": "append_step_v1", "op": "append", "form": "v1", "B": 64, "new": 1, "cached": 5000, "H": 12, "hq": 12,
         "page": 64, "rot": 128, "axes": 1, "inter": False},
        # prompts into bf16 pages, V2, positions of three axes (images among the text)
        {"name": "append_prompts_v2", "op": "append", "form": "v2", "B": 8, "new": 2050, "cached": 37, "H": 8, "hq": 64,
         "page": 128, "rot": 128, "axes": 3, "inter": False},
        # the rows of one decoding step into 4-bit pages, V2, and read back
        {"name": "append4_step_v2", "op": "append4", "form": "v2", "B": 64, "new": 1, "cached": 5000, "H": 8, "hq": 64,
         "page": 64, "rot": 128, "axes": 1, "inter": False},
        # prompts into 4-bit pages, V1, and read back
        {"name": "append4_prompts_v1", "op": "append4", "form": "v1", "B": 8, "new": 2048, "cached": 100, "H": 12, "hq": 12,
         "page": 32, "rot": 128, "axes": 1, "inter": False},
        # a few drafted tokens of one short chat are checked: latency counts
        {"name": "chunk_v2_one_short", "op": "v2", "B": 1, "Hkv": 8, "G": 8, "new": 5, "L": 777, "ragged": False, "page": 16,
         "causal": True},
        # drafted tokens of a batch of long chats checked at once
        {"name": "chunk_v2_verify_32k", "op": "v2", "B": 24, "Hkv": 8, "G": 8, "new": 8, "L": 32768, "ragged": False,
         "page": 64, "causal": True},
        # prompts of all lengths continued over what is cached of them, a few slots of the batch empty
        {"name": "chunk_v2_prompts", "op": "v2", "B": 20, "Hkv": 8, "G": 8, "new": 2048, "L": 16384, "ragged": True,
         "page": 64, "causal": True},
        # drafted tokens of a batch of chats, V1
        {"name": "chunk_v1_verify", "op": "v1", "B": 16, "H": 12, "new": 6, "L": 16384, "ragged": False, "page": 64,
         "causal": True},
        # the last quarter of four prompts of 4096 tokens, V1
        {"name": "chunk_v1_prompts", "op": "v1", "B": 4, "H": 12, "new": 1024, "L": 4096, "ragged": False, "page": 128,
         "causal": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "append4", "v2", "v2", "v1", "v1"])
    if op == "rope":
        d = rng.choice([64, 128])
        parts, fp32 = rng.choice([1, 2]), rng.random() < 0.3
        hq, hk = rng.randint(1, 16), rng.randint(0, 12)
        cap = 16384 * 24 * 256 // ((hq + hk) * parts * d * (2 if fp32 else 1))
        return {"op": op, "total": _log(rng, 1, min(60000, cap)), "hq": hq, "hk": hk, "parts": parts, "d": d,
                "rot": rng.choice([d, d, d // 2, 16 * rng.randint(1, d // 16)]), "axes": rng.choice([1, 1, 2, 3, 4]),
                "inter": rng.random() < 0.4, "back": rng.random() < 0.5, "fp32": fp32, "top": _log(rng, 1, 100000)}
    if op in ("append", "append4"):
        form = rng.choice(["v1", "v2"])
        H = rng.randint(1, 12) if form == "v1" else rng.choice([1, 2, 3, 4, 8])
        hq = H if form == "v1" else H * rng.choice([2, 4, 8])
        B = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, min(8192, 16384 * 24 * 256 // ((hq + 2 * H) * (256 if form == "v1" else 128) * B))))
        page = 16 * rng.choice([1, 2, 3, 4, 8, 16]) if op == "append4" else rng.choice([1, 7, 16, 64, 100, 128])
        return {"op": op, "form": form, "B": B, "new": new, "cached": rng.randint(0, 3000), "H": H, "hq": hq, "page": page,
                "rot": rng.choice([128, 128, 64, 32]), "axes": rng.choice([1, 1, 3]), "inter": rng.random() < 0.4}
    page = 16 * rng.choice([1, 2, 3, 4, 5, 8, 16])
    heads = rng.choice([1, 2, 3, 4, 8]) if op == "v2" else rng.randint(1, 12)
    G = rng.choice([2, 4, 8])
    B = _log(rng, 1, 64)
    new = _log(rng, 1, max(1, min(4096, 16384 // B)))
    keys = 24 * 8 * 32768 if op == "v2" else 16 * 12 * 16384
    flops = heads * B * new * (512 * G if op == "v2" else 1536)
    L = _log(rng, new, max(new, min(40000, keys // (heads * B), int(1.2e12 / flops))))
    case = {"op": op, "B": B, "new": new, "L": L, "ragged": rng.random() < 0.6, "page": page, "causal": rng.random() < 0.8}
    case.update({"Hkv": heads, "G": G} if op == "v2" else {"H": heads})
    return case


def _planes(form):
    return (2, 2) if form == "v1" else (1, 1)


def _spread(top, count, key, low=1):
    """`count` lengths from `low` to `top`, spread over their logarithm; they go by the case alone."""
    rng = random.Random("%s %d %d" % (key, top, count))
    return [_log(rng, low, top) for _ in range(count)]


def _chunks(case):
    """(new tokens, cached tokens with them) of each sequence. Of a ragged batch the first is the longest, and
    one slot in eight is empty."""
    B, n, L = case["B"], case["new"], case["L"]
    if not case["ragged"]:
        return [(n, L)] * B
    out = [(n, L)]
    for i, (a, c) in enumerate(zip(_spread(n, B, "new"), _spread(L, B, "len"))):
        if i:
            out.append((0, 0) if i % 8 == 7 else (a, max(a, c)))
    return out


def _appends(case):
    """(cached tokens, new tokens) of each sequence of a write."""
    B, n = case["B"], case["new"]
    return [((case["cached"] * (i + 1)) // B, max(1, n - 5 * (i % 7)) if n > 1 else 1) for i in range(B)]


# ---------------------------------------------------------------------------------------------
# the 4-bit format, in elementary operations
# ---------------------------------------------------------------------------------------------
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _quantize(x):
    """bf16 rows x [..., 16 * n] to (code bytes uint8 [..., 8 * n], e4m3 scales [..., n]): s = amax / 6
    rounded to e4m3 (448 at most), c = x / s rounded to e2m1, ties to the even code. A bf16 has 8
    significant bits, s has 4 and a border of e2m1 has 3, so a quotient off a border is off by far
    more than 32 bits round: every decision is the exact one."""
    x = x.float().unflatten(-1, (-1, 16))
    top = x.abs().amax(-1)
    s = (top / torch.full_like(top, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn)  # a true division, no product with 1/6
    f = s.float()[..., None]
    y = torch.where(f > 0, x.abs() / f, torch.zeros_like(x))
    c = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    c = (c + 8 * (x < 0)).to(torch.uint8)
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


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _rows(shape, gen, dev, dtype=torch.bfloat16):
    """Rows as projections give them: normal values, some channels several times as large."""
    x = torch.randn(shape, generator=gen, device=dev, dtype=dtype)
    loud = 1.0 + 3.0 * (torch.rand(shape[-1], generator=gen, device=dev) < 0.06)
    return x * loud.to(dtype)


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


def _angles(top, pairs, dev):
    """The table of cosines and sines fp32 [top, pairs, 2] of positions 0 .. top - 1, angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=dev) / pairs)
    a = torch.arange(top, dtype=torch.float64, device=dev)[:, None] * freq
    return torch.stack([a.cos(), a.sin()], -1).float()


def _axes(pairs, n, dev):
    """The axis of each pair: runs of pairs, one for each axis; None for one axis."""
    return None if n == 1 else (torch.arange(pairs, device=dev) * n // pairs).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    op = case["op"]
    s = {"op": op}
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if op == "rope":
        n, d, pairs = case["total"], case["d"], case["rot"] // 2
        dtype = torch.float32 if case["fp32"] else torch.bfloat16
        q = _rows((n + FREE, case["hq"], case["parts"] * d), gen, dev, dtype)
        k = _rows((n + FREE, case["hk"], case["parts"] * d), gen, dev, dtype) if case["hk"] else None
        pos = torch.randint(0, case["top"], (case["axes"], n + FREE), generator=gen, device=dev).to(torch.int32)
        pos[:, n:] = -1
        s.update(q=q, k=k, d=d, pairs=pairs, inter=case["inter"], back=case["back"], table=_angles(case["top"], pairs, dev),
                 pos=pos if case["axes"] > 1 else pos[0], axes=_axes(pairs, case["axes"], dev),
                 out=(torch.zeros_like(q), torch.zeros_like(k) if k is not None else None))
        return s
    if op in ("append", "append4"):
        kp, vp = _planes(case["form"])
        old, new = zip(*_appends(case))
        page, H, width, pairs = case["page"], case["H"], 128 * kp, case["rot"] // 2
        lens = [a + b for a, b in zip(old, new)]
        table, pages = _tables(lens, page, 5, gen, dev)
        total = sum(new)
        # q, k and v are views of one projection, with rows of padding behind
        proj = _rows((total + FREE, case["hq"] + 2 * H, width), gen, dev)
        seq = torch.repeat_interleave(torch.arange(len(new), device=dev), torch.tensor(new, device=dev))
        cu = _offsets(new, dev)
        at = torch.arange(total, device=dev) - cu[seq].long() + torch.tensor(old, device=dev)[seq]
        slots = table[seq, at // page].long() * page + at % page
        free = torch.full((FREE,), -1, device=dev)
        slots = torch.cat([slots, free]).to(torch.int32)
        at = torch.cat([at, free]).to(torch.int32)
        if case["axes"] > 1:  # places of an image's pieces below the position in the sequence
            other = torch.randint(0, 64, (case["axes"] - 1, total + FREE), generator=gen, device=dev).to(torch.int32)
            at = torch.cat([at[None], torch.where(at[None] < 0, -1, other)])
        s.update(q=proj[:, :case["hq"]], k=proj[:, case["hq"]:case["hq"] + H], v=proj[:, case["hq"] + H:], kp=kp, vp=vp,
                 d=128, pairs=pairs, inter=case["inter"], back=False, pos=at, axes=_axes(pairs, case["axes"], dev),
                 table=_angles(max(max(lens), 64), pairs, dev), slots=slots, total=total, width=width, page=page,
                 q_out=torch.zeros((total + FREE, case["hq"], width), dtype=torch.bfloat16, device=dev))
        if op == "append":
            s.update(k_pool=torch.zeros((pages, page, H, width), dtype=torch.bfloat16, device=dev),
                     v_pool=torch.zeros((pages, page, H, width), dtype=torch.bfloat16, device=dev))
        else:
            s.update(pool=torch.zeros((pages, H, page // 16, 1152 * (kp + vp)), dtype=torch.uint8, device=dev),
                     block_table=table, cu=cu, starts=ints(old))
        return s
    kp, vp = _planes(op)
    H = case["Hkv"] if op == "v2" else case["H"]
    new, lens = zip(*_chunks(case))
    table, pages = _tables(lens, case["page"], 3, gen, dev)
    R = case["page"] // 16
    pool = torch.empty((pages, H, R, 1152 * (kp + vp)), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 19) // (H * case["page"]))
    for a in range(0, pages, step):  # rounded rows in every page, a few pages at a time
        n = min(step, pages - a)
        v = torch.randn((n, H, R, 16, 128 * vp), generator=gen, device=dev, dtype=torch.bfloat16)
        pool[a:a + n] = _pack(_rows((n, H, R, 16, 128 * kp), gen, dev), v, kp, vp)
    rows = sum(new) + FREE
    norm = lambda *shape: torch.randn(shape, generator=gen, device=dev)  # noqa: E731
    s.update(pool=pool, block_table=table, page=case["page"], kp=kp, vp=vp, cu=_offsets(new, dev), seqlens=ints(lens),
             new=new, lens=lens, longest=max(new), causal=case["causal"])
    if op == "v2":
        s.update(q=norm(rows, H * case["G"], 128).to(torch.bfloat16), lam=norm(rows, H * case["G"] // 2), G=case["G"],
                 out=torch.zeros((rows, H * case["G"] // 2, 128), dtype=torch.bfloat16, device=dev))
    else:
        s.update(q=norm(rows, H, 256).to(torch.bfloat16), lam=0.2 + 0.6 * torch.rand(H, generator=gen, device=dev),
                 weight=1.0 + 0.1 * norm(256), out=torch.zeros((rows, H, 256), dtype=torch.bfloat16, device=dev))
    return s


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if own:
        da = _da()
        if op == "rope":
            return da.diffattn_rope(s["q"], s["k"], s["table"], s["pos"], s["d"], axes=s["axes"], interleaved=s["inter"],
                                    inverse=s["back"], out=s["out"])
        if op == "append":
            q = da.diffattn_rope_append(s["q"], s["k"], s["v"], s["table"], s["pos"], s["slots"], s["k_pool"], s["v_pool"],
                                        s["d"], axes=s["axes"], interleaved=s["inter"], q_out=s["q_out"])
            return q, s["k_pool"], s["v_pool"]
        if op == "append4":
            q = da.diffattn_rope_kv4_append(s["q"], s["k"], s["v"], s["table"], s["pos"], s["slots"], s["pool"], axes=s["axes"],
                                            interleaved=s["inter"], q_out=s["q_out"])
            return (q,) + tuple(da.diffattn_kv4_gather(s["pool"], s["block_table"], s["cu"], s["total"], s["width"], s["width"],
                                                       starts=s["starts"]))
        if op == "v2":
            return da.diffattn_v2_fwd_kv4(s["q"], s["pool"], s["block_table"], s["cu"], s["seqlens"], s["lam"],
                                          causal=s["causal"], max_seqlen_q=s["longest"], out=s["out"])
        return da.diffattn_fwd_kv4(s["q"], s["pool"], s["block_table"], s["cu"], s["seqlens"], s["lam"], LAMBDA_INIT,
                                   norm_weight=s["weight"], eps=EPS, causal=s["causal"], max_seqlen_q=s["longest"], out=s["out"])
    if op == "rope":
        return tuple(None if x is None else _plain_rotate(s, x, o) for x, o in zip((s["q"], s["k"]), s["out"]))
    if op == "append":
        keep = s["slots"] >= 0
        slot = s["slots"][keep].long()
        s["k_pool"].flatten(0, 1)[slot] = _plain_rotate(s, s["k"], torch.zeros_like(s["k"]))[keep]
        s["v_pool"].flatten(0, 1)[slot] = s["v"][keep]
        return _plain_rotate(s, s["q"], s["q_out"]), s["k_pool"], s["v_pool"]
    if op == "append4":
        _plain_append4(s, _plain_rotate(s, s["k"], torch.zeros_like(s["k"])))
        return (_plain_rotate(s, s["q"], s["q_out"]),) + _plain_gather(s)
    return _plain_chunks(s)


def _bf16_once(x):
    """fp64 to bf16 in one rounding: towards zero to fp32 with the last bit set where anything was cut off, which
    the rounding to bf16's 8 bits then takes the right way."""
    f = x.float()
    bits = f.view(torch.int32)
    back = f.double()
    bits = bits - (back.abs() > x.abs()).to(torch.int32)
    bits = bits | (back != x).to(torch.int32)
    return bits.view(torch.float32).to(torch.bfloat16)


def _plain_rotate(s, x, out):
    """Rows x [total, heads, width] rotated, into `out` where the position is not negative."""
    pos, pairs, d = s["pos"], s["pairs"], s["d"]
    pos = pos if pos.dim() == 2 else pos[None]
    axes = s["axes"].long() if s["axes"] is not None else torch.zeros(pairs, dtype=torch.long, device=x.device)
    live = (pos >= 0).all(0)
    cs = s["table"][pos.clamp(min=0).long()[axes].T, torch.arange(pairs, device=x.device)].double()  # total pairs 2
    c, sn = cs[:, None, None, :, 0], cs[:, None, None, :, 1]
    if s["back"]:
        sn = -sn
    y = x.double().unflatten(-1, (-1, d))  # in 64 bits: the roundings to bf16 and to 4 bits have borders
    turn = y[..., :2 * pairs]
    x1, x2 = (turn[..., 0::2], turn[..., 1::2]) if s["inter"] else (turn[..., :pairs], turn[..., pairs:])
    y1, y2 = x1 * c - x2 * sn, x2 * c + x1 * sn
    turn = torch.stack([y1, y2], -1).flatten(-2) if s["inter"] else torch.cat([y1, y2], -1)
    y = torch.cat([turn, y[..., 2 * pairs:]], -1).flatten(-2)
    y = _bf16_once(y) if x.dtype == torch.bfloat16 else y.to(x.dtype)
    out.copy_(torch.where(live[:, None, None], y, out))
    return out


def _plain_append4(s, k):
    """Each row's codes and scales to their places in the records of its slot."""
    kp, vp, pool = s["kp"], s["vp"], s["pool"]
    R = pool.shape[2]
    keep = s["slots"] >= 0
    slot = s["slots"][keep].long()
    page, rec, key = slot // (16 * R), slot % (16 * R) // 16, slot % 16
    a, h, r = key // 4, key % 4 // 2, key % 2
    planes = pool.unflatten(-1, (kp + vp, 1152))
    codes, scales = planes[..., :1024], planes[..., 1024:]
    c, sc = _quantize(k[keep])                                                   # token H bytes
    codes[..., :kp, :].unflatten(-1, (2, 4, 2, 64)).movedim(-5, -2)[page, :, rec, h, a, r] = c.unflatten(-1, (kp, 64))
    to = scales[..., :kp, :].unflatten(-1, (4, 2, 4, 2, 2)).movedim(-6, -4).movedim(-2, -5)  # P H R a h r p t u
    to[page, :, rec, a, h, r] = sc.view(torch.uint8).unflatten(-1, (kp, 4, 2))
    c, sc = _quantize(s["v"][keep])
    to = codes[..., kp:, :].unflatten(-1, (2, 8, 4, 2, 8)).movedim((-6, -4), (-3, -2))       # P H R i t j p g n
    to[page, :, rec, h, a, r] = c.unflatten(-1, (vp, 8, 8))
    to = scales[..., kp:, :].unflatten(-1, (8, 4, 4)).movedim((-4, -3), (-2, -1))             # P H R t i p g
    to[page, :, rec, a, key % 4] = sc.view(torch.uint8).unflatten(-1, (vp, 8))


def _plain_gather(s):
    """The rows that were written, one sequence behind the other: (K [total, H, .], V)."""
    cu, R = s["cu"].long(), s["pool"].shape[2]
    who = torch.repeat_interleave(torch.arange(cu.numel() - 1, device=cu.device), cu[1:] - cu[:-1])
    pos = s["starts"].long()[who] + torch.arange(who.numel(), device=cu.device) - cu[who]
    page, rec, key = s["block_table"][who, pos // (16 * R)].long(), pos % (16 * R) // 16, pos % 16
    at, row = torch.unique(page * R + rec, return_inverse=True)  # each record that holds a wanted row once
    k, v = _unpack(s["pool"][at // R, :, at % R], s["kp"], s["vp"])              # n H 16 width
    return k[row, :, key].to(torch.bfloat16), v[row, :, key].to(torch.bfloat16)


def _plain_chunks(s):
    out, at, R = s["out"], 0, s["pool"].shape[2]
    H, kp, vp = s["pool"].shape[1], s["kp"], s["vp"]
    for b, (n, L) in enumerate(zip(s["new"], s["lens"])):
        if n == 0:
            continue
        pages = s["block_table"][b, :-(-L // (16 * R))].long()
        sees = torch.arange(L, device=out.device)[None]
        if s["causal"]:
            sees = sees <= L - n + torch.arange(n, device=out.device)[:, None]
        else:
            sees = sees.expand(n, L) >= 0
        for h in range(H):
            k, v = _unpack(s["pool"][pages, h], kp, vp)                          # pages R 16 width
            k, v = k.reshape(-1, 128 * kp)[:L], v.reshape(-1, 128 * vp)[:L]
            if kp == 1:  # V2: G query heads over this head of the cache
                G = s["G"]
                q = s["q"][at:at + n, h * G:(h + 1) * G].float().transpose(0, 1)  # G n 128
                score = q @ k.T / math.sqrt(128)
            else:        # V1: the two maps of this head
                q = s["q"][at:at + n, h].float().unflatten(-1, (2, 128)).transpose(0, 1)
                score = q @ k.unflatten(-1, (2, 128)).permute(1, 2, 0) / math.sqrt(128)
            score = torch.where(sees, score, torch.full_like(score, -1e30))
            p = torch.where(sees, torch.exp(score - score.amax(-1, keepdim=True)), torch.zeros_like(score))
            o = p @ v / p.sum(-1, keepdim=True)
            if kp == 1:
                lam = torch.sigmoid(s["lam"][at:at + n, h * G // 2:(h + 1) * G // 2]).T[..., None]
                out[at:at + n, h * G // 2:(h + 1) * G // 2] = (o[0::2] - lam * o[1::2]).transpose(0, 1).to(torch.bfloat16)
            else:
                o = o[0] - s["lam"][h] * o[1]
                o = o / torch.sqrt((o * o).mean(-1, keepdim=True) + EPS) * s["weight"]
                out[at:at + n, h] = (o * (1.0 - LAMBDA_INIT)).to(torch.bfloat16)
        at += n
    return out


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rope":  # rows in and out, positions, and each used row of the table once
        n, width = case["total"], case["parts"] * case["d"]
        rows = n * (case["hq"] + case["hk"]) * width
        used = min(case["top"], n * case["axes"]) * case["rot"] // 2 * 8
        return {"bytes": rows * 2 * (4 if case["fp32"] else 2) + 4 * n * case["axes"] + used,
                "flops": rows * case["rot"] // case["d"] * 3}
    if op in ("append", "append4"):
        pairs = _appends(case)
        n, width = sum(m for _, m in pairs), 128 * _planes(case["form"])[0]
        used = min(n, max(a + m for a, m in pairs)) * case["rot"] // 2 * 8
        fixed = n * case["hq"] * width * 4 + used + 4 * n * (case["axes"] + 1)
        if op == "append":
            return {"bytes": fixed + n * 2 * case["H"] * width * 4, "flops": n * (case["hq"] + case["H"]) * width * 3}
        # rows read, codes written and read, rows written
        return {"bytes": fixed + n * 2 * case["H"] * width * (2 + 0.5625 + 0.5625 + 2),
                "flops": n * (case["hq"] + case["H"]) * width * 3}
    pairs = _chunks(case)
    new, keys = sum(n for n, _ in pairs), sum(L for n, L in pairs if n)
    seen = sum(n * L - (n * (n - 1) // 2 if case["causal"] else 0) for n, L in pairs)
    if op == "v2":
        Hq = case["Hkv"] * case["G"]
        return {"bytes": keys * case["Hkv"] * 144 + new * Hq * (256 + 128 + 2), "flops": seen * Hq * 512}
    return {"bytes": keys * case["H"] * 288 + new * case["H"] * 1024, "flops": seen * case["H"] * 1536}


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


def _to_8_bits(x):
    """x in 64 bits rounded to 8 significant bits, ties to even (a bf16's value, where its exponent is not small)."""
    m = torch.frexp(x)[0]
    power = x / torch.where(m == 0, torch.ones_like(m), m)  # of two, exactly
    return torch.round(m * 256) / 256 * power  # round: half to even


def _turn64(s, x):
    """Rows x turned, as complex numbers in 64 bits; rows at position -1 are zeros."""
    pos = s["pos"].view(-1, s["pos"].shape[-1]).long()
    y = x.double().reshape(x.shape[0], x.shape[1], -1, s["d"])
    table = torch.view_as_complex(s["table"].double().contiguous())
    table = table.conj() if s["back"] else table
    for i in range(s["pairs"]):
        a = 0 if s["axes"] is None else int(s["axes"][i])
        lo, hi = (2 * i, 2 * i + 1) if s["inter"] else (i, i + s["pairs"])
        z = torch.complex(y[..., lo], y[..., hi]) * table[pos[a].clamp(min=0), i][:, None, None]
        y[..., lo], y[..., hi] = z.real, z.imag
    y = y.flatten(-2)
    y[(pos < 0).any(0)] = 0
    return y


def _read64(records, kp, vp):
    """K and V [n * 16, .] of records [n, bytes] in 64 bits, by the places of the bytes."""
    dev, n = records.device, records.shape[0]
    two = _grid(3, 1, 1, dev)
    two = torch.cat([two, -two])
    eight = _grid(7, 3, 7, dev)
    key, ch = torch.arange(16, device=dev)[:, None], torch.arange(128, device=dev)[None]
    k_code = key % 4 // 2 * 512 + key // 4 * 128 + key % 2 * 64 + ch // 32 * 16 + ch % 32 // 2
    k_scale = 1024 + key // 4 * 32 + key % 2 * 16 + ch // 32 * 4 + key % 4 // 2 * 2 + ch % 32 // 16
    v_code = key % 4 // 2 * 512 + ch // 16 * 64 + key // 4 * 16 + key % 2 * 8 + ch % 16 // 2
    v_scale = 1024 + ch // 16 * 16 + key // 4 * 4 + key % 4

    def plane(p, code_at, scale_at):
        byte = records[:, 1152 * p + code_at.flatten()].view(n, 16, 128)
        c = two[torch.where(ch % 2 == 0, byte & 15, byte >> 4).int()]
        return (c * eight[records[:, 1152 * p + scale_at.flatten()].view(n, 16, 128).int()]).flatten(0, 1)

    return (torch.cat([plane(p, k_code, k_scale) for p in range(kp)], -1),
            torch.cat([plane(kp + p, v_code, v_scale) for p in range(vp)], -1))


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "rope":
        return tuple(None if x is None else _turn64(s, x) for x in (s["q"], s["k"]))
    if op == "append":
        rows = s["slots"] >= 0
        k_pool, v_pool = (s[n].double().flatten(0, 1) for n in ("k_pool", "v_pool"))
        k_pool[s["slots"][rows].long()] = _turn64(s, s["k"])[rows]
        v_pool[s["slots"][rows].long()] = s["v"][rows].double()
        return _turn64(s, s["q"]), k_pool.view(s["k_pool"].shape), v_pool.view(s["v_pool"].shape)
    if op == "append4":
        n = s["total"]
        return _turn64(s, s["q"]), _round64(_to_8_bits(_turn64(s, s["k"])[:n])), _round64(s["v"][:n])
    H, R = s["pool"].shape[1], s["pool"].shape[2]
    out, first = s["out"].double(), 0
    for b, (n, L) in enumerate(_chunks(case)):
        pages = s["block_table"][b, :-(-L // (16 * R))].long()
        for h in range(H):
            if n == 0:
                break
            k, v = _read64(s["pool"][pages, h].flatten(0, 1), s["kp"], s["vp"])
            k, v = k[:L], v[:L]
            for lo in range(0, n, 256):  # a few queries at a time
                hi = min(n, lo + 256)
                rows = slice(first + lo, first + hi)
                hidden = torch.arange(L, device=k.device)[None] > torch.arange(L - n + lo, L - n + hi, device=k.device)[:, None]

                def attend(q, key):
                    score = q.double() @ key.transpose(0, 1) * 128 ** -0.5
                    if case["causal"]:
                        score.masked_fill_(hidden, -math.inf)
                    return torch.softmax(score, -1) @ v

                if op == "v2":
                    for p in range(h * case["G"] // 2, (h + 1) * case["G"] // 2):
                        gate = torch.sigmoid(s["lam"][rows, p].double())[:, None]
                        out[rows, p] = attend(s["q"][rows, 2 * p], k) - gate * attend(s["q"][rows, 2 * p + 1], k)
                else:
                    o = attend(s["q"][rows, h, :128], k[:, :128]) - s["lam"][h].double() * attend(s["q"][rows, h, 128:], k[:, 128:])
                    o = o * torch.rsqrt(o.square().mean(-1, keepdim=True) + EPS) * s["weight"].double()
                    out[rows, h] = (1 - LAMBDA_INIT) * o
        first += n
    return out
