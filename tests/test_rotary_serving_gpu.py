"""Rotary positions in a server's steps over a bf16 paged cache: plan, turn and append, prefill the chunks over
the pages, then single tokens; every step's outputs against one causal pass over all tokens so far, turned by
diffattn_rope, bit for bit in the rows and within assert_bf16's tolerance in the outputs."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from tests.gpu_util import assert_bf16

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


@pytest.mark.parametrize("form", ["v1", "v2"])
def test_steps_over_bf16_pages(form):
    gen, B, H, G, page, pages = torch.Generator().manual_seed(11), 2, 2, 4, 128, 12
    hq, kw, vw = (H, 256, 256) if form == "v1" else (H * G, 128, 128)
    steps = [[130, 40], [3, 129], [1, 1], [1, 1]]
    tab = da.diffattn_rope_table(torch.as_tensor(10000.0 ** (-np.arange(64) / 64), device=DEV), 512)
    k_pool = torch.zeros((pages, page, H, kw), dtype=torch.bfloat16, device=DEV)
    v_pool = torch.zeros((pages, page, H, vw), dtype=torch.bfloat16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    seqlens, table, ring, state = torch.zeros(B, **i32), torch.zeros((B, 4), **i32), torch.randperm(pages, generator=gen).to(**i32), None
    state = torch.tensor([0, pages], **i32)
    lam1 = torch.tensor([0.3, 0.6], device=DEV)
    past = [[] for _ in range(B)]
    for new in steps:
        total = sum(new)
        plan = da.diffattn_paged_plan(seqlens, dev32(new), table, ring, state, page, total)
        seqlens, state, cu = plan["seqlens"], plan["ring_state"], plan["cu_seqlens_q"]
        proj = torch.randn((total, hq + H, kw), generator=gen).to(torch.bfloat16).to(DEV)
        q, k, v = proj[:, :hq], proj[:, hq:], torch.randn((total, H, vw), generator=gen).to(torch.bfloat16).to(DEV)
        lam = torch.randn((total, hq // 2), generator=gen).to(DEV)
        turned = da.diffattn_rope_append(q, k, v, tab, plan["positions"], plan["slot_map"], k_pool, v_pool)
        if max(new) == 1:
            out = (da.diffattn_decode_paged(turned, k_pool, v_pool, table, seqlens, lam1, 0.3) if form == "v1"
                   else da.diffattn_v2_decode_paged(turned, k_pool, v_pool, table, seqlens, lam))
        elif form == "v1":
            out = da.diffattn_fwd_paged(turned, k_pool, v_pool, cu, seqlens, table, lam1, 0.3)
        else:
            out = da.diffattn_v2_fwd_paged(turned, k_pool, v_pool, lam, cu, seqlens, table)
        at = 0
        for b, n in enumerate(new):
            past[b].append((q[at:at + n], k[at:at + n], v[at:at + n], lam[at:at + n]))
            qa, ka, va, la = (torch.cat(x) for x in zip(*past[b]))
            L = len(ka)
            qt, kt = da.diffattn_rope(qa, ka, tab, torch.arange(L, dtype=torch.int32, device=DEV))
            slots = (table[b, torch.arange(L, device=DEV) // page].long() * page + torch.arange(L, device=DEV) % page)
            assert torch.equal(k_pool.view(-1, H, kw)[slots], kt) and torch.equal(v_pool.view(-1, H, vw)[slots], va)
            assert torch.equal(turned[at:at + n], qt[L - n:])
            ends = dev32([0, L])
            whole = (da.diffattn_fwd_varlen(qt, kt, va, ends, lam1, 0.3) if form == "v1"
                     else da.diffattn_v2_fwd_varlen(qt, kt, va, la, ends))
            assert_bf16(out[at:at + n], whole[L - n:])
            at += n
    da.diffattn_device_status()
