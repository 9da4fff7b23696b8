"""Chunks over the 4-bit cache without a GPU: pins of the reference's chunk forms, and every refusal of the calls."""
import ctypes

import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from oracle import diffattn_ref as ref
from oracle import kv4_ref as kv4


def random_pool(rng, pages, H, R, kp):
    pool = rng.integers(0, 256, (pages, H, R, 2 * kp, 1152)).astype(np.uint8)
    pool[..., 1024:] = rng.integers(0x28, 0x38, pool[..., 1024:].shape)
    return pool.reshape(pages, H, R, 2304 * kp)


def test_reference_of_one_token_is_the_decode():
    rng = np.random.default_rng(1)
    table, lens = rng.permutation(6).reshape(2, 3), [33, 48]
    q, lam = rng.normal(size=(2, 2, 256)), rng.uniform(0.2, 0.8, 2)
    pool = random_pool(rng, 6, 2, 1, 2)
    a, _ = kv4.fwd(q, pool, table, [0, 1, 2], lens, lam, 0.3)
    b, _ = kv4.decode(q, pool, table, lens, lam, 0.3)
    assert np.allclose(a, b, atol=1e-13)
    q, lam = rng.normal(size=(2, 8, 128)), rng.normal(size=(2, 4))
    pool = random_pool(rng, 6, 2, 1, 1)
    a, _ = kv4.v2_fwd(q, pool, table, [0, 1, 2], lens, lam)
    b, _ = kv4.v2_decode(q, pool, table, lens, lam)
    assert np.allclose(a, b, atol=1e-13)


@pytest.mark.parametrize("causal", [False, True])
def test_reference_of_a_whole_prompt_is_the_prefill(causal):
    rng = np.random.default_rng(2)
    pool, n = random_pool(rng, 3, 1, 1, 2), 40
    k, v = kv4.sequence_rows(pool, 2, [[2, 0, 1]], 0, n)
    q = rng.normal(size=(n, 1, 256))
    a, _ = kv4.fwd(q, pool, [[2, 0, 1]], [0, n], [n], [0.4], 0.2, causal=causal)
    assert np.allclose(a, ref.diffattn_fwd(q[None], k[None], v[None], [0.4], 0.2, causal=causal)[0], atol=1e-12)
    parts = [kv4.fwd(q[lo:hi], pool, [[2, 0, 1]], [0, hi - lo], [hi if causal else n], [0.4], 0.2, causal=causal)[0]
             for lo, hi in ((0, 7), (7, 8), (8, n))]
    assert np.allclose(np.concatenate(parts), a, atol=1e-12)


def test_reference_of_hidden_rows_and_no_keys():
    rng = np.random.default_rng(3)
    pool = random_pool(rng, 2, 1, 1, 1)
    q, lam = rng.normal(size=(9, 2, 128)), rng.normal(size=(9, 1))
    a, _ = kv4.v2_fwd(q, pool, [[0], [1], [1]], [0, 5, 7, 7], [3, 0, 8], lam)
    assert np.all(a[:2] == 0) and np.all(np.any(a[2:5] != 0, axis=(1, 2))) and np.all(a[5:7] == 0) and np.all(np.isnan(a[7:]))


P = ctypes.c_void_p
ARG, SHAPE, ALIGN, WORKSPACE = -1, -2, -4, -8


def v1(**kw):
    n = ctypes.c_size_t()
    da.lib().diffattn_fwd_kv4_workspace_size(max(0, kw.get("longest", 7)), 128, 256, ctypes.byref(n))
    a = dict(q=64, pool=128, table=4, cu=8, lens=12, out=256, lam=16, w=32, eps=1e-5, longest=7, total=20, B=3, H=2, d=128, dv=256, pages=9,
             page=16, width=4, ke=0, ve=0, flags=7, ws=512, bytes=n.value)
    a.update(kw)
    return da.lib().diffattn_fwd_kv4(P(a["q"]), P(a["pool"]), P(a["table"]), P(a["cu"]), P(a["lens"]), P(a["out"]), P(a["lam"]), 0.5, P(a["w"]),
                                     a["eps"], a["longest"], a["total"], a["B"], a["H"], a["d"], a["dv"], a["pages"], a["page"], a["width"],
                                     a["ke"], a["ve"], a["flags"], P(a["ws"]), a["bytes"], None)


def v2(**kw):
    n = ctypes.c_size_t()
    da.lib().diffattn_v2_fwd_kv4_workspace_size(max(0, kw.get("longest", 7)), 16, 2, 128, ctypes.byref(n))
    a = dict(q=64, pool=128, table=4, cu=8, lens=12, out=256, lam=16, longest=7, total=20, B=3, H=2, Hq=16, d=128, pages=9, page=16, width=4, ke=0,
             ve=0, flags=1, ws=512, bytes=n.value)
    a.update(kw)
    return da.lib().diffattn_v2_fwd_kv4(P(a["q"]), P(a["pool"]), P(a["table"]), P(a["cu"]), P(a["lens"]), P(a["lam"]), P(a["out"]), a["longest"],
                                        a["total"], a["B"], a["Hq"], a["H"], a["d"], a["pages"], a["page"], a["width"], a["ke"], a["ve"],
                                        a["flags"], P(a["ws"]), a["bytes"], None)


COMMON = [(dict(q=None), ARG), (dict(pool=None), ARG), (dict(table=None), ARG), (dict(cu=None), ARG), (dict(lens=None), ARG),
          (dict(out=None), ARG), (dict(lam=None), ARG), (dict(flags=8), ARG), (dict(ke=65), ARG), (dict(ve=-65), ARG), (dict(longest=-1), SHAPE),
          (dict(total=-1), SHAPE), (dict(total=1 << 30, H=16, Hq=128), SHAPE), (dict(B=0), SHAPE), (dict(B=8193), SHAPE), (dict(d=64), SHAPE),
          (dict(pages=0), SHAPE), (dict(page=0), SHAPE), (dict(page=24), SHAPE), (dict(pages=1 << 27), SHAPE), (dict(width=0), SHAPE),
          (dict(width=(1 << 26) + 1), SHAPE), (dict(total=1 << 20, width=1 << 26), SHAPE), (dict(q=72), ALIGN), (dict(pool=136), ALIGN),
          (dict(out=264), ALIGN), (dict(table=6), ALIGN), (dict(cu=6), ALIGN), (dict(lens=6), ALIGN), (dict(lam=6), ALIGN),
          (dict(ws=None), WORKSPACE), (dict(ws=128), WORKSPACE), (dict(bytes=1000), WORKSPACE)]


@pytest.mark.parametrize("change,want", COMMON + [(dict(eps=0.0), ARG), (dict(dv=128), SHAPE), (dict(H=0), SHAPE), (dict(H=65536), SHAPE),
                                                   (dict(w=24), ALIGN)])
def test_v1_refuses(change, want):
    assert v1(**change) == want
    assert "diffattn_fwd_kv4:" in da.lib().diffattn_last_error_string().decode()


@pytest.mark.parametrize("change,want", COMMON + [(dict(flags=2), ARG), (dict(H=0), SHAPE), (dict(Hq=6), SHAPE), (dict(Hq=32), SHAPE),
                                                   (dict(Hq=2), SHAPE)])
def test_v2_refuses(change, want):
    assert v2(**change) == want
    assert "diffattn_v2_fwd_kv4:" in da.lib().diffattn_last_error_string().decode()


def test_workspace_sizes():
    L, n = da.lib(), ctypes.c_size_t()
    assert L.diffattn_fwd_kv4_workspace_size(5, 128, 256, None) == ARG and L.diffattn_v2_fwd_kv4_workspace_size(5, 8, 1, 128, None) == ARG
    for args in ((-1, 128, 256), (5, 64, 256), (5, 128, 128)):
        assert L.diffattn_fwd_kv4_workspace_size(*args, ctypes.byref(n)) == SHAPE
    for args in ((-1, 8, 1, 128), (5, 8, 0, 128), (5, 6, 1, 128), (5, 8, 1, 64)):
        assert L.diffattn_v2_fwd_kv4_workspace_size(*args, ctypes.byref(n)) == SHAPE
    for longest in (0, 1, 8, 9, 33, 5000):  # what the binding keeps for streams of other libraries covers all
        assert 0 < da.diffattn_fwd_kv4_workspace_size(longest) <= da.diffattn_fwd_kv4_workspace_size(1 << 20)
        assert 0 < da.diffattn_v2_fwd_kv4_workspace_size(longest, 4, 2) <= da.diffattn_v2_fwd_kv4_workspace_size(1 << 20, 8, 1)


def test_binding_refuses_tensors_without_a_device():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        da.diffattn_fwd_kv4(torch.zeros(4, 2, 256, dtype=torch.bfloat16), torch.zeros(1, 2, 1, 4608, dtype=torch.uint8), i[None], i, i[:1],
                            torch.zeros(2))
    with pytest.raises(ValueError):
        da.diffattn_v2_fwd_kv4(torch.zeros(4, 4, 128, dtype=torch.bfloat16), torch.zeros(1, 2, 1, 2304, dtype=torch.uint8), i[None], i, i[:1],
                               torch.zeros(4, 2))
