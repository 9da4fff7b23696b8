"""The packed backward passes whatever their workspace holds: the last sequence's tile reaches into rows behind it."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from tests.gpu_util import assert_grad, to64

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


@pytest.mark.parametrize("lens,behind", [([200, 1, 77], 3), ([5], 400), ([130, 0], 1)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("grouped", [False, True])
def test_gradients_whatever_the_workspace_holds(lens, behind, norm, grouped):
    gen = torch.Generator().manual_seed(3)
    total, H, Hn = sum(lens) + behind, 2, 1
    heads, width = (H + Hn, 128) if grouped else (H, 256)
    q, k = (torch.randn((total, heads, width), generator=gen).to(torch.bfloat16).to(DEV) / 11 for _ in range(2))
    v, dy = (torch.randn((total, H, 256), generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    lam, B, N = torch.tensor([0.4, 0.7], device=DEV), len(lens), max(lens)
    if grouped:
        _, o_pre, stats = da.diffattn_gda_fwd_train_varlen(q, k, v, cu, lam, H, 0.3, norm=norm)
        size = da.diffattn_gda_bwd_varlen_workspace_size(B, N, total, H, Hn)
        run = lambda ws: da.diffattn_gda_bwd_varlen(q, k, v, o_pre, stats, dy, cu, lam, H, 0.3, norm=norm, workspace=ws)  # noqa: E731
    else:
        _, o_pre, stats = da.diffattn_fwd_train_varlen(q, k, v, cu, lam, 0.3, norm=norm)
        size = da.diffattn_bwd_varlen_workspace_size(B, N, total, H, 128, 256)
        run = lambda ws: da.diffattn_bwd_varlen(q, k, v, o_pre, stats, dy, cu, lam, 0.3, norm=norm, workspace=ws)  # noqa: E731
    want = run(torch.zeros(size, dtype=torch.uint8, device=DEV))
    got = run(torch.full((size,), 255, dtype=torch.uint8, device=DEV))  # NaN in every type
    for name in ("dq", "dk", "dv", "dlam"):
        assert torch.isfinite(got[name].float()).all(), name
        if name != "dlam":
            assert_grad(got[name], to64(want[name]), name=name)
    assert torch.allclose(got["dlam"], want["dlam"], rtol=1e-3, atol=1e-3)
