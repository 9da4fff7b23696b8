"""V1 chunks over the 4-bit cache at exponents of V at which the norm is formed at another power of two than the
cache's (beyond 2^32 either way): the norm's eps is as large as the mean square, so that it shows in every output.
Against the float64 reference within the bound of tests/test_chunk_kv4_gpu.py."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from tests.test_chunk_kv4_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.lib()
    yield
    da.diffattn_device_status()


@pytest.mark.parametrize("v_exp", [-64, -40, -33, -32, 32, 33, 40, 63])
@pytest.mark.parametrize("new,n", [(2, 70), (90, 260), (3, 3000), (90, 2000)])  # the last two in pieces
def test_the_norms_eps_at_far_exponents(new, n, v_exp):
    c = Case("v1", [new], [n], 2, 16, v_exp=v_exp)
    eps = float(np.float32(max(0.02 * 4.0 ** v_exp, 2.0 ** -126)))
    c.kw["eps"] = eps
    got = c.run()
    c.check(got, eps=eps)
    if v_exp > -63:  # eps and the mean square both count: without the one or the other the output differs in earnest
        plain = c.want(eps=1e-30 * eps)[0]
        rows = slice(0, new)
        assert np.median(np.abs(plain[rows] - c.want(eps=eps)[0][rows]) / np.abs(plain[rows])) > 0.02
