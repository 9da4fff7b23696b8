"""Scratch that the binding lends to calls over the 4-bit cache on streams of other libraries: decodes hold no more
than decodes need, and chunks beside them have their own."""
import numpy as np
import pytest
import torch

import differential_attention_gb300 as da
from tests.test_chunk_kv4_gpu import Case
from tests.test_kv4_edges_gpu import ForeignStream

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    da.build()
    da.lib()
    yield
    da.diffattn_device_status()


@pytest.mark.parametrize("form", ["v1", "v2"])
def test_decodes_on_foreign_streams_hold_a_decodes_scratch(form):
    c = Case(form, [1, 1], [300, 41], 2, 16, behind=0)
    q, pool, table, cu, lens, lam = c.args()
    decode = da.diffattn_decode_kv4 if form == "v1" else da.diffattn_v2_decode_kv4
    want, chunk = decode(q, pool, table, lens, lam), c.run()
    torch.cuda.synchronize()
    kept = dict(da._lent_buffers)
    da._lent_buffers.clear()
    try:
        s = ForeignStream()
        out = [torch.empty_like(want) for _ in range(4)]
        decode(q, pool, table, lens, lam, out=out[0], stream=s.handle)
        need = max(da.diffattn_decode_kv4_workspace_size(1, 1), da.diffattn_v2_decode_kv4_workspace_size(1, 8, 1))
        assert sum(buffer.numel() for buffer, _ in da._lent_buffers.values()) <= need
        # decodes and chunks in turn, of two such streams
        t = ForeignStream()
        chunks = [torch.full_like(chunk, 5.0) for _ in range(4)]
        for i in range(1, 4):
            c.run(out=chunks[i], stream=(s, t)[i % 2].handle)
            decode(q, pool, table, lens, lam, out=out[i], stream=(s, t)[i % 2].handle)
            c.run(out=chunks[0], stream=t.handle)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in out) and all(torch.equal(o, chunk) for o in chunks)
        s.close()
        t.close()
    finally:
        torch.cuda.synchronize()
        da._lent_buffers.clear()
        da._lent_buffers.update(kept)
