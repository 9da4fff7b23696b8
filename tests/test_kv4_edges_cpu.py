"""What the 4-bit cache's calls refuse or promise, as far as it shows without a GPU."""
import types

import pytest

import differential_attention_gb300 as da


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
