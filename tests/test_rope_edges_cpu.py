"""What the calls on rotary positions say of strides that they refuse."""
import pytest

import differential_attention_gb300 as da
from tests.test_rope_cpu import ALIGN, append_call, rope_call, strides

FAR = (1 << 36) + 128


@pytest.mark.parametrize("call", [rope_call, append_call, lambda **kw: append_call(True, **kw)])
@pytest.mark.parametrize("bad", [FAR, 1 << 62, 252, 0, -128])
def test_a_refused_stride_is_named_with_its_limits(call, bad):
    assert call(st=strides((256, 128), (128, 128), (256, bad), (128, 128))) == ALIGN
    said = da.lib().diffattn_last_error_string().decode()
    assert f"stride 5 ({bad})" in said and "multiple of 16 bytes" in said and "2^36" in said
