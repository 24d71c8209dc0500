"""Sizes past the library's 32-bit ones are refused by the binding: passed on,
2^32 + 5 rows would arrive as 5."""
import pytest
import torch

BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
LONG = 2 ** 32 + 5


@pytest.fixture(scope="module")
def tw():
    from activation_sparse_feed_gate_amd import tw as mod

    return mod


def m(*shape, dtype=BF):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda tw: tw.layernorm(m(LONG, 16), m(16, dtype=F32)),
    lambda tw: tw.layernorm_backward(m(LONG, 16), m(LONG, 16), m(16, dtype=F32), m(LONG, dtype=F32), m(LONG, dtype=F32)),
    lambda tw: tw.quantize_rows(m(LONG, 16)),
    lambda tw: tw.quantize_rows(m(2, LONG)),
    lambda tw: tw.layernorm_quantize(m(LONG, 16), m(16, dtype=F32)),
    lambda tw: tw.quant_linear(m(LONG, 16), m(8, 16, dtype=I8), m(8, dtype=F32)),
    lambda tw: tw.quant_linear(m(4, 16), m(LONG, 16, dtype=I8), m(LONG, dtype=F32)),
    lambda tw: tw.quant_gateup(m(LONG, 16), m(8, 16, dtype=I8), m(8, dtype=F32), m(8, 16, dtype=I8), m(8, dtype=F32)),
    lambda tw: tw.tw_gate_dense(m(LONG, 128), m(128, 128), m(LONG, 128, dtype=F32)),
])
def test_sizes_past_32_bits_are_refused(tw, call):
    with pytest.raises(ValueError, match=r"below 2\^31"):
        call(tw)
