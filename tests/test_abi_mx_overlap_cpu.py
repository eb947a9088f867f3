"""CPU checks: the conversions read and write in no fixed order, so buffers that overlap are refused before any launch."""
import ctypes

import pytest

from expert_routed_grouped_amd import moe

P = ctypes.c_void_p
A, B, C = 0x10000000, 0x20000000, 0x30000000  # never dereferenced
ROWS, K = 64, 256
N = ROWS * K


@pytest.mark.parametrize("codes,scales", [
    (A, C), (A + 16, C), (A + 2 * N - 4, C), (A - N // 2 + 4, C),      # codes inside x, at its end, into its start
    (B, A), (B, A + 2 * N - 1), (B, A - N // 32 + 1),                  # scales likewise
    (B, B), (B, B + N // 2 - 1), (B, B - N // 32 + 1),                 # codes and scales
])
def test_quantize_mx4_refuses_overlap(codes, scales):
    assert moe.lib().moe_quantize_mx4(P(A), moe.MOE_BF16, ROWS, K, P(codes), P(scales), None) == -2


@pytest.mark.parametrize("fmt,bytes_", [(moe.MOE_MXFP4, N // 2), (moe.MOE_MXFP8, N)])
@pytest.mark.parametrize("dtype,size", [(moe.MOE_F32, 4), (moe.MOE_BF16, 2)])
def test_dequantize_mx_refuses_overlap(fmt, bytes_, dtype, size):
    f = moe.lib().moe_dequantize_mx
    for out in (A, A + bytes_ - 16, A - size * N + 16, B, B + N // 32 - 16, B - size * N + 16):
        assert f(P(A), P(B), fmt, ROWS, K, P(out), dtype, None) == -2
