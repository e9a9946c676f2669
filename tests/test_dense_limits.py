"""Largest sizes of the dense-expert entry points (no GPU: nothing is enqueued).

Inside a limit a call goes on to its next check (here: an address that is not aligned); past it
the call is refused, because its 32-bit byte counts, its bounded waits or its grid do not reach."""
import ctypes

import pytest

import trellis_quantized_moe_gemv_b200.build as tqbuild

FAKE, MISALIGNED = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
BIG = ctypes.c_size_t(1 << 62)
BF16 = 1
UNSUPPORTED, ALIGNMENT = 2, 3
MOST = 2 ** 25 - 512                  # D, F of a SwiGLU block; columns of rows in 8 bits


@pytest.fixture(scope="module")
def lib():
    tqbuild.build()
    from trellis_quantized_moe_gemv_b200 import api
    return api.lib()


@pytest.mark.parametrize("D,F", [(MOST, 8), (8, MOST), (MOST, MOST)])
def test_swiglu_up_to_its_limit(lib, D, F):
    for d, f, want in ((D, F, ALIGNMENT), (D + 8 * (D == MOST), F + 8 * (F == MOST), UNSUPPORTED),
                       (D if D == 8 else 2 ** 30 + 64, F if F == 8 else 2 ** 30 + 64, UNSUPPORTED)):
        assert lib.swiglu_forward(FAKE, FAKE, MISALIGNED, BF16, 1, d, f, FAKE, None, None) == want
        assert lib.swiglu_backward(FAKE, FAKE, None, FAKE, MISALIGNED, BF16, 1, d, f, FAKE, FAKE, FAKE, FAKE, BIG, None) == want
        assert (lib.swiglu_backward_workspace_size(1, d, f, 1) > 0) == (want == ALIGNMENT)


def test_byte_counts_stay_in_32_bits():
    # a row's rest in fp32, and in 16 bits, from the first column on
    assert MOST * 4 < 2 ** 31 <= (2 ** 30 + 64) * 2


def test_rows_in_8_bits_up_to_their_limit(lib):
    for cols, want in ((MOST, ALIGNMENT), (MOST + 8, UNSUPPORTED)):
        assert lib.fp8_block_quantize(MISALIGNED, BF16, 1, cols, 1, FAKE, FAKE, None) == want
        assert lib.fp8_block_dequantize(MISALIGNED, FAKE, 1, cols, 1, FAKE, BF16, None) == want
    assert lib.fp8_block_quantize(MISALIGNED, BF16, 1, MOST + 8, 128, FAKE, FAKE, None) == ALIGNMENT


def test_plan_query(lib):
    plan = (ctypes.c_int32 * 5)()
    assert lib.swiglu_backward_plan(3, 100, 72, plan) == 1 and lib.swiglu_backward_plan(0, 128, 72, plan) == 1
    assert lib.swiglu_backward_plan(3, 128, 72, None) == 1
    assert lib.swiglu_backward_plan(3, MOST + 8, 72, plan) == UNSUPPORTED
    assert lib.swiglu_backward_plan(3, 128, 72, plan) == 0
    words, tile, split_dw, split_dx, gateup = plan
    assert words == 2 and tile in (128, 256, 512) and gateup in (128, 256, 512) and split_dw >= 1 and split_dx >= 1
