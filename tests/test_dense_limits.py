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


@pytest.mark.parametrize("T,D,F,words", [(3, 136, 72, 2), (500, 520, 520, 2), (65, 136, 2680, 2), (612, 400, 2928, 1),
                                         (2900, 400, 2928, 1), (777, 1032, 392, 1), (1064, 1000, 504, 1),
                                         (1111, 1000, 504, 1), (8192, 4096, 1024, 1)])
def test_second_words_where_the_gradients_launch_is_no_longer_for_them(lib, T, D, F, words):
    """148 SMs.  Where every pair has one tile at most, dw tiles of both words run over 2 ceil(T / 64)
    blocks of K and dx tiles over 2 ceil(F / 64): with no more tokens than outputs the words are
    free but for their own bytes, which may take a third of a microsecond."""
    plan = (ctypes.c_int32 * 5)()
    assert lib.swiglu_backward_plan(T, D, F, plan) == 0 and plan[0] == words


def test_workspace_holds_what_the_form_and_its_words_need(lib):
    size = lib.swiglu_backward_workspace_size
    up = lambda n: (n + 255) // 256 * 256
    for T, D, F, arrays in ((500, 520, 520, 4), (1064, 1000, 504, 2)):       # no K in pieces
        assert size(T, D, F, 0) == arrays * up(2 * T * F)
        assert size(T, D, F, 1) == arrays * up(2 * T * F) + up(2 * T * D)


def test_products_of_few_rows_may_need_a_workspace(lib):
    size, call = lib.fp8_block_linear_workspace_size, lib.fp8_block_linear
    assert size(16, 1024, 4096) == 0 and size(16, 16384, 4096) > 0
    for n in (0, size(16, 16384, 4096) - 1):
        ws = FAKE if n else None
        assert call(FAKE, BF16, FAKE, FAKE, 16, 16384, 4096, FAKE, BF16, 0, ws, ctypes.c_size_t(n), None) == 4
