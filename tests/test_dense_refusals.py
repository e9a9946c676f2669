"""Host-side checks of the dense-expert entry points (no GPU: nothing is enqueued) and of their
Python wrappers."""
import ctypes

import pytest
import torch

import trellis_quantized_moe_gemv_b200.build as tqbuild

FAKE = ctypes.c_void_p(0x10000)        # 16-byte aligned, never dereferenced
MISALIGNED = ctypes.c_void_p(0x10004)
BIG = ctypes.c_size_t(1 << 40)
F16, BF16, F32 = 0, 1, 2
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def api():
    tqbuild.build()
    from trellis_quantized_moe_gemv_b200 import api
    return api


@pytest.fixture(scope="module")
def lib(api):
    return api.lib()


def test_quantize_and_dequantize(lib):
    q = lib.fp8_block_quantize      # x, dtype, rows, cols, block_rows, out, scales, stream
    assert q(FAKE, 3, 4, 128, 1, FAKE, FAKE, None) == INVALID
    assert q(FAKE, F32, -1, 128, 1, FAKE, FAKE, None) == INVALID
    assert q(FAKE, F32, 4, 0, 1, FAKE, FAKE, None) == INVALID
    assert q(FAKE, F32, 4, 100, 1, FAKE, FAKE, None) == INVALID          # cols % 8
    assert q(FAKE, F32, 4, 128, 2, FAKE, FAKE, None) == INVALID          # block_rows
    assert q(None, F32, 4, 128, 1, FAKE, FAKE, None) == INVALID
    assert q(FAKE, F32, 4, 128, 1, None, FAKE, None) == INVALID
    assert q(FAKE, F32, 4, 128, 1, FAKE, None, None) == INVALID
    assert q(MISALIGNED, F32, 4, 128, 1, FAKE, FAKE, None) == ALIGNMENT
    assert q(FAKE, F32, 4, 128, 1, FAKE, MISALIGNED, None) == ALIGNMENT
    assert q(FAKE, F32, 1 << 41, 128, 128, FAKE, FAKE, None) == UNSUPPORTED   # more blocks than a grid has
    assert q(None, F32, 0, 128, 1, None, None, None) == OK
    d = lib.fp8_block_dequantize    # q, scales, rows, cols, block_rows, out, dtype, stream
    assert d(FAKE, FAKE, 4, 128, 1, FAKE, 5, None) == INVALID
    assert d(FAKE, FAKE, 4, 12, 1, FAKE, F32, None) == INVALID
    assert d(FAKE, FAKE, 4, 128, 64, FAKE, F32, None) == INVALID
    assert d(FAKE, None, 4, 128, 1, FAKE, F32, None) == INVALID
    assert d(FAKE, FAKE, 4, 128, 1, MISALIGNED, F32, None) == ALIGNMENT
    assert d(None, None, 0, 128, 1, None, F32, None) == OK


def test_products(lib):
    g = lib.fp8_block_gemm          # x, s_x, w, s_w, M, N, K, y, y_dtype, accumulate, stream
    assert g(FAKE, FAKE, FAKE, FAKE, 4, 4, 100, FAKE, F32, 0, None) == INVALID      # K % 16
    assert g(FAKE, FAKE, FAKE, FAKE, 4, 4, 0, FAKE, F32, 0, None) == INVALID
    assert g(FAKE, FAKE, FAKE, FAKE, -1, 4, 128, FAKE, F32, 0, None) == INVALID
    assert g(FAKE, FAKE, FAKE, FAKE, 4, 4, 128, FAKE, 9, 0, None) == INVALID
    assert g(FAKE, FAKE, FAKE, FAKE, 4, 4, 128, FAKE, BF16, 1, None) == UNSUPPORTED  # accumulate in 16 bits
    assert g(FAKE, None, FAKE, FAKE, 4, 4, 128, FAKE, F32, 0, None) == INVALID
    assert g(FAKE, FAKE, FAKE, FAKE, (1 << 31) - 1, 4, 128, FAKE, F32, 0, None) == UNSUPPORTED
    assert g(FAKE, FAKE, MISALIGNED, FAKE, 4, 4, 128, FAKE, F32, 0, None) == ALIGNMENT
    assert g(None, None, None, None, 0, 4, 128, None, F32, 0, None) == OK
    assert g(None, None, None, None, 4, 0, 128, None, F32, 0, None) == OK
    need = lib.fp8_block_linear_workspace_size(33, 4, 144)
    assert need == 4864 + 512            # 33 x 144 E4M3 bytes and 33 x 2 scales, in units of 256
    assert lib.fp8_block_linear_workspace_size(16, 4, 144) == 0      # one kernel
    assert lib.fp8_block_linear_workspace_size(16, 64 * 1024, 1 << 20) > 0   # its share of K does not fit a CTA
    assert lib.fp8_block_linear_workspace_size(33, 4, 100) == 0
    lin = lib.fp8_block_linear      # x, dtype, w, s_w, M, N, K, y, y_dtype, accumulate, ws, bytes, stream
    assert lin(FAKE, 3, FAKE, FAKE, 33, 4, 144, FAKE, F32, 0, FAKE, BIG, None) == INVALID
    assert lin(FAKE, F32, FAKE, FAKE, 33, 4, 144, FAKE, F32, 0, FAKE, ctypes.c_size_t(need - 1), None) == WORKSPACE
    assert lin(FAKE, F32, FAKE, FAKE, 33, 4, 144, FAKE, F32, 0, None, BIG, None) == WORKSPACE
    assert lin(FAKE, F32, FAKE, FAKE, 33, 4, 144, FAKE, F32, 0, MISALIGNED, BIG, None) == ALIGNMENT
    assert lin(MISALIGNED, F32, FAKE, FAKE, 33, 4, 144, FAKE, F32, 0, FAKE, BIG, None) == ALIGNMENT
    assert lin(FAKE, F32, FAKE, None, 33, 4, 144, FAKE, F32, 0, FAKE, BIG, None) == INVALID
    assert lin(FAKE, F32, FAKE, FAKE, 33, 4, 144, FAKE, F16, 1, FAKE, BIG, None) == UNSUPPORTED
    assert lin(None, F32, None, None, 0, 4, 144, None, F32, 0, None, 0, None) == OK


def _saved(api, **other):
    st = api.TqSwigluSaved()
    for name in ("x", "s_x", "g", "s_g", "u", "s_u"):
        setattr(st, name, other.get(name, 0x10000))
    return ctypes.byref(st)


def test_swiglu(lib, api):
    f = lib.swiglu_forward          # x, w_gate, w_up, dtype, T, D, F, h, saved, stream
    assert f(FAKE, FAKE, FAKE, F32, 4, 128, 64, FAKE, None, None) == UNSUPPORTED
    assert f(FAKE, FAKE, FAKE, 7, 4, 128, 64, FAKE, None, None) == INVALID
    assert f(FAKE, FAKE, FAKE, BF16, 4, 100, 64, FAKE, None, None) == INVALID        # D % 8
    assert f(FAKE, FAKE, FAKE, BF16, 4, 128, 60, FAKE, None, None) == INVALID        # F % 8
    assert f(FAKE, FAKE, FAKE, BF16, -4, 128, 64, FAKE, None, None) == INVALID
    assert f(FAKE, None, FAKE, BF16, 4, 128, 64, FAKE, None, None) == INVALID
    assert f(FAKE, FAKE, FAKE, BF16, (1 << 31) - 8, 128, 64, FAKE, None, None) == UNSUPPORTED
    assert f(FAKE, FAKE, MISALIGNED, BF16, 4, 128, 64, FAKE, None, None) == ALIGNMENT
    assert f(FAKE, FAKE, FAKE, BF16, 4, 128, 64, FAKE, _saved(api, s_g=None), None) == INVALID
    assert f(FAKE, FAKE, FAKE, BF16, 4, 128, 64, FAKE, _saved(api, u=0x10004), None) == ALIGNMENT
    assert f(None, FAKE, FAKE, BF16, 0, 128, 64, None, None, None) == OK
    # dg and du in two words each (a small problem), and x as bf16
    assert lib.swiglu_backward_workspace_size(3, 136, 72, 0) == 4 * 512
    assert lib.swiglu_backward_workspace_size(3, 136, 72, 1) == 4 * 512 + 1024
    assert lib.swiglu_backward_workspace_size(3, 100, 72, 1) == 0
    need = ctypes.c_size_t(4 * 512)
    b = lib.swiglu_backward     # dh, x, saved, w_gate, w_up, dtype, T, D, F, dx, dw_gate, dw_up, ws, bytes, stream

    def call(dh=FAKE, x=FAKE, saved=None, wg=FAKE, dtype=BF16, T=3, D=136, F=72, dx=FAKE, dwg=FAKE, ws=FAKE, n=need):
        return b(dh, x, saved, wg, FAKE, dtype, T, D, F, dx, dwg, FAKE, ws, n, None)

    assert call(dtype=F16) == UNSUPPORTED
    assert call(dtype=F32) == UNSUPPORTED
    assert call(dtype=-1) == INVALID
    assert call(D=100) == INVALID and call(F=1) == INVALID and call(T=-1) == INVALID
    assert call(x=None) == INVALID                                   # neither x nor saved
    assert call(saved=_saved(api)) == INVALID                        # both
    assert call(x=None, saved=_saved(api, g=None), n=BIG) == INVALID
    assert call(x=None, saved=_saved(api)) == WORKSPACE              # needs room for x
    assert call(dh=None) == INVALID and call(dwg=None) == INVALID and call(dx=None) == INVALID
    assert call(dx=MISALIGNED) == ALIGNMENT and call(dwg=MISALIGNED) == ALIGNMENT and call(ws=MISALIGNED) == ALIGNMENT
    assert call(ws=None) == WORKSPACE and call(n=ctypes.c_size_t(2047)) == WORKSPACE


def test_wrappers_refuse_before_the_library_is_called(api):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    w = torch.zeros(64, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.fp8_block_quantize(x)
    with pytest.raises(ValueError, match="CUDA"):
        api.swiglu_forward(x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        api.fp8_block_linear(x, w.to(torch.float8_e4m3fn), torch.ones(1, 1))
    with pytest.raises(TypeError):
        api.fp8_block_quantize(x.double())
    with pytest.raises(TypeError):
        api.fp8_block_gemm(x, torch.ones(4, 1), w.to(torch.float8_e4m3fn), torch.ones(1, 1))
    with pytest.raises(ValueError, match="exactly one"):
        api.swiglu_backward(torch.zeros(4, 64, dtype=torch.bfloat16), w, w)
    with pytest.raises(ValueError, match="matrix"):
        api.swiglu_forward(x[0], w, w)
