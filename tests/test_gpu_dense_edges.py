"""Dense-expert operators where kernels hand work over: the one-launch product's stored tokens,
the second words of dg and du, wide and split gradient tiles, large tensors.  Compared with
their 64-bit definitions, or bit by bit where the same sums are taken another way."""
import numpy as np
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32, FP8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def api():
    import trellis_quantized_moe_gemv_b200.build as b
    b.build()
    from trellis_quantized_moe_gemv_b200 import api as A
    A.device_status(clear=True)
    return A


@pytest.fixture(autouse=True)
def no_flags(api):
    yield
    torch.cuda.synchronize()
    assert api.device_status(clear=True) == 0


def f64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def rand(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


# ----------------------------------------------------------------------------- one-launch product

@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 1024, 4096), (16, 128, 8192), (5, 19000, 2816), (16, 200, 144)])
def test_one_launch_product_uses_the_scales_of_its_own_tokens(api, M, N, K):
    """Calls in a row on inputs whose block scales differ by powers of two from call to call and
    row to row: a scale read before its storing warp has written it (an earlier call's value lies
    there) is off by a factor.  Bit for bit the product of the stored operands."""
    assert api.fp8_block_linear_workspace_size(M, N, K) == 0
    w, s_w = api.fp8_block_quantize(rand((N, K), 1, F32, K ** -0.5), 128)
    g = torch.Generator().manual_seed(2)
    xs = []
    for i in range(8):
        size = torch.exp2(torch.randint(-30, 31, (M, -(-K // 128)), generator=g).float())
        x = torch.randn(M, K, generator=g) * size.repeat_interleave(128, 1)[:, :K]
        xs.append(x.to((F32, BF16)[i & 1]).cuda())
    want = [api.fp8_block_gemm(*api.fp8_block_quantize(x), w, s_w, out_dtype=F32) for x in xs]
    torch.cuda.synchronize()
    for _ in range(25):
        got = [api.fp8_block_linear(x, w, s_w, out_dtype=F32) for x in xs]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
