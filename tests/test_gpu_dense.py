"""The dense-expert operators on the GPU against their 64-bit definitions.

Tolerances.  u = 2^-24.  A sum of n products in fp32, in any order and with rounded or truncated
additions, is off by at most n * 2^-23 of the sum of magnitudes (gamma_n with the larger
unit).  The fast exponential and division are taken as 2^-18 relative.  A result rounded to
type t adds finfo(t).eps / 2 of its value.  Where all sums are exact (small integers, power
of two scales) the results must be equal."""
import numpy as np
import pytest
import torch

from oracle import dense as OD

pytestmark = pytest.mark.gpu

BF16, F16, F32, FP8 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn
HALF = {t: torch.finfo(t).eps / 2 for t in (BF16, F16, F32)}
LEAST = {BF16: 2.0 ** -133, F16: 2.0 ** -24, F32: 2.0 ** -149}     # half a step near zero, at most
FAST = 2.0 ** -18


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


def ints(shape, seed, most, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype).cuda()


def close(got, want, tol, dtype):
    got = f64(got)
    err = np.abs(got - want)
    lim = tol + HALF[dtype] * (np.abs(want) + tol) + LEAST[dtype]
    assert np.all(err <= lim), "max err/tol %.3e at %s" % (np.max(err / lim), np.unravel_index(np.argmax(err / lim), err.shape))


# ----------------------------------------------------------------------------- storage

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("rows,cols,block_rows", [(1, 8, 1), (3, 128, 1), (5, 136, 1), (17, 1000, 1), (300, 264, 1),
                                                  (1, 8, 128), (128, 128, 128), (129, 136, 128), (300, 1000, 128)])
def test_quantize_is_exactly_the_definition(api, dtype, rows, cols, block_rows):
    x = rand((rows, cols), 11 * rows + cols, F32)
    x *= torch.exp2(torch.randint(-9, 5, (rows, 1), generator=torch.Generator().manual_seed(1)).float()).cuda()
    x = x.to(dtype)
    if rows > 2:
        x[1] = 0.0                                   # a row (and its blocks) of zeros
    q, s = api.fp8_block_quantize(x, block_rows)
    wq, ws = OD.quantize(f64(x), block_rows)
    np.testing.assert_array_equal(f64(s), ws)
    np.testing.assert_array_equal(f64(q), wq)
    for t in (F32, BF16, F16):
        got = api.fp8_block_dequantize(q, s, block_rows, out_dtype=t)
        want = torch.from_numpy(wq * OD.spread(ws, rows, cols, block_rows)).to(F32).to(t)   # exact in fp32
        assert torch.equal(got.cpu(), want)


def test_quantize_extreme_values(api):
    x = torch.zeros(12, 128)
    x[0, 3] = torch.finfo(F32).max
    x[1, 3] = float("inf"); x[1, 4] = 2.0
    x[2, 3] = float("-inf")                          # nothing finite but zeros
    x[3, 3] = float("nan"); x[3, 5] = 448.0
    x[4, 3] = 2.0 ** -149                            # least subnormal: scale 2^-126
    x[5, 3] = 1e-38; x[5, 4] = -1e-39
    x[6, 3] = 448.0; x[6, 4] = 2.0 ** -10; x[6, 5] = 2.0 ** -10 * 1.5   # ties next to E4M3's least step
    x[7, 3] = 449.0                                  # just past: scale 2
    x[8, :] = float("nan")
    x[9, 3] = -0.0; x[9, 4] = -2.0 ** -30; x[9, 5] = 1.0
    x[10, 0] = 464.0; x[10, 1] = 3.5
    x[11, 127] = 1.0 + 1.0 / 16.0                    # tie
    xd = x.cuda()
    for block_rows in (1, 128):
        q, s = api.fp8_block_quantize(xd, block_rows)
        wq, ws = OD.quantize(f64(xd), block_rows)
        np.testing.assert_array_equal(f64(s), ws)
        np.testing.assert_array_equal(f64(q), wq)    # NaN equals NaN here


def test_quantize_writes_nothing_else(api):
    buf = torch.full((4 + 7 * 136 + 64,), 7, dtype=torch.uint8, device="cuda")[:7 * 136 + 64]
    out, sc = buf[:7 * 136].view(FP8).view(7, 136), torch.full((9, 2), -5.0, device="cuda")
    api.fp8_block_quantize(rand((7, 136), 3), out=out, scales=sc[:7])
    torch.cuda.synchronize()
    assert (buf[7 * 136:] == 7).all() and (sc[7:] == -5.0).all() and (sc[:7] > 0).all()


# ----------------------------------------------------------------------------- FP8 product

SHAPES = [(1, 1, 16), (1, 128, 128), (2, 7, 112), (16, 129, 144), (17, 256, 384), (33, 1001, 272), (64, 200, 2064),
          (65, 64, 128), (128, 300, 1040), (129, 130, 128), (255, 256, 256), (257, 1000, 400), (520, 513, 1168),
          # the pair kernel: several rounds of tiles, a ragged one in every size
          (1300, 1500, 272), (257, 9503, 144), (2100, 1030, 1168), (4100, 5000, 48), (1500, 1300, 1024),
          (1500, 1300, 1536), (1100, 2050, 2000),
          # one launch up to 128 blocks of a row, two beyond
          (9, 513, 2048), (16, 200, 1024), (16, 200, 8208), (3, 20000, 2064)]


def exact_operands(M, N, K, seed):
    """Integers up to 3 with power-of-two scales 2^-2 .. 2^2: every partial sum is a multiple of
    2^-4 below 9 K 2^4, exact in fp32 for K < 2^13."""
    g = torch.Generator().manual_seed(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    s_x = torch.exp2(torch.randint(-2, 3, (M, kb), generator=g).float()).cuda()
    s_w = torch.exp2(torch.randint(-2, 3, (nb, kb), generator=g).float()).cuda()
    return ints((M, K), seed + 1, 3, FP8), s_x, ints((N, K), seed + 2, 3, FP8), s_w


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_of_integers_is_exact(api, M, N, K):
    x, s_x, w, s_w = exact_operands(M, N, K, M + N + K)
    want, _ = OD.block_product(f64(x), f64(s_x), f64(w), f64(s_w))
    got = api.fp8_block_gemm(x, s_x, w, s_w, out_dtype=F32)
    np.testing.assert_array_equal(f64(got), want)
    for t in (BF16, F16):
        got = api.fp8_block_gemm(x, s_x, w, s_w, out_dtype=t)
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(F32).to(t))
    out = torch.ones(M, N, device="cuda")
    api.fp8_block_gemm(x, s_x, w, s_w, out=out, accumulate=True)
    np.testing.assert_array_equal(f64(out), want + 1.0)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(api, dtype, M, N, K):
    x = rand((M, K), M * 7 + K, dtype)
    w, s_w = api.fp8_block_quantize(rand((N, K), N, F32, K ** -0.5), 128)
    s_w = s_w * 1.37                                  # any fp32 scale
    q, s = OD.quantize(f64(x))
    want, mag = OD.block_product(q, s, f64(w), f64(s_w))
    got = api.fp8_block_linear(x, w, s_w, out_dtype=F32)
    # n = K + the scale product, its use and the block's addition
    close(got, want, (K + 4) * 2.0 ** -23 * mag, F32)
    # the same bits as the two calls, and in the same call again
    xq, sx = api.fp8_block_quantize(x)
    for _ in range(2):
        assert torch.equal(got, api.fp8_block_gemm(xq, sx, w, s_w, out_dtype=F32))
    y16 = api.fp8_block_linear(x, w, s_w)
    assert y16.dtype == BF16 and torch.equal(y16, got.to(BF16))


@pytest.mark.parametrize("M", [5, 200, 6500])
def test_product_keeps_nan_to_its_row_and_writes_nothing_else(api, M):
    N, K = 301, 272
    x, s_x, w, s_w = exact_operands(M, N, K, 5)
    want, _ = OD.block_product(f64(x), f64(s_x), f64(w), f64(s_w))
    x = x.clone()
    x.view(torch.uint8)[2, 131] = 0x7F
    buf = torch.full((M + 3, N), -9.0, device="cuda")
    api.fp8_block_gemm(x, s_x, w, s_w, out=buf[:M])
    got = f64(buf)
    assert np.isnan(got[2]).all() and (got[M:] == -9.0).all()
    keep = [i for i in range(M) if i != 2]
    np.testing.assert_array_equal(got[keep], want[keep])


def test_zero_sizes(api):
    w, s_w = api.fp8_block_quantize(rand((130, 32), 1), 128)
    assert api.fp8_block_linear(torch.empty(0, 32, device="cuda"), w, s_w).shape == (0, 130)
    none = torch.empty(0, 32, dtype=FP8, device="cuda")
    assert api.fp8_block_linear(rand((3, 32), 1), none, torch.empty(0, 1, device="cuda")).shape == (3, 0)
    q, s = api.fp8_block_quantize(torch.empty(0, 136, device="cuda"))
    assert q.shape == (0, 136) and s.shape == (0, 2)
    wg = rand((64, 32), 2, BF16)
    x, dh = torch.empty(0, 32, dtype=BF16, device="cuda"), torch.empty(0, 64, dtype=BF16, device="cuda")
    assert api.swiglu_forward(x, wg, wg).shape == (0, 64)
    dx, a, b = api.swiglu_backward(dh, wg, wg, x=x)
    assert dx.shape == (0, 32) and not a.any() and not b.any()


# ----------------------------------------------------------------------------- SwiGLU

def swiglu_inputs(T, D, F, seed, dtype=BF16):
    return (rand((T, D), seed, dtype), rand((F, D), seed + 1, dtype, D ** -0.5), rand((F, D), seed + 2, dtype, D ** -0.5))


def forward_oracle(x, a, b):
    """h, g, u and the errors that fp32 sums allow each."""
    x, a, b = f64(x), f64(a), f64(b)
    h, g, u = OD.swiglu(x, a, b)
    n = (x.shape[1] + 1) * 2.0 ** -23
    dg, du = n * (np.abs(x) @ np.abs(a).T), n * (np.abs(x) @ np.abs(b).T)
    # |silu'| <= 1.1, |silu(g)| <= |g|
    dh = 1.1 * (np.abs(u) + du) * dg + np.abs(g) * du + FAST * (np.abs(h) + 1.1 * np.abs(u) * dg + np.abs(g) * du)
    return h, g, u, dh, dg, du


T_SHAPES = [(1, 8, 8), (1, 128, 64), (2, 136, 72), (7, 1000, 504), (16, 256, 128), (17, 512, 200), (33, 64, 1000),
            (64, 264, 136), (128, 1032, 264), (129, 128, 128), (256, 256, 256), (300, 1000, 504), (513, 72, 392),
            # the pair kernel: one round, a last round halved in width, several rounds
            (1280, 72, 1280), (2000, 136, 1400), (4100, 64, 2600)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,D,F", T_SHAPES)
def test_forward(api, dtype, T, D, F):
    x, a, b = swiglu_inputs(T, D, F, T + D + F, dtype)
    h, _, _, tol, _, _ = forward_oracle(x, a, b)
    buf = torch.full((T + 2, F), 3.0, dtype=dtype, device="cuda")
    got = api.swiglu_forward(x, a, b, out=buf[:T])
    close(got, h, tol, dtype)
    assert (buf[T:] == 3.0).all()
    assert torch.equal(got, api.swiglu_forward(x, a, b))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,D,F", T_SHAPES)
def test_forward_saves_its_activations(api, dtype, T, D, F):
    x, a, b = swiglu_inputs(T, D, F, T + D + F, dtype)
    h, g, u, tol, dg, du = forward_oracle(x, a, b)
    saved = api.SwigluSaved.empty(T, D, F)
    close(api.swiglu_forward(x, a, b, saved=saved), h, tol, dtype)
    q, s = api.fp8_block_quantize(x)
    assert torch.equal(saved.x.view(torch.uint8), q.view(torch.uint8)) and torch.equal(saved.s_x, s)
    for q, s, want, off in ((saved.g, saved.s_g, g, dg), (saved.u, saved.s_u, u, du)):
        sc = OD.spread(f64(s), T, F)
        # the scale's exponent is that of a largest value within `off` of the true one
        for r in range(T):
            for j in range(s.shape[1]):
                c = slice(128 * j, 128 * (j + 1))
                top, d = np.abs(want[r, c]).max(), off[r, c].max()
                assert top - d <= 448.0 * sc[r, c][0] and top + d >= 224.0 * sc[r, c][0]
        y = want / sc
        lim = off + sc * OD.e4m3_half_step((np.abs(y) + off / sc) * (1 + 1e-12))
        assert np.all(np.abs(f64(q) * sc - want) <= lim)


def grads_oracle(g, u, dh, x, a, b, eg, eu):
    """Gradients of the values g, u, x and the errors that g and u off by eg and eu, bf16 dg and
    du, and fp32 sums allow."""
    dg, du = OD.swiglu_factor_grads(g, u, dh)
    # d(silu')/dg is at most 1/2 in magnitude
    edg = np.abs(dh) * (1.1 * eu + 0.5 * (np.abs(u) + eu) * eg)
    edu = np.abs(dh) * 1.1 * eg
    # s (1 + g (1 - s)): 1 - s is off by 2^-23 and FAST of s, times |g| s
    edg += np.abs(dh) * (np.abs(u) + eu) * FAST * (1.1 + np.abs(g))
    edu += np.abs(dh) * (np.abs(g) + eg) * FAST
    edg += HALF[BF16] * (np.abs(dg) + edg) + 2.0 ** -133
    edu += HALF[BF16] * (np.abs(du) + edu) + 2.0 ** -133
    F, T = dg.shape[1], dg.shape[0]
    mg, mu = np.abs(dg) + edg, np.abs(du) + edu
    tol = (edg @ np.abs(a) + edu @ np.abs(b) + (2 * F + 1) * 2.0 ** -23 * (mg @ np.abs(a) + mu @ np.abs(b)),
           edg.T @ np.abs(x) + (T + 1) * 2.0 ** -23 * (mg.T @ np.abs(x)),
           edu.T @ np.abs(x) + (T + 1) * 2.0 ** -23 * (mu.T @ np.abs(x)))
    return OD.swiglu_grads(dg, du, x, a, b), tol


B_SHAPES = [(1, 8, 8), (1, 128, 64), (3, 136, 72), (64, 64, 64), (65, 264, 200), (128, 256, 256), (200, 1000, 136),
            (257, 520, 264), (300, 72, 504),
          # tiles halved in width, whole, and whole with dx tiles filling up behind uneven dw tiles
          (700, 1032, 392), (1500, 1096, 1200), (1300, 2600, 1400),
          # K of the weight gradients split (many tokens), of dx (wide F), of both
          (8000, 136, 72), (4100, 520, 264), (70, 264, 4000), (1000, 72, 2056)]


@pytest.mark.parametrize("T,D,F", B_SHAPES)
def test_backward(api, T, D, F):
    x, a, b = swiglu_inputs(T, D, F, T + D + F)
    dh = rand((T, F), 99, BF16, 0.1)
    _, g, u, _, eg, eu = forward_oracle(x, a, b)
    want, tol = grads_oracle(g, u, f64(dh), f64(x), f64(a), f64(b), eg, eu)
    got = api.swiglu_backward(dh, a, b, x=x)
    for y, w, t in zip(got, want, tol):
        close(y, w, t, BF16)
    for y, z in zip(got, api.swiglu_backward(dh, a, b, x=x)):
        assert torch.equal(y, z)


@pytest.mark.parametrize("T,D,F", B_SHAPES)
def test_backward_from_saved(api, T, D, F):
    x, a, b = swiglu_inputs(T, D, F, T + D + F)
    dh = rand((T, F), 99, BF16, 0.1)
    saved = api.SwigluSaved.empty(T, D, F)
    api.swiglu_forward(x, a, b, saved=saved)
    vx = f64(saved.x) * OD.spread(f64(saved.s_x), T, D)
    g, u = (f64(q) * OD.spread(f64(s), T, F) for q, s in ((saved.g, saved.s_g), (saved.u, saved.s_u)))
    zero = np.zeros_like(g)
    want, tol = grads_oracle(g, u, f64(dh), vx, f64(a), f64(b), zero, zero)
    for y, w, t in zip(api.swiglu_backward(dh, a, b, saved=saved), want, tol):
        close(y, w, t, BF16)


@pytest.mark.parametrize("T,D,F", [(1, 8, 8), (70, 200, 136), (64, 256, 256), (200, 264, 320), (130, 520, 72),
                                   (1500, 1096, 1200), (1300, 2600, 1400), (8000, 136, 72), (70, 264, 4000),
                                   (1000, 72, 2056)])
def test_gradients_of_integers_are_exact(api, T, D, F):
    """g = 64 makes s = 1 in fp32 (e^-64 < 2^-24), so dg = dh u and du = 64 dh: with integers
    every product and sum is exact, and the result is the exact sum rounded once to bf16."""
    saved = api.SwigluSaved.empty(T, D, F)
    x, u = ints((T, D), 1, 3, FP8), ints((T, F), 2, 3, FP8)
    saved.x.copy_(x); saved.u.copy_(u)
    saved.g.copy_(torch.full((T, F), 64.0).to(FP8))
    for s in (saved.s_x, saved.s_g, saved.s_u):
        s.fill_(1.0)
    dh, a, b = ints((T, F), 3, 2, BF16), ints((F, D), 4, 3, BF16), ints((F, D), 5, 3, BF16)
    dg, du = f64(dh) * f64(u), 64.0 * f64(dh)
    want = OD.swiglu_grads(dg, du, f64(x), f64(a), f64(b))
    bufs = [torch.full((n + 1, D), 5.0, dtype=BF16, device="cuda") for n in (T, F, F)]
    got = api.swiglu_backward(dh, a, b, saved=saved, dx=bufs[0][:T], dw_gate=bufs[1][:F], dw_up=bufs[2][:F])
    for y, w, buf in zip(got, want, bufs):
        assert torch.equal(y.cpu(), torch.from_numpy(w).to(F32).to(BF16))
        assert (buf[-1] == 5.0).all()


@pytest.mark.parametrize("T,D,F", [(3000, 2048, 2904), (814, 5992, 3416), (2600, 2304, 2600), (8000, 1160, 1032),
                                   (2050, 4104, 1160)])
def test_many_tiles(api, T, D, F):
    """Sizes with several rounds of tiles, some taken two at a time with a last one past the
    matrix, against the definition in 64 bits (on the GPU); guard rows and scales stay."""
    x, a, b = swiglu_inputs(T, D, F, 77)
    dh = rand((T, F), 78, BF16, 0.1)
    X, A, B, DH = (v.double() for v in (x, a, b, dh))
    g, u = X @ A.t(), X @ B.t()
    n = (D + 1) * 2.0 ** -23
    eg, eu = n * (X.abs() @ A.abs().t()), n * (X.abs() @ B.abs().t())
    h = g * torch.sigmoid(g) * u
    tol = 1.1 * (u.abs() + eu) * eg + g.abs() * eu + 2 * FAST * (h.abs() + (u.abs() + g.abs()) * 1.1 * (eg + eu))

    def check(got, want, tol):
        lim = tol + HALF[BF16] * (want.abs() + tol) + LEAST[BF16]
        assert bool(((got.double() - want).abs() <= lim).all())

    buf = torch.full((T + 1, F), 3.0, dtype=BF16, device="cuda")
    check(api.swiglu_forward(x, a, b, out=buf[:T]), h, tol)
    assert (buf[T] == 3.0).all()
    saved = api.SwigluSaved(T, D, F)
    saved.buffer.fill_(0xA5)
    before = saved.buffer.clone()
    check(api.swiglu_forward(x, a, b, out=buf[:T], saved=saved), h, tol)
    assert (buf[T] == 3.0).all()
    inside = torch.zeros_like(saved.buffer, dtype=torch.bool)      # the parts; between them nothing is written
    for at, size in zip(saved._at, (T * D, 4 * T * -(-D // 128), T * F, 4 * T * -(-F // 128), T * F, 4 * T * -(-F // 128))):
        inside[at:at + size] = True
    assert torch.equal(saved.buffer[~inside], before[~inside])
    q, s = api.fp8_block_quantize(x)
    assert torch.equal(saved.x.view(torch.uint8), q.view(torch.uint8)) and torch.equal(saved.s_x, s)
    vals = []
    for q, s, want, off in ((saved.g, saved.s_g, g, eg), (saved.u, saved.s_u, u, eu)):
        sc = s.double().repeat_interleave(128, 1)[:, :F]
        y = q.double() * sc
        # half a step of E4M3 at most: 2^-4 of the value, or of the least normal value 2^-6
        lim = off + 2.0 ** -4 * torch.maximum(want.abs() + off, sc * 2.0 ** -6)
        assert bool(((y - want).abs() <= lim).all())
        vals.append(y)
    sx = saved.s_x.double().repeat_interleave(128, 1)[:, :D]
    cases = [(dict(x=x), X, g, u, eg, eu), (dict(saved=saved), saved.x.double() * sx, vals[0], vals[1], 0.0, 0.0)]
    for kw, xv, gv, uv, dg_, du_ in cases:
        sg = torch.sigmoid(gv)
        dg, du = DH * uv * sg * (1 + gv * (1 - sg)), DH * gv * sg
        e1 = DH.abs() * (1.1 * du_ + 0.5 * (uv.abs() + du_) * dg_ + (uv.abs() + du_) * FAST * (1.1 + gv.abs()))
        e2 = DH.abs() * (1.1 * dg_ + (gv.abs() + dg_) * FAST)
        e1 = e1 + HALF[BF16] * (dg.abs() + e1) + 2.0 ** -133
        e2 = e2 + HALF[BF16] * (du.abs() + e2) + 2.0 ** -133
        m1, m2 = dg.abs() + e1, du.abs() + e2
        bufs = [torch.full((r + 1, D), 5.0, dtype=BF16, device="cuda") for r in (T, F, F)]
        got = api.swiglu_backward(dh, a, b, dx=bufs[0][:T], dw_gate=bufs[1][:F], dw_up=bufs[2][:F], **kw)
        kx, kw_ = (2 * F + 1) * 2.0 ** -23, (T + 1) * 2.0 ** -23
        check(got[0], dg @ A + du @ B, e1 @ A.abs() + e2 @ B.abs() + kx * (m1 @ A.abs() + m2 @ B.abs()))
        check(got[1], dg.t() @ xv, e1.t() @ xv.abs() + kw_ * (m1.t() @ xv.abs()))
        check(got[2], du.t() @ xv, e2.t() @ xv.abs() + kw_ * (m2.t() @ xv.abs()))
        assert all((v[-1] == 5.0).all() for v in bufs)


def test_large_gates_and_nan_rows(api):
    """|g| up to 1e4: e^-g overflows or vanishes; a row with a NaN leaves the others alone."""
    T, D, F = 40, 64, 72
    x, a, b = swiglu_inputs(T, D, F, 8)
    a = a * 3000
    h, g, u, tol, _, _ = forward_oracle(x, a, b)
    assert np.abs(g).max() > 5000
    close(api.swiglu_forward(x, a, b), h, tol, BF16)
    saved = api.SwigluSaved.empty(T, D, F)
    close(api.swiglu_forward(x, a, b, saved=saved), h, tol, BF16)
    x[3, 5] = float("nan")
    for got in (api.swiglu_forward(x, a, b), api.swiglu_forward(x, a, b, saved=saved)):
        got = f64(got)
        assert np.isnan(got[3]).all() and np.isfinite(np.delete(got, 3, 0)).all()
    assert np.isnan(f64(saved.g)[3]).all() and (f64(saved.s_g)[3] == 1.0).all()
    dx, _, _ = api.swiglu_backward(rand((T, F), 9, BF16), a, b, saved=saved)
    assert np.isnan(f64(dx)[3]).all() and np.isfinite(np.delete(f64(dx), 3, 0)).all()


# ----------------------------------------------------------------------------- together and in use

def test_gradient_of_a_training_step_against_differences(api):
    """loss = sum(h * dh): the change along a direction from the gradient, against the 64-bit
    loss at two points."""
    T, D, F = 70, 136, 72
    x, a, b = swiglu_inputs(T, D, F, 21)
    dh = rand((T, F), 22, BF16, 0.1)
    grads = [f64(v) for v in api.swiglu_backward(dh, a, b, x=x)]
    vals = [f64(v) for v in (x, a, b)]
    rng = np.random.default_rng(23)
    for i in range(3):
        d = rng.standard_normal(vals[i].shape)
        step = 1e-4
        lo, hi = ([v + (sgn * step * d if j == i else 0) for j, v in enumerate(vals)] for sgn in (-1, 1))
        diff = sum(sgn * (OD.swiglu(*p)[0] * f64(dh)).sum() for sgn, p in ((-1, lo), (1, hi))) / (2 * step)
        # each gradient is off by at most 2^-8 of the magnitudes it sums plus its rounding 2^-8
        dg, du = OD.swiglu_factor_grads(*OD.swiglu(*vals)[1:], f64(dh))
        mags = (np.abs(dg) @ np.abs(vals[1]) + np.abs(du) @ np.abs(vals[2]), np.abs(dg).T @ np.abs(vals[0]),
                np.abs(du).T @ np.abs(vals[0]))
        assert abs((grads[i] * d).sum() - diff) <= (2.0 ** -7 * mags[i] * np.abs(d)).sum()


@pytest.mark.parametrize("T", [1, 9, 200])
def test_dense_expert_next_to_the_routed_ones(api, T):
    from oracle import layer as OL
    from trellis_quantized_moe_gemv_b200 import inputs
    layer = inputs.small_layer(31, E=12, D=256, F=128)
    D, FS, k = 256, 336, 4
    dl = api.DeviceLayer.from_synthetic(layer)
    rng = np.random.default_rng(32)
    x = inputs.random_activations(rng, (T, D), "bf16")
    logits = inputs.normal_logits(rng, T, 12)
    a, b = rand((FS, D), 33, BF16, D ** -0.5), rand((FS, D), 34, BF16, D ** -0.5)
    shared = api.SharedExpert.from_dense(a, b, rand((D, FS), 35, BF16, FS ** -0.5))
    xd = torch.from_numpy(x).to(BF16).cuda()
    ld = torch.from_numpy(logits).cuda()
    routed = api.moe_layer(dl, xd, ld, k).clone()
    got = api.moe_layer(dl, xd, ld, k, shared=shared)
    res = OL.moe_layer(layer, x, logits, k)
    h = api.swiglu_forward(xd, a, b)                   # tested above
    q, s = OD.quantize(f64(h))
    y, mag = OD.block_product(q, s, f64(shared.w_down), f64(shared.s_down))
    close(got, res["out"] + y, res["bound"] + 1e-6 * np.abs(res["out"]) + 1e-12 + (FS + 5) * 2.0 ** -23 * (mag + np.abs(res["out"])), F32)
    assert torch.equal(api.moe_layer(dl, xd, ld, k), routed)      # without it, as before
    # captured, with other inputs at the replay
    xh, lh = torch.from_numpy(x).to(BF16).pin_memory(), torch.from_numpy(logits).pin_memory()
    graph = api.MoeGraph(dl, xh, lh, k, shared=shared)
    x2 = inputs.random_activations(rng, (T, D), "bf16")
    xh.copy_(torch.from_numpy(x2).to(BF16))
    out = graph.replay()
    graph.stream.synchronize()
    again = api.moe_layer(dl, torch.from_numpy(x2).to(BF16).cuda(), ld, k, shared=shared)
    assert torch.equal(out, again.cpu())


def train_step(api, s, bufs):
    """Forward with saved activations, backward from them, the FP8 product of the saved input."""
    h = api.swiglu_forward(s["x"], s["a"], s["b"], out=bufs["h"], saved=bufs["saved"])
    grads = api.swiglu_backward(s["dh"], s["a"], s["b"], saved=bufs["saved"], dx=bufs["dx"], dw_gate=bufs["da"],
                                dw_up=bufs["db"], ws=bufs["ws"])
    y = api.fp8_block_gemm(bufs["saved"].x, bufs["saved"].s_x, s["w"], s["s_w"], out=bufs["y"])
    return (h, y) + tuple(grads)


def step_state(api, T, D, F, seed):
    x, a, b = swiglu_inputs(T, D, F, seed)
    w, s_w = api.fp8_block_quantize(rand((200, D), seed + 5), 128)
    return dict(x=x, a=a, b=b, dh=rand((T, F), seed + 4, BF16), w=w, s_w=s_w)


def step_buffers(api, T, D, F, ws=None):
    e = lambda *n, dtype=BF16: torch.empty(n, dtype=dtype, device="cuda")
    if ws is None:
        ws = e(api.swiglu_backward_workspace_size(T, D, F, True), dtype=torch.uint8)
    return dict(h=e(T, F), dx=e(T, D), da=e(F, D), db=e(F, D), y=e(T, 200, dtype=F32), ws=ws,
                saved=api.SwigluSaved.empty(T, D, F))


@pytest.mark.parametrize("T", [20, 300])
def test_a_captured_step_replays_on_new_inputs_and_two_share_a_workspace(api, T):
    D, F = 272, 136
    s = step_state(api, T, D, F, 50)
    other = step_state(api, T, D, F, 60)
    want = [[t.clone() for t in train_step(api, v, step_buffers(api, T, D, F))] for v in (s, other)]
    bufs = step_buffers(api, T, D, F)
    bufs2 = step_buffers(api, T, D, F, bufs["ws"])
    graphs = []
    for b in (bufs, bufs2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = train_step(api, s, b)
        graphs.append((g, out))
    for v in (0, 1):
        if v:
            for key in s:
                s[key].copy_(other[key])
        for g, out in graphs:
            for t in out:
                t.fill_(0)
            g.replay()
        for g, out in graphs:
            torch.cuda.synchronize()
            for t, w in zip(out, want[v]):
                assert torch.equal(t, w)


def test_first_calls_of_one_size_allow_capture_of_another():
    """In a process of its own: after one eager call of each entry point, other sizes (other
    kernels of the same entry points) are captured on their first call."""
    import os
    import subprocess
    import sys
    code = """
import torch
from trellis_quantized_moe_gemv_b200 import api
def state(T, D, F):
    g = torch.Generator().manual_seed(T)
    r = lambda *n: (torch.randn(*n, generator=g)).bfloat16().cuda()
    return r(T, D), r(F, D) / 8, r(F, D) / 8, r(T, F), *api.fp8_block_quantize(r(96, D), 128)
def calls(x, a, b, dh, w, s_w):
    saved = api.SwigluSaved(x.shape[0], x.shape[1], a.shape[0])
    h = api.swiglu_forward(x, a, b)
    h2 = api.swiglu_forward(x, a, b, saved=saved)
    return (h, h2, *api.swiglu_backward(dh, a, b, x=x), *api.swiglu_backward(dh, a, b, saved=saved),
            api.fp8_block_linear(x, w, s_w, out_dtype=torch.float32),
            api.fp8_block_gemm(saved.x, saved.s_x, w, s_w, out_dtype=torch.float32))
calls(*state(1, 64, 64))
torch.cuda.synchronize()
for T, F in ((17, 64), (40, 64), (100, 64), (1000, 2400)):
    s = state(T, 264 * 16, F) if F == 64 else state(T, 64, F)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = calls(*s)
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(out, calls(*s)):
        assert torch.equal(x, y)
print("captured", api.device_status())
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "captured 0", r.stdout + r.stderr


@pytest.mark.parametrize("T", [8, 150, 1500])
def test_a_chain_of_calls_on_the_same_buffers_without_waiting(api, T):
    """Each call reads what the one before it wrote (the launches overlap: a kernel may start
    before the one before it ends), into the same buffers again and again."""
    D, F = 256, 136
    w1, s1 = api.fp8_block_quantize(rand((D, 192), 1, F32, 192 ** -0.5), 128)
    w2, s2 = api.fp8_block_quantize(rand((F, 192), 2, F32, 192 ** -0.5), 128)
    a, b = rand((F, D), 3, BF16, D ** -0.5), rand((F, D), 4, BF16, D ** -0.5)
    ins = [rand((T, 192), 10 + i, BF16) for i in range(6)]
    e = lambda *n: torch.empty(n, dtype=BF16, device="cuda")
    x, dh, h, dx, da, db = e(T, D), e(T, F), e(T, F), e(T, D), e(F, D), e(F, D)
    saved = api.SwigluSaved(T, D, F)
    ws = torch.empty(max(api.fp8_block_linear_workspace_size(T, max(D, F), 192), 16), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(api.swiglu_backward_workspace_size(T, D, F, True), dtype=torch.uint8, device="cuda")

    def step(v, wait):
        calls = [lambda: api.fp8_block_linear(v, w1, s1, out=x, ws=ws),
                 lambda: api.fp8_block_linear(v, w2, s2, out=dh, ws=ws),
                 lambda: api.swiglu_backward(dh, a, b, x=x, dx=dx, dw_gate=da, dw_up=db, ws=ws2),
                 lambda: api.swiglu_forward(dx, a, b, out=h, saved=saved),
                 lambda: api.swiglu_backward(h, a, b, saved=saved, dx=dx, dw_gate=da, dw_up=db, ws=ws2)]
        for f in calls:
            f()
            if wait:
                torch.cuda.synchronize()
        return [t.clone() for t in (x, dh, h, dx, da, db)]

    want = [step(v, True) for v in ins]
    for _ in range(5):
        got = [step(v, False) for v in ins]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_on_another_stream(api):
    T, D, F = 100, 272, 136
    s = step_state(api, T, D, F, 70)
    want = [t.clone() for t in train_step(api, s, step_buffers(api, T, D, F))]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    outs = []
    for _ in range(20):       # outputs and workspaces come from the allocator, on the other stream
        h = api.swiglu_forward(s["x"], s["a"], s["b"], stream=st)
        g = api.swiglu_backward(s["dh"], s["a"], s["b"], x=s["x"], stream=st)
        y = api.fp8_block_linear(s["x"], s["w"], s["s_w"], out_dtype=F32, stream=st)
        outs.append((h, y, g))
    st.synchronize()
    ref = api.swiglu_backward(s["dh"], s["a"], s["b"], x=s["x"])
    for h, y, g in outs:
        assert torch.equal(y, want[1])
        close(h, f64(want[0]), HALF[BF16] * np.abs(f64(want[0])), BF16)    # another order of the sums
        assert all(torch.equal(p, q) for p, q in zip(g, ref))


def test_wrappers_refuse_mismatched_tensors(api):
    x, a, b = swiglu_inputs(4, 64, 72, 1)
    with pytest.raises(ValueError, match="inputs"):
        api.swiglu_forward(x[:, :32].contiguous(), a, b)
    with pytest.raises(ValueError, match="contiguous"):
        api.swiglu_forward(rand((64, 4), 1, BF16).t(), a, b)
    with pytest.raises(ValueError, match="shape"):
        api.swiglu_forward(x, a, b[:8])
    with pytest.raises(TypeError):
        api.swiglu_forward(x.half(), a, b)
    with pytest.raises(ValueError, match="shape"):
        api.swiglu_forward(x, a, b, saved=api.SwigluSaved.empty(4, 64, 64))
    with pytest.raises(api.TQError, match="UNSUPPORTED"):
        api.swiglu_backward(torch.zeros(4, 72, dtype=F16, device="cuda"), a.half(), b.half(), x=x.half())
    with pytest.raises(api.TQError, match="INVALID"):
        api.swiglu_forward(rand((4, 60), 1, BF16), rand((72, 60), 1, BF16), rand((72, 60), 1, BF16))
    buf = torch.zeros(4 * 64 + 8, dtype=BF16, device="cuda")
    with pytest.raises(api.TQError, match="ALIGNMENT"):
        api.swiglu_forward(buf[1:257].view(4, 64), a, b)
    w, s_w = api.fp8_block_quantize(rand((130, 64), 1), 128)
    with pytest.raises(ValueError, match="shape"):
        api.fp8_block_linear(x, w, s_w[:1])
    with pytest.raises(ValueError, match="accumulate"):
        api.fp8_block_linear(x, w, s_w, accumulate=True)
    with pytest.raises(api.TQError, match="UNSUPPORTED"):
        api.fp8_block_linear(x, w, s_w, out=torch.zeros(4, 130, dtype=BF16, device="cuda"), accumulate=True)
    with pytest.raises(api.TQError, match="WORKSPACE"):
        api.fp8_block_linear(rand((40, 64), 1), w, s_w, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="block_rows"):
        api.fp8_block_quantize(x, 64)


def test_offsets_past_32_bits(api):
    """Rows past element 2^31 of the activations and of the result."""
    K, N, M = 16, 16384, 140000                       # y has 2.29e9 elements
    x, s_x, w, s_w = exact_operands(300, N, K, 3)
    big, sb = x.repeat(467, 1)[:M].contiguous(), s_x.repeat(467, 1)[:M].contiguous()
    y = api.fp8_block_gemm(big, sb, w, s_w)
    ref = api.fp8_block_gemm(x, s_x, w, s_w)
    for r in (0, 131071, 131072, M - 300):
        part = y[r:r + 300]
        at = (torch.arange(part.shape[0]) + r) % 300
        assert torch.equal(part, ref[at.cuda()])
    del y, big
    rows, cols = 70000, 32768                         # 2.29e9 elements
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    tail = rand((40, cols), 4, BF16)
    x[-40:] = tail
    q, s = api.fp8_block_quantize(x)
    wq, ws = api.fp8_block_quantize(tail)
    assert torch.equal(q[-40:].view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s[-40:], ws)
    assert not q[65500:65600].view(torch.uint8).any()
