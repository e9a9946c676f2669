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


# ----------------------------------------------------------------------------- gradient layouts

def whole(shape, g, most):
    return torch.randint(-most, most + 1, shape, generator=g).float()


def exact_block(T, D, F, seed, most_dh, gate):
    """A SwiGLU block whose every sum is a whole number.  x has a column of ones that W_gate alone
    reads, so g = `gate` (>= 52: s = 1 / (1 + e^-g) is 1 in fp32), h = g u, dg = dh u and du = g dh;
    each row of W_up holds two values +-2, so |u| <= 12, which 8 bits hold exactly next to x <= 3."""
    g = torch.Generator().manual_seed(seed)
    x, dh = whole((T, D), g, 3), whole((T, F), g, most_dh)
    x[:, 0] = 1.0
    a, b = torch.zeros(F, D), torch.zeros(F, D)
    a[:, 0] = gate
    for _ in range(2):
        at = torch.randint(1, D, (F,), generator=g)
        b[torch.arange(F), at] = torch.randint(0, 2, (F,), generator=g).float() * 4 - 2
    return [t.to(BF16).cuda() for t in (x, a, b, dh)]


def rounded(v):
    """float64 whole numbers as fp32 (exact below 2^24), then bf16: one rounding, to even."""
    return v.float().to(BF16)


def check_gradients(api, x, a, b, dh, words, must_differ):
    """Both forms of the gradient against the exact sums rounded once.  They are taken from the first
    bf16 words of dg and du; the weight gradients from 8-bit activations from `words` of them."""
    T, D = x.shape
    F = a.shape[0]
    X, A, B, DH = (v.double() for v in (x, a, b, dh))
    g, u = X @ A.t(), X @ B.t()
    dg, du = DH * u, DH * g
    first = [v.to(F32).to(BF16).double() for v in (dg, du)]
    # dg and du fit two words, and every partial sum an fp32 significand
    for v, w in zip((dg, du), first):
        assert torch.equal((v - w).to(F32).to(BF16).double(), v - w)
    unit = 4.0 if bool((du % 4 == 0).all()) else 1.0
    assert float((dg.abs().t() @ X.abs()).max()) < 2 ** 24 and float((du.abs().t() @ X.abs()).max()) < unit * 2 ** 24
    assert float((first[0].abs() @ A.abs() + first[1].abs() @ B.abs()).max()) < unit * 2 ** 24
    want = [rounded(first[0] @ A + first[1] @ B), rounded(first[0].t() @ X), rounded(first[1].t() @ X)]
    want_saved = want if words == 1 else [want[0], rounded(dg.t() @ X), rounded(du.t() @ X)]
    if must_differ:      # the test would see a second word that is missing
        assert not torch.equal(want_saved[1], want[1]) and not torch.equal(want_saved[2], want[2])
    saved = api.SwigluSaved(T, D, F)
    h = api.swiglu_forward(x, a, b, saved=saved)
    assert torch.equal(h, rounded(g * u))
    assert torch.equal(api.swiglu_forward(x, a, b), h)
    for kw, want in ((dict(x=x), want), (dict(saved=saved), want_saved)):
        bufs = [torch.full((n + 1, D), 5.0, dtype=BF16, device="cuda") for n in (T, F, F)]
        got = api.swiglu_backward(dh, a, b, dx=bufs[0][:T], dw_gate=bufs[1][:F], dw_up=bufs[2][:F], **kw)
        for name, y, w in zip(("dx", "dw_gate", "dw_up"), got, want):
            assert torch.equal(y, w), (name, sorted(kw))
        assert all(bool((v[-1] == 5.0).all()) for v in bufs)


# sizes, and the layout (148 SMs) that they are here for
LAYOUTS = [
    # tiles taken two at a time: whole, the last one with and without columns in its second half
    ((2130, 1024, 1096), dict(words=1, tile=512, split_dw=1, split_dx=1)),
    ((1629, 1296, 784), dict(words=1, tile=512, split_dw=1, split_dx=1)),
    ((1373, 1576, 672), dict(words=1, tile=512, split_dw=1, split_dx=1)),
    # and with K of dx in pieces
    ((1626, 512, 3144), dict(words=1, tile=512, split_dw=1, split_dx=4)),
    ((1615, 264, 3120), dict(words=1, tile=512, split_dw=1, split_dx=4)),
    ((2069, 560, 2064), dict(words=1, tile=512, split_dw=1, split_dx=2)),
    ((1577, 1328, 5576), dict(words=1, tile=512, split_dw=1, split_dx=4)),
    # projections taken two at a time, the last one with and without columns in its second half
    ((281, 1296, 7184), dict(words=1, tile=256, split_dw=1, split_dx=4, gateup_tile=512)),
    ((258, 1432, 7840), dict(words=1, tile=256, split_dw=1, split_dx=4, gateup_tile=512)),
    # halved and whole tiles, K of either kind in pieces
    ((65, 144, 64), dict(words=1, tile=128, split_dw=1, split_dx=1)),
    ((1330, 304, 1328), dict(words=1, tile=128, split_dw=1, split_dx=2)),
    ((1047, 136, 64), dict(words=1, tile=128, split_dw=4, split_dx=1)),
    ((1773, 128, 2392), dict(words=1, tile=128, split_dw=2, split_dx=4)),
    ((452, 3536, 336), dict(words=1, tile=256, split_dw=1, split_dx=1)),
    ((109, 2960, 1664), dict(words=1, tile=256, split_dw=1, split_dx=4)),
    ((4197, 136, 64), dict(words=1, tile=256, split_dw=16, split_dx=1)),
    ((1805, 136, 568), dict(words=1, tile=256, split_dw=4, split_dx=2)),
]


@pytest.mark.parametrize("shape,plan", LAYOUTS)
def test_every_layout_of_the_gradients_is_exact_on_whole_numbers(api, shape, plan):
    chosen = api.swiglu_backward_plan(*shape)
    assert plan == {k: chosen[k] for k in plan}
    x, a, b, dh = exact_block(*shape, 5, 2, 64.0)
    check_gradients(api, x, a, b, dh, 1, False)


# two words, in tiles of either width, with K of dx whole and in pieces
TWO_WORDS = [
    ((65, 128, 72), dict(words=2, tile=128, split_dw=1, split_dx=1)),
    ((500, 520, 520), dict(words=2, tile=128, split_dw=1, split_dx=1)),
    ((67, 128, 480), dict(words=2, tile=128, split_dw=1, split_dx=4)),
    ((65, 3128, 72), dict(words=2, tile=256, split_dw=1, split_dx=1)),
    ((65, 136, 2680), dict(words=2, tile=256, split_dw=1, split_dx=16)),
]


@pytest.mark.parametrize("shape,plan", TWO_WORDS)
def test_weight_gradients_take_two_words_where_the_layout_has_time_for_them(api, shape, plan):
    """dg = dh u and du = 60 dh with |dh| up to 255 (63 where F is large, for sums below 2^24) need up
    to 12 bits, four more than a bf16 word has: the weight gradients are those of both words, each
    with the tokens it belongs to."""
    chosen = api.swiglu_backward_plan(*shape)
    assert plan == {k: chosen[k] for k in plan}
    x, a, b, dh = exact_block(*shape, 6, 63 if shape[2] > 2000 else 255, 60.0)
    check_gradients(api, x, a, b, dh, 2, True)


# ----------------------------------------------------------------------------- the gate's range

@pytest.mark.parametrize("T", [2, 300])
def test_gates_over_the_whole_range_of_the_exponential(api, T):
    """g = -100, -99.5 ... 100 exactly, u = 1, dh = 1: h, dg and du within the documented error of the
    fast exponential and division, (4 + 1.2 |g|) 2^-23 of s, and its flush to 0 where s < 1.2e-38."""
    gates = torch.arange(-200, 201).float() / 2
    F, D = 408, 16
    gates = torch.cat([gates, torch.zeros(F - gates.numel())])
    a, b, x = torch.zeros(F, D), torch.zeros(F, D), torch.zeros(T, D)
    a[:, 0], b[:, 1], x[:, :2] = gates, 1.0, 1.0
    x, a, b = (t.to(BF16).cuda() for t in (x, a, b))
    assert torch.equal(a[:, 0].cpu().float(), gates)                  # at most 8 bits each
    g = f64(gates)
    s = OD.sigmoid(g)
    off = (4 + 1.2 * np.abs(g)) * 2.0 ** -23 * s + np.where(s < 1.2e-38, s, 0.0)       # of s
    half, tiny = torch.finfo(BF16).eps / 2, 2.0 ** -133
    h = g * s
    tol = np.abs(g) * off + 2.0 ** -22 * np.abs(h)                    # two fp32 products
    got = f64(api.swiglu_forward(x, a, b))
    assert np.all(np.abs(got - h) <= tol + half * (np.abs(h) + tol) + tiny)
    # x = (1, 1, 0, ...): column 0 of dw_gate is the sum of dg over the tokens, column 1 of dw_up that of du
    dh = torch.zeros(T, F, dtype=BF16, device="cuda")
    dh[-1] = 1.0
    _, da, db = api.swiglu_backward(dh, a, b, x=x)
    dg, du = OD.swiglu_factor_grads(g, np.ones(F), np.ones(F))
    # s (1 + g (1 - s)): 1 - s is off by s's error and a rounding
    e1 = off * (1 + np.abs(g) * (1 - s)) + s * np.abs(g) * (off + 2.0 ** -23) + 2.0 ** -21 * s * (1 + np.abs(g))
    e2 = np.abs(g) * off + 2.0 ** -22 * np.abs(du)
    for got, want, e in ((f64(da)[:, 0], dg, e1), (f64(db)[:, 1], du, e2)):
        e = e + half * (np.abs(want) + e) + tiny                       # dg and du in bf16
        assert np.all(np.abs(got - want) <= e + half * (np.abs(want) + e) + tiny)


# ----------------------------------------------------------------------------- next to the routed GEMM

@pytest.mark.parametrize("T", [339, 340, 700])
def test_dense_expert_next_to_the_routed_experts_of_a_prefill_batch(api, T):
    """From 340 tokens on the routed part is the GEMM.  The sum is the routed result plus the dense
    expert's, added by its FP8 product; captured, it is the same."""
    from trellis_quantized_moe_gemv_b200 import inputs
    layer = inputs.small_layer(31, E=12, D=256, F=128)
    D, FS, k = 256, 336, 4
    dl = api.DeviceLayer.from_synthetic(layer)
    rng = np.random.default_rng(33)
    x = torch.from_numpy(inputs.random_activations(rng, (T, D), "bf16")).to(BF16)
    logits = torch.from_numpy(inputs.normal_logits(rng, T, 12))
    a, b = rand((FS, D), 33, BF16, D ** -0.5), rand((FS, D), 34, BF16, D ** -0.5)
    shared = api.SharedExpert.from_dense(a, b, rand((D, FS), 35, BF16, FS ** -0.5))
    xd, ld = x.cuda(), logits.cuda()
    routed = api.moe_layer(dl, xd, ld, k).clone()
    got = api.moe_layer(dl, xd, ld, k, shared=shared).clone()
    h = api.swiglu_forward(xd, a, b)
    q, s = OD.quantize(f64(h))
    y, mag = OD.block_product(q, s, f64(shared.w_down), f64(shared.s_down))
    want = f64(routed) + y
    assert np.all(np.abs(f64(got) - want) <= (FS + 5) * 2.0 ** -23 * (mag + np.abs(want)))
    assert torch.equal(got, api.fp8_block_linear(h, shared.w_down, shared.s_down, out=routed, accumulate=True))
    graph = api.MoeGraph(dl, x.pin_memory(), logits.pin_memory(), k, shared=shared)
    out = graph.replay()
    graph.stream.synchronize()
    assert torch.equal(out, got.cpu())


# ----------------------------------------------------------------------------- past 2^31 elements

def test_many_rows_past_32_bit_offsets(api):
    """h, dg, du and the 8-bit g and u have 2.2e9 elements; whole numbers, so results are exact."""
    T, D, F = 270000, 64, 8192
    x, a, b, dh_rows = exact_block(300, D, F, 7, 2, 64.0)
    big = x.repeat(900, 1)
    assert big.shape == (T, D) and T * F > 2 ** 31
    X, A, B, DH = (v.double() for v in (x, a, b, dh_rows))
    u = X @ B.t()
    want = rounded(64.0 * u)
    places = (0, 261900, 262200, T - 300)           # 2^31 / F = 262144 lies in the second
    saved = api.SwigluSaved(T, D, F)
    for h in (api.swiglu_forward(big, a, b), api.swiglu_forward(big, a, b, saved=saved)):
        for r in places:
            assert torch.equal(h[r:r + 300], want)
        del h
    dh = torch.zeros(T, F, dtype=BF16, device="cuda")
    for r in places:
        dh[r:r + 300] = dh_rows
    dg, du = DH * u, 64.0 * DH
    dx_want = rounded(dg @ A + du @ B)
    n = len(places)
    assert float((dg.abs().t() @ X.abs()).max()) * n < 2 ** 24 and float((DH.abs().t() @ X.abs()).max()) * n < 2 ** 24
    for kw in (dict(x=big), dict(saved=saved)):
        dx, da, db = api.swiglu_backward(dh, a, b, **kw)
        assert torch.equal(da, rounded(n * (dg.t() @ X))) and torch.equal(db, rounded(n * (du.t() @ X)))
        for r in places:
            assert torch.equal(dx[r:r + 300], dx_want)
        dx[0:300] = 0
        for r in places:
            dx[r:r + 300] = 0
        assert not dx.any()


def test_large_weights_past_32_bit_offsets(api):
    """Weights and their gradients have 2.15e9 elements each."""
    T, D, F = 16, 46400, 46400
    assert D * F > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(8)
    pick = lambda shape, most: torch.randint(-most, most + 1, shape, generator=g, device="cuda")
    x, dh = pick((T, D), 3).to(BF16), pick((T, F), 2).to(BF16)
    x[:, 0] = 1.0
    a, b = torch.zeros(F, D, dtype=BF16, device="cuda"), torch.zeros(F, D, dtype=BF16, device="cuda")
    a[:, 0] = 64.0
    at = torch.randint(1, D, (F,), generator=g, device="cuda")
    b[torch.arange(F, device="cuda"), at] = 2.0
    u = 2.0 * x.double()[:, at]
    assert torch.equal(api.swiglu_forward(x, a, b), rounded(64.0 * u))
    dx, da, db = api.swiglu_backward(dh, a, b, x=x)
    dg, du, X = dh.double() * u, 64.0 * dh.double(), x.double()
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    want.index_add_(1, at, 2.0 * du)
    want[:, 0] += 64.0 * dg.sum(1)
    assert float(dg.abs().sum(1).max()) < 2 ** 24                      # in units of 64
    assert torch.equal(dx, rounded(want))
    for f in (0, 20000, 46280, F - 100):                               # 2^31 / D = 46282.4
        assert torch.equal(da[f:f + 100], rounded(dg[:, f:f + 100].t() @ X))
        assert torch.equal(db[f:f + 100], rounded(du[:, f:f + 100].t() @ X))


# ----------------------------------------------------------------------------- calls at once

class Step:
    """A training step and a serving product of one stream, on buffers of their own."""

    def __init__(self, api, T, D, F, seed):
        self.api = api
        self.x, self.dh = rand((T, D), seed, BF16), rand((T, F), seed + 1, BF16, 0.1)
        self.a, self.b = rand((F, D), seed + 2, BF16, D ** -0.5), rand((F, D), seed + 3, BF16, D ** -0.5)
        self.w, self.s_w = api.fp8_block_quantize(rand((D, F), seed + 4, F32, F ** -0.5), 128)
        self.saved = api.SwigluSaved(T, D, F)
        e = lambda *n, dtype=BF16: torch.empty(n, dtype=dtype, device="cuda")
        self.h, self.dx, self.da, self.db, self.y = e(T, F), e(T, D), e(F, D), e(F, D), e(T, D, dtype=F32)
        self.ws = e(max(api.swiglu_backward_workspace_size(T, D, F, s) for s in (True, False)), dtype=torch.uint8)
        self.ws2 = e(max(api.fp8_block_linear_workspace_size(T, D, F), 16), dtype=torch.uint8)

    def run(self):
        api, grads = self.api, dict(dx=self.dx, dw_gate=self.da, dw_up=self.db, ws=self.ws)
        api.swiglu_forward(self.x, self.a, self.b, out=self.h, saved=self.saved)
        api.fp8_block_linear(self.h, self.w, self.s_w, out=self.y, ws=self.ws2)
        api.swiglu_backward(self.dh, self.a, self.b, x=self.x, **grads)
        api.swiglu_backward(self.dh, self.a, self.b, saved=self.saved, **grads)
        api.fp8_block_linear(self.h, self.w, self.s_w, out=self.y, accumulate=True, ws=self.ws2)

    def results(self):
        return [t.clone() for t in (self.h, self.dx, self.da, self.db, self.y)]


SIZES = [((5, 512, 1040), (700, 264, 400)), ((200, 1024, 512), (1500, 520, 1200)), ((1500, 1096, 1200), (1300, 2600, 1392))]


@pytest.mark.parametrize("sizes", SIZES)
def test_two_streams_at_once(api, sizes):
    """Steps of different sizes on two streams, whose kernels run next to and behind one another, have
    the bits that they have alone."""
    steps = [Step(api, *s, 100 * i) for i, s in enumerate(sizes)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s in steps:
            for t in (s.h, s.dx, s.da, s.db, s.y):
                t.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(10):
            for st, s in zip(streams, steps):
                with torch.cuda.stream(st):
                    s.run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.results(), w))


@pytest.mark.parametrize("sizes", SIZES)
def test_two_branches_of_a_captured_graph(api, sizes):
    """The same as two branches of one graph, forked behind a kernel that fills their inputs and
    joined in front of one that reads their results."""
    steps = [Step(api, *s, 100 * i + 50) for i, s in enumerate(sizes)]
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    inputs = [[s.x.clone() for s in steps], [s.x * 0.5 for s in steps]]
    want = []
    for xs in inputs:
        for s, x in zip(steps, xs):
            s.x.copy_(x)
            s.run()
        torch.cuda.synchronize()
        want.append([s.results() for s in steps])
    source = [x.clone() for x in inputs[0]]
    copies = [[torch.empty_like(t) for t in (s.h, s.dx, s.da, s.db, s.y)] for s in steps]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for s, x in zip(steps, source):
            s.x.copy_(x)
        side.wait_stream(main)
        steps[0].run()
        with torch.cuda.stream(side):
            steps[1].run()
        main.wait_stream(side)
        for s, c in zip(steps, copies):
            for t, o in zip((s.h, s.dx, s.da, s.db, s.y), c):
                o.copy_(t)
    for n in range(6):
        for x, v in zip(source, inputs[n % 2]):
            x.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for c, w in zip(copies, want[n % 2]):
            assert all(torch.equal(a, b) for a, b in zip(c, w))
