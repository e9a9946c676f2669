"""Cases of the dense-expert operators: the gated feed-forward block (SwiGLU) with its
gradient, the same with its activations kept in 8 bits, and the 8-bit matrix product with
a scale for each block of 128.

A routed layer's tokens also pass a dense expert that every token uses.  Its gate and up
projections are ``swiglu``; a training step adds ``swiglu_grad`` (the projections are
computed again from x) or, where the activations of the forward pass are to be kept in
8 bits until the backward pass, ``swiglu_saved`` (forward and backward as one step); its
FP8-stored projections at serving time are ``fp8_linear``.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128
# products of the sizes of the largest listed cases: no drawn case costs more
MOST_FFN = 8192 * 4096 * 1024
MOST_FP8 = 8192 * 4096 * 4096


def listed():
    return [
        # one token through the dense expert of the 384-expert layer's shape (decoding)
        {"name": "swiglu-t1", "op": "swiglu", "T": 1, "D": 4096, "F": 1024, "dtype": "bf16"},
        # the decode batch of the benchmark, an expert eight times as wide
        {"name": "swiglu-t16-wide", "op": "swiglu", "T": 16, "D": 4096, "F": 8192, "dtype": "bf16"},
        # a ragged batch between decoding and prefill, fp16, sizes that fill no tile
        {"name": "swiglu-t203-ragged", "op": "swiglu", "T": 203, "D": 2056, "F": 1000, "dtype": "f16"},
        # the prefill batch of the benchmark
        {"name": "swiglu-t8192", "op": "swiglu", "T": 8192, "D": 4096, "F": 1024, "dtype": "bf16"},
        # backward pass of a short ragged micro-batch
        {"name": "grad-t1111-ragged", "op": "swiglu_grad", "T": 1111, "D": 1000, "F": 504, "dtype": "bf16"},
        # backward pass of a full training batch
        {"name": "grad-t8192", "op": "swiglu_grad", "T": 8192, "D": 4096, "F": 1024, "dtype": "bf16"},
        # a training step with 8-bit activations, small and ragged
        {"name": "saved-t777-ragged", "op": "swiglu_saved", "T": 777, "D": 1032, "F": 392, "dtype": "bf16"},
        # a training step with 8-bit activations, full batch
        {"name": "saved-t8192", "op": "swiglu_saved", "T": 8192, "D": 4096, "F": 1024, "dtype": "bf16"},
        # one token through a square FP8 projection
        {"name": "fp8-m1", "op": "fp8_linear", "M": 1, "N": 4096, "K": 4096, "dtype": "bf16", "out": "bf16"},
        # a decode batch through a wide FP8 projection
        {"name": "fp8-m16-wide", "op": "fp8_linear", "M": 16, "N": 16384, "K": 4096, "dtype": "bf16", "out": "bf16"},
        # ragged in every size, fp32 result
        {"name": "fp8-m333-ragged", "op": "fp8_linear", "M": 333, "N": 1001, "K": 2064, "dtype": "f16", "out": "f32"},
        # the prefill batch through the square projection
        {"name": "fp8-m8192", "op": "fp8_linear", "M": 8192, "N": 4096, "K": 4096, "dtype": "bf16", "out": "bf16"},
    ]


def _log(rng, low, high, step=1):
    """A multiple of `step` in [low, high], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(low, min(high, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["swiglu", "swiglu", "swiglu_grad", "swiglu_saved", "fp8_linear", "fp8_linear"])
    if op == "fp8_linear":
        N, K = _log(rng, 64, 16384), _log(rng, 128, 8192, 16)
        M = min(_log(rng, 1, 8192), max(1, MOST_FP8 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "out": rng.choice(["bf16", "f16", "f32"])}
    train = op != "swiglu"
    D, F = _log(rng, 128, 8192, 8), _log(rng, 64, 8192, 8)
    T = min(_log(rng, 64 if train else 1, 8192), max(1, MOST_FFN // (D * F)))
    return {"op": op, "T": T, "D": D, "F": F, "dtype": "bf16" if train else rng.choice(["bf16", "f16"])}


def work(case):
    if case["op"] == "fp8_linear":
        M, N, K = case["M"], case["N"], case["K"]
        e_in, e_out = (4 if case[k] == "f32" else 2 for k in ("dtype", "out"))
        scales = 4 * -(-N // BLOCK) * -(-K // BLOCK)
        return {"bytes": e_in * M * K + N * K + scales + e_out * M * N, "flops": 2 * M * N * K}
    T, D, F = case["T"], case["D"], case["F"]
    x, h, w = 2 * T * D, 2 * T * F, 4 * F * D      # w: both weight matrices
    if case["op"] == "swiglu":
        return {"bytes": x + w + h, "flops": 4 * T * D * F}
    if case["op"] == "swiglu_grad":                # reads x, w, dh; writes dx, dw
        return {"bytes": 2 * x + 2 * w + h, "flops": 12 * T * D * F}
    # the step reads x, w, dh and writes h, dx, dw; the 8-bit x, g and u are written once and read once
    kept = T * D + 2 * T * F + 4 * T * (-(-D // BLOCK) + 2 * -(-F // BLOCK))
    return {"bytes": 2 * x + 2 * w + 2 * h + 2 * kept, "flops": 12 * T * D * F}


def _activations(T, D, g):
    """N(0,1) rows of uneven size with a few channels thirty times as large, as the input of a
    feed-forward block has them."""
    x = torch.randn(T, D, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device="cuda"))
    big = torch.randint(0, D, (max(1, D // 512),), generator=g, device="cuda")
    x[:, big] *= 30.0
    return x


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    dt = DT[case["dtype"]]
    if case["op"] == "fp8_linear":
        M, N, K = case["M"], case["N"], case["K"]
        x = _activations(M, K, g).to(dt)
        # a stored FP8 weight: E4M3 values and one fp32 scale for each 128 x 128 block
        n_b, k_b = -(-N // BLOCK), -(-K // BLOCK)
        w = torch.zeros(n_b * BLOCK, k_b * BLOCK, device="cuda")
        w[:N, :K] = torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)
        blocks = w.view(n_b, BLOCK, k_b, BLOCK)
        s_w = (blocks.abs().amax(dim=(1, 3)) / 448.0).contiguous()
        q = (blocks / s_w[:, None, :, None]).clamp(-448.0, 448.0).reshape(n_b * BLOCK, k_b * BLOCK)
        return {"op": case["op"], "x": x, "w": q[:N, :K].contiguous().to(torch.float8_e4m3fn), "s_w": s_w,
                "out": DT[case["out"]]}
    T, D, F = case["T"], case["D"], case["F"]
    x = _activations(T, D, g).to(dt)
    w_gate = (torch.randn(F, D, generator=g, device="cuda") / math.sqrt(D)).to(dt)
    w_up = (torch.randn(F, D, generator=g, device="cuda") / math.sqrt(D)).to(dt)
    state = {"op": case["op"], "x": x, "w_gate": w_gate, "w_up": w_up}
    if case["op"] != "swiglu":
        state["dh"] = (0.1 * torch.randn(T, F, generator=g, device="cuda")).to(dt)
    return state


def run(state):
    if own:
        return _run_own(state)
    return _run_plain(state)


# ------------------------------------------------------------------------- the framework's calls

def _run_own(s):
    from trellis_quantized_moe_gemv_b200 import api
    if s["op"] == "fp8_linear":
        return api.fp8_block_linear(s["x"], s["w"], s["s_w"], out_dtype=s["out"])
    if s["op"] == "swiglu":
        return api.swiglu_forward(s["x"], s["w_gate"], s["w_up"])
    if s["op"] == "swiglu_grad":
        return api.swiglu_backward(s["dh"], s["w_gate"], s["w_up"], x=s["x"])
    T, D = s["x"].shape
    saved = api.SwigluSaved.empty(T, D, s["w_gate"].shape[0], s["x"].device)
    h = api.swiglu_forward(s["x"], s["w_gate"], s["w_up"], saved=saved)
    return (h,) + tuple(api.swiglu_backward(s["dh"], s["w_gate"], s["w_up"], saved=saved))


# ------------------------------------------------------------------------- plain forms

def _e4m3_blocks(x):
    """fp32 [R, C] as E4M3 times one power of two for each row and 128 columns, as the fp32
    values it stands for: the smallest 2^e >= 2^-126 with max|x| <= 448 * 2^e."""
    R, C = x.shape
    c_b = -(-C // BLOCK)
    b = torch.nn.functional.pad(x, (0, c_b * BLOCK - C)).view(R, c_b, BLOCK)
    m, e = torch.frexp(b.abs().amax(dim=2, keepdim=True))
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    e = torch.where(m > 0, e, torch.zeros_like(e))
    q = torch.ldexp(b, -e).to(torch.float8_e4m3fn).to(torch.float32)
    return torch.ldexp(q, e).view(R, c_b * BLOCK)[:, :C]


def _run_plain(s):
    if s["op"] == "fp8_linear":
        N, K = s["w"].shape
        scale = s["s_w"].repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
        return (_e4m3_blocks(s["x"].float()) @ (s["w"].float() * scale).t()).to(s["out"])
    dt = s["x"].dtype
    x, w_gate, w_up = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    g, u = x @ w_gate.t(), x @ w_up.t()
    if s["op"] == "swiglu":
        return (g * torch.sigmoid(g) * u).to(dt)
    out = ()
    if s["op"] == "swiglu_saved":
        out = ((g * torch.sigmoid(g) * u).to(dt),)
        x, g, u = _e4m3_blocks(x), _e4m3_blocks(g), _e4m3_blocks(u)
    dh = s["dh"].float()
    sig = torch.sigmoid(g)
    dg = dh * u * (sig * (1.0 + g * (1.0 - sig)))
    du = dh * (g * sig)
    return out + ((dg @ w_gate + du @ w_up).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt))


# ------------------------------------------------------------------------- 64 bits

def _stored64(v):
    """What a float64 matrix becomes when each row's blocks of 128 are stored as E4M3 (3 mantissa
    bits, least exponent -6, nearest even, largest 448) times 2^e: rounding to the step of
    each value's own binade."""
    R, C = v.shape
    out = torch.empty_like(v)
    for c in range(0, C, BLOCK):
        b = v[:, c:c + BLOCK]
        top = b.abs().max(dim=1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 448.0))
        e = torch.where(top > 448.0 * torch.exp2(e), e + 1, e)          # log2 may fall either way next to a power
        e = torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(min=-126.0)
        e = torch.where(top > 0, e, torch.zeros_like(e))
        y = b / torch.exp2(e)
        binade = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).clamp(min=-6.0)
        step = torch.exp2(binade - 3.0)
        out[:, c:c + BLOCK] = torch.round(y / step) * step * torch.exp2(e)   # torch.round: ties to even
    return out


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if s["op"] == "fp8_linear":
        N, K = s["w"].shape
        y = torch.zeros(x.shape[0], N, dtype=torch.float64, device=x.device)
        xs, w = _stored64(x), s["w"].to(torch.float64)
        for k in range(0, K, BLOCK):
            part = xs[:, k:k + BLOCK] @ w[:, k:k + BLOCK].t()
            y += part * s["s_w"][:, k // BLOCK].double().repeat_interleave(BLOCK)[:N]
        return y
    a, b = s["w_gate"].double(), s["w_up"].double()
    g, u = torch.einsum("td,fd->tf", x, a), torch.einsum("td,fd->tf", x, b)
    h = g / (1.0 + torch.exp(-g)) * u
    if s["op"] == "swiglu":
        return h
    saved = s["op"] == "swiglu_saved"
    if saved:
        x, g, u = _stored64(x), _stored64(g), _stored64(u)
    e = torch.exp(-g)
    dh = s["dh"].double()
    du = dh * g / (1.0 + e)
    dg = dh * u * ((1.0 + e) + g * e) / (1.0 + e) ** 2
    dx = torch.einsum("tf,fd->td", dg, a) + torch.einsum("tf,fd->td", du, b)
    grads = (dx, torch.einsum("tf,td->fd", dg, x), torch.einsum("tf,td->fd", du, x))
    return (h,) + grads if saved else grads
