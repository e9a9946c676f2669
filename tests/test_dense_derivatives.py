"""Derivatives asked for through the dense-expert calls, which record no history: refused, not lost
(no GPU needed: the refusal comes before any look at the device)."""
import pytest
import torch
from torch.autograd import forward_ad

BF16, FP8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def api():
    from trellis_quantized_moe_gemv_b200 import api
    return api


def tensors():
    return dict(x=torch.zeros(4, 128, dtype=BF16), w=torch.zeros(64, 128, dtype=BF16), dh=torch.zeros(4, 64, dtype=BF16),
                w8=torch.zeros(64, 128).to(FP8), x8=torch.zeros(4, 128).to(FP8), s_w=torch.ones(1, 1), s_x=torch.ones(4, 1))


def calls(api, t):
    shared = api.SharedExpert(t["w"], t["w"], t["w8"], t["s_w"])
    return {"swiglu_forward": (lambda: api.swiglu_forward(t["x"], t["w"], t["w"]), "x"),
            "swiglu_backward": (lambda: api.swiglu_backward(t["dh"], t["w"], t["w"], x=t["x"]), "dh"),
            "fp8_block_linear": (lambda: api.fp8_block_linear(t["x"], t["w8"], t["s_w"]), "x"),
            "fp8_block_gemm": (lambda: api.fp8_block_gemm(t["x8"], t["s_x"], t["w8"], t["s_w"]), "x8"),
            "fp8_block_quantize": (lambda: api.fp8_block_quantize(t["x"]), "x"),
            "fp8_block_dequantize": (lambda: api.fp8_block_dequantize(t["x8"], t["s_x"]), "x8"),
            "shared_expert": (lambda: api.shared_expert(shared, t["x"]), "x")}


NAMES = ("swiglu_forward", "swiglu_backward", "fp8_block_linear", "fp8_block_gemm", "fp8_block_quantize",
         "fp8_block_dequantize", "shared_expert")


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_that_requires_a_gradient_is_refused(api, name):
    t = tensors()
    call, first = calls(api, t)[name]
    t[first].requires_grad_(True)
    with pytest.raises(ValueError, match="requires a gradient"):
        call()
    # without gradients the call goes on to its other checks
    for off in (torch.no_grad, torch.inference_mode):
        with off(), pytest.raises(ValueError, match="CUDA"):
            call()
    t[first].requires_grad_(False)
    with pytest.raises(ValueError, match="CUDA"):
        call()


def test_a_result_of_recorded_operations_is_refused(api):
    x = (torch.zeros(4, 128, requires_grad=True) * 2).to(BF16)
    with pytest.raises(ValueError, match="requires a gradient"):
        api.swiglu_forward(x, torch.zeros(64, 128, dtype=BF16), torch.zeros(64, 128, dtype=BF16))


def test_a_forward_mode_tangent_is_refused(api):
    t = tensors()
    with forward_ad.dual_level():
        x = forward_ad.make_dual(t["x"], torch.ones_like(t["x"]))
        with pytest.raises(ValueError, match="tangent"):
            api.swiglu_forward(x, t["w"], t["w"])
        with pytest.raises(ValueError, match="CUDA"):
            api.swiglu_forward(t["x"], t["w"], t["w"])


def test_later_arguments_are_looked_at_too(api):
    t = tensors()
    w = t["w"].clone().requires_grad_(True)
    for check in (lambda: api._require_dense(w, BF16, (64, 128), "w_up", -1), lambda: api._require_matrix(w, BF16, "w_gate", -1)):
        with pytest.raises(ValueError, match="requires a gradient"):
            check()
