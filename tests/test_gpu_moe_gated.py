"""The activations of moe_layer's gated hidden rows over their whole range, their far
tails multiplied by large gates, against the definitions in float64."""
import numpy as np
import pytest
import torch

from oracle import activation_ref
from fp8_quantized_generative_b200 import workloads as wl

from ffn_bounds import F16_TINY, assert_within, round_f16
from parity import assert_no_device_error, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


# Relative error of an activation on its own argument.  e^x from an exponent x that took
# four roundings of 2^-24 of |x| (the argument's square, its product with a constant, the
# constant, the sum): 4 * 2^-24 |x|, and |x| <= |ln |act(z)|| + 2 ln(2 + |z|) for each of them.
# Besides: the GELU fit evaluated in fp32, 6.6e-6 < 2^-17, and 2^-21 for the intrinsics.
def act_rel(z, act):
    with np.errstate(divide="ignore"):
        x = np.abs(np.log(np.maximum(np.abs(act), 1e-300))) + 2.0 * np.log(2.0 + np.abs(z))
    return 2.0 ** -17 + 2.0 ** -21 + 4 * 2.0 ** -24 * x


@pytest.mark.parametrize("act", [None, "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [1, 3])
def test_gated_tails(fq, act, T):
    """Hidden rows fp16(act(z) * gate) for z over [-20, 20] with gates of up to 2^45 (the largest that
    fp16 rows of 8192 values can have) that bring the product to about 100: the activation's
    relative accuracy everywhere, its far negative tail included."""
    F, K, N = 4096, 16, 16
    f32 = np.float32
    z_want = np.linspace(-20.0, 20.0, F).astype(f32)
    with np.errstate(divide="ignore"):
        gate_want = np.clip(100.0 / np.abs(activation_ref(z_want, act)), 1.0, 2.0 ** 45).astype(f32)
    one = torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    Wu = np.zeros((1, 2 * F, K), np.uint8)
    Wu[0, :, 0] = one
    Wu[0, :F, 0] |= np.where(z_want < 0, 0x80, 0).astype(np.uint8)
    su = np.concatenate([np.abs(z_want), gate_want])[None]
    # a row of ones has the codes of 448 and the scale fl(1 / 448): one product, two roundings
    acc_s = f32(448.0) * (f32(1.0) / f32(448.0))
    z = (np.sign(z_want) * (acc_s * np.abs(z_want))).astype(f32).astype(np.float64)
    gate = (acc_s * gate_want).astype(f32).astype(np.float64)
    Wd, sd = fq.quantize_weight_per_channel(wl.random_f16((1, N, F), seed=1).cuda())
    ws = fq.moe_layer_workspace(T, 1, F, N, "cuda")
    fq.moe_layer(torch.ones((T, K), dtype=torch.float16, device="cuda"),
                 torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda"),
                 torch.from_numpy(Wu).cuda(), torch.from_numpy(su).cuda(), Wd, sd, activation=act, gated=True, workspace=ws)
    got = to_np(ws[:T * F * 2].view(torch.float16)).reshape(T, F)
    a = activation_ref(z, act)
    if act == "silu":
        a = z / (1.0 + np.exp(-z))                # (the tanh forms of the definition cancel in their tails)
    elif act == "gelu_tanh":
        a = z / (1.0 + np.exp(-2.0 * np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3)))
    ref = a * gate
    bound = round_f16((act_rel(z, a) + 2.0 ** -23) * np.abs(ref) + F16_TINY * 2.0 ** -10, ref)
    assert_within(got, np.broadcast_to(ref, got.shape), np.broadcast_to(bound, got.shape), str(act))
    assert_no_device_error()
