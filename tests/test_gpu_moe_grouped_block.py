"""A gated MoE FFN past moe_layer's token limit, as the documentation has it: router,
dispatch, grouped up projection, the gate in torch, grouped down projection with the
combine, residual; against the float64 definition from the hidden rows."""
import numpy as np
import pytest
import torch

from oracle import moe_out_ref
from fp8_quantized_generative_b200 import workloads as wl

from ffn_bounds import F16_HALF, F16_TINY, ONE_OPS, assert_within, sum_bound
from parity import assert_no_device_error, to_np

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,E", [(129, 6), (300, 16), (61, 3)])
def test_gated_block(T, E):
    import fp8_quantized_generative_b200 as fq
    topk, K, F = 2, 272, 144
    X = wl.random_f16((T, K), seed=T).cuda()
    Wu, su = fq.quantize_weight_per_channel(wl.random_f16((E, 2 * F, K), seed=2, std=0.08).cuda())
    Wd, sd = fq.quantize_weight_per_channel(wl.random_f16((E, K, F), seed=3, std=0.08).cuda())
    r = fq.moe_route(wl.random_f16((T, E), seed=4).cuda(), topk)
    Xg, sg = fq.quantize_rows_dispatch(X, r.token_rows, T * topk)
    Z = fq.moe_grouped_linear(Xg, sg, r.offsets, Wu, su)
    H = torch.nn.functional.silu(Z[:, :F]) * Z[:, F:]
    out = X + fq.moe_grouped_linear_combine(*fq.quantize_rows_dynamic(H), r.offsets, Wd, sd, r.row_token, r.row_weight, T)
    assert_no_device_error()
    experts, hidden = to_np(r.experts), to_np(H)[to_np(r.token_rows).reshape(-1)]   # by (token, choice)
    ref, terms = moe_out_ref(hidden, experts, to_np(r.weights), to_np(Wd), to_np(sd), to_np(X))
    parts = 0.0   # sum of the contributions' absolute values
    for j in range(topk):
        only = np.where(np.arange(topk) == j, experts, -1)
        parts = parts + np.abs(moe_out_ref(hidden, only, to_np(r.weights), to_np(Wd), to_np(sd))[0])
    # three fp16 roundings: each contribution, their sum, the sum with the residual; each of a value that
    # may lie `err` from the exact one
    err = sum_bound(F, terms) + ONE_OPS * terms
    err = err + F16_HALF * (parts + err) + topk * F16_TINY
    err = err + F16_HALF * (parts + err) + F16_TINY
    err = err + F16_HALF * (np.abs(ref) + err) + F16_TINY
    assert_within(to_np(out), ref, err, "out")
