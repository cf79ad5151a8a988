"""moe_layer at sizes that reach every form of its kernels (tests/moe_forms.py),
with even choices and with one expert that every token chose; against the
float64 definition (oracle.ffn)."""
import numpy as np
import pytest
import torch

from oracle import moe_hidden_ref, moe_out_ref
from fp8_quantized_generative_b200 import _lib
from fp8_quantized_generative_b200 import workloads as wl

from ffn_bounds import assert_within, moe_hidden_bound, moe_out_bound
from moe_forms import LAYERS
from parity import Guards, assert_no_device_error, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("hot", [False, True])
@pytest.mark.parametrize("layer", LAYERS, ids=lambda c: "-".join(map(str, c)))
def test_forms(fq, layer, hot):
    T, E, topk, K, F, N, gated = layer
    seed, g = T + E + F, np.random.default_rng(T + N)
    X = wl.random_f16((T, K), seed=seed).cuda()
    Wu, su = fq.quantize_weight_per_channel(wl.random_f16((E, 2 * F if gated else F, K), seed=seed + 1, std=0.08).cuda())
    Wd, sd = fq.quantize_weight_per_channel(wl.random_f16((E, N, F), seed=seed + 2, std=0.08).cuda())
    ex = g.integers(0, E, (T, topk)).astype(np.int32)
    if hot:
        ex[:, 0] = E // 2
    ex[g.random((T, topk)) < 0.05] = -1
    w = np.where(ex < 0, np.float32(np.nan), g.random((T, topk), dtype=np.float32))
    residual = wl.random_f16((T, N), seed=seed + 3).cuda()
    guards = Guards()
    out = guards((T, N), torch.float16, float("nan"), "out")
    ws = guards((int(_lib.fp8q_moe_layer_workspace_bytes(T, topk, F, N)),), torch.uint8, 0xFF, "workspace")
    args = (X, torch.from_numpy(ex).cuda(), torch.from_numpy(w).cuda(), Wu, su, Wd, sd)
    call = dict(activation="gelu", gated=gated, residual=residual)
    fq.moe_layer(*args, **call, workspace=ws, out=out)
    guards.check(str(layer))
    assert_no_device_error()
    used = ex.reshape(-1) >= 0
    hidden = to_np(ws[:T * topk * F * 2].view(torch.float16)).reshape(T * topk, F)
    h, z, terms = moe_hidden_ref(to_np(X), ex, to_np(Wu), to_np(su), "gelu", gated)
    assert_within(hidden[used], h[used], moe_hidden_bound(K, h, z, terms, gated)[used], "hidden")
    ref, terms = moe_out_ref(np.where(used[:, None], hidden, 0), ex, w, to_np(Wd), to_np(sd), to_np(residual))
    assert_within(to_np(out), ref, moe_out_bound(F, ref, terms, to_np(residual)), "out")
    for _ in range(5):   # the same bits in every run: no atomic's order reaches them
        assert torch.equal(bits(fq.moe_layer(*args, **call)), bits(out))
