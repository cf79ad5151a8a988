"""Pins of the FFN oracle (oracle/ffn.py): closed forms, hand-worked cases,
torch's own functions in float64, and plain restatements."""
import math

import numpy as np
import pytest
import torch

from oracle import (activation_ref, e4m3_encode, linear_epilogue_ref, linear_ref, moe_layer_ref, moe_out_ref, moe_ref,
                    quant_rows, route_ref)
from fp8_quantized_generative_b200 import workloads as wl


@pytest.mark.parametrize("name,fn", [
    ("none", lambda z: z), (None, lambda z: z), ("relu", torch.relu), ("gelu", torch.nn.functional.gelu),
    ("gelu_tanh", lambda z: torch.nn.functional.gelu(z, approximate="tanh")), ("silu", torch.nn.functional.silu)])
def test_activations_against_torch(name, fn):
    z = np.linspace(-12, 12, 4001)
    ref = fn(torch.from_numpy(z)).numpy()
    assert np.allclose(activation_ref(z, name), ref, rtol=1e-12, atol=1e-14)   # torch's gelu cancels in its tail
    with pytest.raises(ValueError):
        activation_ref(z, "tanh")


def test_epilogue_by_hand():
    # x = (1, 2), w rows (1, 1) and (2, -1); scales 0.5 and (2, 4): z = (3, 0) + bias (-4, 1)
    Xq = e4m3_encode(np.array([[1.0, 2.0]], np.float32))
    Wq = e4m3_encode(np.array([[1.0, 1.0], [2.0, -1.0]], np.float32))
    y, terms = linear_epilogue_ref(Xq, [0.5], Wq, [2.0, 4.0], bias=[-4.0, 1.0], activation="relu", residual=[[10.0, 20.0]])
    assert y.tolist() == [[10.0, 21.0]] and terms.tolist() == [[3.0, 8.0]]


@pytest.mark.parametrize("x_fmt", ["e4m3", "e5m2"])
def test_epilogue_without_parts_is_the_linear(x_fmt):
    Xq, s_x = quant_rows(wl.random_f16((5, 48), 1).numpy(), x_fmt)
    Wq, s_w = quant_rows(wl.random_f16((7, 48), 2).numpy())
    y, _ = linear_epilogue_ref(Xq, s_x, Wq, s_w, x_fmt=x_fmt)
    assert np.array_equal(y.astype(np.float16), linear_ref(Xq, s_x, Wq, s_w, x_fmt))


def test_route_by_hand():
    inf, nan = math.inf, math.nan
    L = np.array([[0, 2, 2, 1], [-inf, nan, -inf, -inf], [inf, 0, inf, 5], [nan, -inf, 3, nan]], np.float16)
    r = route_ref(L, 2)
    assert r["experts"].tolist() == [[1, 2], [0, 2], [0, 2], [2, 1]]
    assert r["weights"].tolist() == [[0.5, 0.5], [0, 0], [0.5, 0.5], [1, 0]]
    assert r["offsets"].tolist() == [0, 2, 4, 8, 8]
    assert r["row_token"].tolist() == [1, 2, 0, 3, 0, 1, 2, 3]
    assert r["token_rows"].tolist() == [[2, 4], [0, 5], [1, 6], [7, 3]]
    a = route_ref(L[:1], 2, renormalize=False)["weights"][0]
    total = 2 + math.exp(-2) + math.exp(-1)
    assert np.allclose(a, 1 / total, rtol=1e-15)


def test_route_matches_the_host_harness():
    L = wl.random_f16((200, 24), 5).numpy()
    r = route_ref(L, 2)
    experts = wl.route_top2(L, 2)
    row_token, offsets = wl.group_by_expert(experts, 24)
    assert np.array_equal(r["experts"], experts) and np.array_equal(r["offsets"], offsets)
    assert np.array_equal(r["row_token"], row_token)
    assert np.allclose(r["weights"], wl.gate_weights(L, experts), rtol=1e-6)
    assert np.array_equal(np.sort(r["token_rows"], 1), wl.token_rows(row_token, 200, 2))


def test_layer_without_activation_is_the_grouped_chain():
    T, E, K, F, N = 9, 4, 32, 16, 24
    X = wl.random_f16((T, K), 1).numpy()
    Wu, su = (a.reshape(s) for a, s in zip(quant_rows(wl.random_f16((E * F, K), 2).numpy()), ((E, F, K), (E, F))))
    Wd, sd = (a.reshape(s) for a, s in zip(quant_rows(wl.random_f16((E * N, F), 3).numpy()), ((E, N, F), (E, N))))
    r = route_ref(wl.random_f16((T, E), 4).numpy(), 2)
    out, h = moe_layer_ref(X, r["experts"], r["weights"], Wu, su, Wd, sd, None)
    xq, sx = quant_rows(X)
    H = moe_ref(xq[r["row_token"]], sx[r["row_token"]], r["offsets"], Wu, su)
    assert np.array_equal(H[r["token_rows"].reshape(-1)], h)
    hq, sh = quant_rows(H)
    y = moe_ref(hq, sh, r["offsets"], Wd, sd).astype(np.float64)   # rounded to fp16 there, exact here
    ref, bound = np.zeros((T, N)), np.zeros((T, N))
    for row, t in enumerate(r["row_token"]):
        ref[t] += r["row_weight"][row] * y[row]
        # y16 is y to half an fp16 step: |y16 - y| <= 2^-11 |y| <= 2^-11 |y16| / (1 - 2^-11) (or 2^-25 below
        # the normal range), and the sums are the same but for float64 rounding
        bound[t] += r["row_weight"][row] * (2.0 ** -11 * (1 + 2.0 ** -10) * np.abs(y[row]) + 2.0 ** -25)
    assert np.all(np.abs(out - ref) <= bound + 1e-12)


def test_gated_and_missing_choices_by_hand():
    # one expert, K = 1 value (padded to 2): gate weight 1, up weight 2; hidden = relu(3) * 6 = 18; down 0.5 -> 9
    X = np.array([[3.0, 0.0], [-3.0, 0.0], [1.0, 0.0]], np.float16)
    Wu = e4m3_encode(np.array([[448.0, 0.0], [448.0, 0.0]], np.float32))[None]
    su = np.array([[1 / 448.0, 2 / 448.0]])
    Wd, sd = e4m3_encode(np.array([[448.0]], np.float32))[None], np.array([[0.5 / 448.0]])
    ex = np.array([[0, -1], [0, 0], [-1, -1]])
    w = np.array([[2.0, np.nan], [1.0, 1.0], [np.nan, np.nan]])
    out, h = moe_layer_ref(X, ex, w, Wu, su, Wd, sd, "relu", gated=True, residual=[[1.0], [2.0], [3.0]])
    assert np.allclose(h[[0, 2], 0].astype(float), [18.0, 0.0]) and np.all(h[[1, 4, 5]] == 0)
    assert np.allclose(out[:, 0], [2.0 * 9.0 + 1.0, 2.0, 3.0], rtol=1e-6)
    same, _ = moe_out_ref(h, ex, w, Wd, sd)
    assert np.allclose(same[:, 0], [18.0, 0.0, 0.0], rtol=1e-6)
