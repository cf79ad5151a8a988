"""moe_route past 1024 tokens (two launches) with many experts: every index equal
to the plain router's, weights within the rounding of their formula."""
import numpy as np
import pytest
import torch

from oracle import route_ref
from fp8_quantized_generative_b200 import workloads as wl

from parity import assert_no_device_error, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


@pytest.mark.parametrize("T,E,topk", [(1025, 65, 8), (1100, 129, 6), (4097, 128, 2), (2051, 257, 8), (1537, 512, 5),
                                      (1301, 513, 7), (1027, 1000, 8), (2049, 1024, 3), (5003, 1, 1), (4111, 2, 2)])
@pytest.mark.parametrize("renormalize,skewed", [(True, False), (False, True)])
def test_many(fq, T, E, topk, renormalize, skewed):
    logits = wl.random_f16((T, E), seed=T + E)
    if skewed:   # most tokens choose the same few experts; some logits are switched off
        logits[: T * 3 // 4, : max(1, E // 50)] += 8.0
        logits[::7, E // 2:E - 1] = float("-inf")
    r = fq.moe_route(logits.cuda(), topk, renormalize=renormalize)
    L = logits.numpy()
    ref = route_ref(L, topk, renormalize)
    for name in ("experts", "offsets", "row_token", "token_rows"):
        got = to_np(getattr(r, name))
        assert got.dtype == np.int32 and np.array_equal(got, ref[name]), name
    # e^d: d exact to 2^-24 |d|, the function to 2 steps (2^-22); a sum of E terms rounded half a step each at
    # most (E / 32 a lane and five shuffles); the division
    d = np.abs(np.take_along_axis(L.astype(np.float64), ref["experts"].astype(np.int64), 1)
               - L.astype(np.float64).max(1, keepdims=True))
    d = np.where(np.isfinite(d), d, 0.0)
    bound = 2.0 ** -24 * (d + 16 + E / 32 + 5) * ref["weights"] + 2.0 ** -126
    assert np.all(np.abs(to_np(r.weights).astype(np.float64) - ref["weights"]) <= bound)
    assert np.array_equal(to_np(r.row_weight)[to_np(r.token_rows).reshape(-1)], to_np(r.weights).reshape(-1))
    assert_no_device_error()
