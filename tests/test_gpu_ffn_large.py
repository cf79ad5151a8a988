"""linear_epilogue, moe_layer and moe_route where offsets pass 32 bits or the sizes are the
largest: outputs, residuals and expert weights of more than 2^31 elements, 2^22 tokens."""
import numpy as np
import pytest
import torch

from oracle import linear_epilogue_ref, moe_hidden_ref, moe_out_ref
from fp8_quantized_generative_b200 import workloads as wl

from ffn_bounds import assert_within, linear_epilogue_bound, moe_hidden_bound, moe_out_bound
from parity import assert_no_device_error, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    yield m
    torch.cuda.empty_cache()


def codes(shape, seed):
    """E4M3 codes of moderate finite values, either sign."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.randint(0x20, 0x48, shape, generator=g, dtype=torch.uint8, device="cuda")
    return c.bitwise_or_(torch.randint(0, 2, shape, generator=g, dtype=torch.uint8, device="cuda").mul_(0x80))


@pytest.mark.parametrize("M,N", [(66000, 33000), (65, 1 << 25), (16, (1 << 27) + 8)])
def test_outputs_past_2_31_elements(fq, M, N):
    assert M * N > 2 ** 31
    K = 16
    Xq, Wq = codes((M, K), 1), codes((N, K), 2)
    s_x = torch.linspace(0.5, 1.5, M, device="cuda")
    s_w = torch.linspace(0.01, 0.02, N, device="cuda")
    bias = torch.linspace(-1, 1, N, device="cuda").half()
    Y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    n = min(M * N, 1 << 26)
    pattern = torch.randn(n, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").half()
    flat = Y.view(-1)
    for at in range(0, M * N, n):
        flat[at:at + n] = pattern[:min(n, M * N - at)]
    rows, cols = [0, M // 2, M - 2, M - 1], torch.cat([torch.arange(0, N, 4099), torch.arange(N - 40, N)]).cuda()
    residual = Y[rows][:, cols].clone()
    fq.linear_epilogue(Xq, s_x, Wq, s_w, bias=bias, activation="silu", residual=Y, out=Y)
    assert_no_device_error()
    got = Y[rows][:, cols]
    b, r = to_np(bias[cols]), to_np(residual)
    y, terms = linear_epilogue_ref(to_np(Xq[rows]), to_np(s_x[rows]), to_np(Wq[cols]), to_np(s_w[cols]), b, "silu", r)
    terms = terms + np.abs(b.astype(np.float64))[None, :]
    assert_within(to_np(got), y, linear_epilogue_bound(K, y, terms, r), f"{M}x{N}")


def test_expert_weights_past_2_31_bytes(fq):
    T, E, topk, K, F, N = 3, 80, 2, 8192, 2048, 24
    Wu, Wd = codes((E, 2 * F, K), 1), codes((E, N, F), 2)
    assert Wu.numel() > 2 ** 31
    su = torch.linspace(0.001, 0.002, E * 2 * F, device="cuda").view(E, 2 * F)
    sd = torch.linspace(0.01, 0.02, E * N, device="cuda").view(E, N)
    X = wl.random_f16((T, K), seed=4).cuda()
    ex = np.array([[79, 0], [78, 79], [79, -1]], np.int32)
    w = np.array([[0.25, 0.75], [0.5, 0.5], [1.0, np.nan]], np.float32)
    ws = fq.moe_layer_workspace(T, topk, F, N, "cuda")
    out = fq.moe_layer(X, torch.from_numpy(ex).cuda(), torch.from_numpy(w).cuda(), Wu, su, Wd, sd, gated=True, workspace=ws)
    assert_no_device_error()
    pick = [0, 78, 79]   # the oracle gets the chosen experts alone
    small = np.searchsorted(pick, ex).astype(np.int32)
    small[ex < 0] = -1
    used = ex.reshape(-1) >= 0
    hidden = to_np(ws[:T * topk * F * 2].view(torch.float16)).reshape(T * topk, F)
    h, z, terms = moe_hidden_ref(to_np(X), small, to_np(Wu[pick]), to_np(su[pick]), "silu", True)
    assert_within(hidden[used], h[used], moe_hidden_bound(K, h, z, terms, True)[used], "hidden")
    ref, terms = moe_out_ref(np.where(used[:, None], hidden, 0), small, w, to_np(Wd[pick]), to_np(sd[pick]))
    assert_within(to_np(out), ref, moe_out_bound(F, ref, terms), "out")


def test_widest_layer(fq):
    """N = 2^20 outputs, 128 tokens, eight choices: 2^30 partial sums."""
    T, E, topk, K, F, N = 128, 3, 8, 48, 16, 1 << 20
    Wu, Wd = codes((E, F, K), 1), codes((E, N, F), 2)
    su, sd = torch.full((E, F), 0.01, device="cuda"), torch.linspace(0.01, 0.02, E * N, device="cuda").view(E, N)
    X = wl.random_f16((T, K), seed=4).cuda()
    g = np.random.default_rng(5)
    ex = g.integers(-1, E, (T, topk)).astype(np.int32)
    w = g.random((T, topk), dtype=np.float32)
    ws = fq.moe_layer_workspace(T, topk, F, N, "cuda")
    out = fq.moe_layer(X, torch.from_numpy(ex).cuda(), torch.from_numpy(w).cuda(), Wu, su, Wd, sd, activation="relu",
                       workspace=ws)
    assert_no_device_error()
    cols = torch.cat([torch.arange(0, N, 8191), torch.arange(N - 24, N)]).cuda()
    used = ex.reshape(-1) >= 0
    hidden = np.where(used[:, None], to_np(ws[:T * topk * F * 2].view(torch.float16)).reshape(T * topk, F), 0)
    ref, terms = moe_out_ref(hidden, ex, w, to_np(Wd[:, cols].contiguous()), to_np(sd[:, cols].contiguous()))
    assert_within(to_np(out[:, cols].contiguous()), ref, moe_out_bound(F, ref, terms), "out")


@pytest.mark.parametrize("E,topk", [(8, 2), (3, 3)])
def test_route_of_most_tokens(fq, E, topk):
    """2^22 tokens; the rows against torch's stable sorts."""
    T = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(E)
    logits = torch.randn((T, E), generator=g, device="cuda").half()
    logits[:T // 2, 1] = 9.0
    r = fq.moe_route(logits, topk)
    order = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    assert torch.equal(r.experts, order.indices[:, :topk].int())
    flat = r.experts.reshape(-1)
    place = torch.sort(flat, stable=True).indices   # grouped row -> (token, choice)
    assert torch.equal(r.offsets[1:], torch.cumsum(torch.bincount(flat, minlength=E), 0).int()) and int(r.offsets[0]) == 0
    assert torch.equal(r.row_token, (place // topk).int())
    assert torch.equal(r.token_rows.reshape(-1)[place], torch.arange(T * topk, dtype=torch.int32, device="cuda"))
    assert torch.equal(r.row_weight, r.weights.reshape(-1)[place])
    assert float((r.weights.sum(1) - 1).abs().max()) <= (topk + 4) * 2.0 ** -24   # each weight and the sum rounded
    assert_no_device_error()
