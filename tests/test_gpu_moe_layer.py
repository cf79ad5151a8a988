"""moe_layer on the GPU against its float64 definition (oracle.ffn), in two
steps: the fp16 hidden rows that the call leaves in its workspace against the
exact ones, and the output against the exact result from those hidden rows
(their E4M3 codes are then the same on both sides).  Guard-banded buffers,
NaN-filled before the call."""
import numpy as np
import pytest
import torch

from oracle import moe_hidden_ref, moe_out_ref
from fp8_quantized_generative_b200 import _lib
from fp8_quantized_generative_b200 import workloads as wl

from ffn_bounds import assert_within, moe_hidden_bound, moe_out_bound
from parity import Guards, assert_no_device_error, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


def layer(fq, E, K, F, N, gated, seed):
    up = 2 * F if gated else F
    Wu, su = fq.quantize_weight_per_channel(wl.random_f16((E, up, K), seed=seed, std=0.08).cuda())
    Wd, sd = fq.quantize_weight_per_channel(wl.random_f16((E, N, F), seed=seed + 1, std=0.08).cuda())
    return Wu, su, Wd, sd


def choices(T, E, topk, seed):
    experts = wl.route_top2(wl.random_f16((T, E), seed=seed).numpy(), topk).astype(np.int32)
    weights = np.random.default_rng(seed).random((T, topk), dtype=np.float32)
    return experts, weights


def check(fq, T, E, topk, K, F, N, act="silu", gated=False, use_res=True, seed=0, experts=None, in_place=False):
    X = wl.random_f16((T, K), seed=seed + 5).cuda()
    Wu, su, Wd, sd = layer(fq, E, K, F, N, gated, seed)
    ex, w = choices(T, E, topk, seed + 9) if experts is None else (np.asarray(experts, np.int32), None)
    if w is None:
        w = np.random.default_rng(seed).random((T, topk), dtype=np.float32)
    w = np.where(ex < 0, np.float32(np.nan), w)   # not read
    residual = wl.random_f16((T, N), seed=seed + 7).cuda()
    g = Guards()
    out = g((T, N), torch.float16, float("nan"), "out")
    ws = g((int(_lib.fp8q_moe_layer_workspace_bytes(T, topk, F, N)),), torch.uint8, 0xFF, "workspace")
    if in_place:
        out.copy_(residual)
    res = (out if in_place else residual) if use_res else None
    fq.moe_layer(X, torch.from_numpy(ex).cuda(), torch.from_numpy(w).cuda(), Wu, su, Wd, sd, activation=act,
                 gated=gated, residual=res, workspace=ws, out=out)
    what = f"T={T} E={E} k={topk} {K}-{F}-{N} {act} gated={gated}"
    g.check(what)
    assert_no_device_error()
    used = ex.reshape(-1) >= 0
    hidden = to_np(ws[:T * topk * F * 2].view(torch.float16)).reshape(T * topk, F)
    Wu_, su_, Wd_, sd_ = (to_np(t) for t in (Wu, su, Wd, sd))
    h, z, terms = moe_hidden_ref(to_np(X), ex, Wu_, su_, act, gated)
    assert_within(hidden[used], h[used], moe_hidden_bound(K, h, z, terms, gated)[used], what + " hidden")
    rr = to_np(residual) if use_res else None
    ref, terms = moe_out_ref(np.where(used[:, None], hidden, 0), ex, w, Wd_, sd_, rr)
    assert_within(to_np(out), ref, moe_out_bound(F, ref, terms, rr), what)
    return out


@pytest.mark.parametrize("T,E,topk,K,F,N", [
    (1, 1, 1, 16, 16, 8), (1, 8, 2, 128, 64, 136), (1, 64, 2, 2048, 1024, 2048), (2, 5, 5, 144, 272, 264),
    (8, 64, 4, 528, 80, 72), (13, 20, 3, 1040, 272, 1000), (16, 6, 2, 256, 48, 520), (17, 40, 8, 272, 144, 24),
    (33, 3, 1, 1296, 96, 392), (64, 64, 2, 512, 256, 512), (65, 12, 3, 208, 112, 88), (128, 16, 8, 160, 128, 104),
])
@pytest.mark.parametrize("gated", [False, True])
def test_shapes(fq, T, E, topk, K, F, N, gated):
    check(fq, T, E, topk, K, F, N, gated=gated, seed=T + K)


@pytest.mark.parametrize("act", [None, "none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_activations(fq, act, gated):
    check(fq, 6, 8, 2, 272, 144, 136, act=act, gated=gated, use_res=False)


@pytest.mark.parametrize("K,F", [(8192, 16), (16, 8192), (4096, 2048)])
def test_long_rows(fq, K, F):
    for T in (3, 40):
        check(fq, T, 4, 2, K, F, 136, seed=T)


@pytest.mark.parametrize("T,E,K,F,N,gated", [
    (128, 8, 8192, 2432, 8, False), (128, 8, 8192, 1216, 8, True), (128, 8, 16, 8192, 2432, False),
    (32, 64, 8176, 272, 16, False),
])
def test_longest_rows_with_many_units(fq, T, E, K, F, N, gated):
    """The longest rows beside the row lists of many choices, and enough units for wide ones."""
    check(fq, T, E, 8, K, F, N, gated=gated, seed=T + F)


@pytest.mark.parametrize("T", [9, 64, 128])
def test_all_tokens_to_one_expert(fq, T):
    """More rows than one segment holds."""
    ex = np.full((T, 2), 3, np.int32)
    ex[:, 1] = 1
    check(fq, T, 5, 2, 2064, 176, 264, experts=ex, seed=T)


def test_same_expert_twice_in_a_token(fq):
    check(fq, 5, 4, 3, 272, 80, 72, experts=[[2, 2, 2], [0, 1, 0], [3, 3, 1], [1, 1, 1], [2, 0, 2]])


@pytest.mark.parametrize("use_res", [False, True])
def test_padded_tokens_and_missing_choices(fq, use_res):
    ex = choices(12, 7, 3, 4)[0]
    ex[8:] = -1
    ex[2] = -1
    ex[5, 1] = -1
    out = check(fq, 12, 7, 3, 144, 96, 80, experts=ex, use_res=use_res)
    if not use_res:
        assert bool((out[8:] == 0).all()) and bool((out[2] == 0).all())


def test_no_token_has_an_expert(fq):
    check(fq, 4, 7, 2, 144, 96, 80, experts=np.full((4, 2), -1))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_large_negative_products(fq, act, gated):
    """Up projections from -2^9 to -2^84: hidden rows of zeros, whatever multiplies them."""
    T, K, F, N = 3, 64, 16, 16
    X = torch.full((T, K), 1.0, dtype=torch.float16, device="cuda")
    Wu, su = fq.quantize_weight_per_channel(torch.full((1, 2 * F if gated else F, K), 0.125, dtype=torch.float16,
                                                       device="cuda"))
    Wu[:, :F] |= 0x80
    su = su * torch.exp2(torch.arange(F, device="cuda") * 5.0 + 6.0).repeat(2 if gated else 1)
    if gated:
        su[:, F:] = 0.125 / 448
    Wd, sd = fq.quantize_weight_per_channel(wl.random_f16((1, N, F), seed=1).cuda())
    ws = fq.moe_layer_workspace(T, 1, F, N, "cuda")
    out = fq.moe_layer(X, torch.zeros((T, 1), dtype=torch.int32, device="cuda"), torch.ones((T, 1), device="cuda"),
                       Wu, su, Wd, sd, activation=act, gated=gated, workspace=ws)
    assert bool((ws[:T * F * 2].view(torch.float16) == 0).all())
    assert bool((out == 0).all())
    assert_no_device_error()


def test_residual_in_place(fq):
    check(fq, 10, 8, 2, 272, 144, 136, in_place=True)


def test_bad_expert_is_reported_and_adds_nothing(fq):
    Wu, su, Wd, sd = layer(fq, 4, 144, 96, 80, False, 1)
    X = wl.random_f16((2, 144), seed=2).cuda()
    w = torch.ones((2, 2), device="cuda")
    bad = fq.moe_layer(X, torch.tensor([[1, 4], [-2, 3]], dtype=torch.int32, device="cuda"), w, Wu, su, Wd, sd)
    assert fq.device_error() == 0x8
    good = fq.moe_layer(X, torch.tensor([[1, -1], [-1, 3]], dtype=torch.int32, device="cuda"), w, Wu, su, Wd, sd)
    assert fq.device_error() == 0
    assert torch.equal(bad, good)


def test_no_tokens(fq):
    Wu, su, Wd, sd = layer(fq, 4, 144, 96, 80, False, 1)
    out = fq.moe_layer(torch.empty((0, 144), dtype=torch.float16, device="cuda"),
                       torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                       torch.empty((0, 2), dtype=torch.float32, device="cuda"), Wu, su, Wd, sd)
    assert out.shape == (0, 80)


def test_repeats_bitwise_and_across_streams(fq):
    """The same call again, and two calls at once on two streams (a workspace each): the same bits."""
    T, E, topk, K, F, N = 24, 16, 4, 528, 272, 264
    Wu, su, Wd, sd = layer(fq, E, K, F, N, True, 3)
    X = [wl.random_f16((T, K), seed=s).cuda() for s in (1, 2)]
    pick = [tuple(torch.from_numpy(a).cuda() for a in choices(T, E, topk, s)) for s in (3, 4)]
    ref = [fq.moe_layer(x, *c, Wu, su, Wd, sd, gated=True) for x, c in zip(X, pick)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fq.moe_layer(X[i], *pick[i], Wu, su, Wd, sd, gated=True))
    torch.cuda.synchronize()
    for i in range(2):
        for y in got[i]:
            assert torch.equal(y.view(torch.int16), ref[i].view(torch.int16))


def test_two_graphs_share_a_workspace(fq):
    """Two captured layers on one workspace, replayed in turn with new inputs."""
    T, E, topk, K, F, N = 6, 8, 2, 272, 144, 136
    Wu, su, Wd, sd = layer(fq, E, K, F, N, False, 3)
    ws = fq.moe_layer_workspace(T, topk, F, N, "cuda")
    X = torch.zeros((T, K), dtype=torch.float16, device="cuda")
    ex = torch.zeros((T, topk), dtype=torch.int32, device="cuda")
    w = torch.zeros((T, topk), dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphs, outs = [], []
        for act in ("silu", "relu"):
            out = torch.zeros((T, N), dtype=torch.float16, device="cuda")
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                fq.moe_layer(X, ex, w, Wu, su, Wd, sd, activation=act, workspace=ws, out=out)
            graphs.append(gr)
            outs.append(out)
        for seed in (5, 6, 7):
            X.copy_(wl.random_f16((T, K), seed=seed))
            a, b = choices(T, E, topk, seed)
            ex.copy_(torch.from_numpy(a))
            w.copy_(torch.from_numpy(b))
            for i, act in enumerate(("silu", "relu")):
                graphs[i].replay()
            s.synchronize()
            for i, act in enumerate(("silu", "relu")):
                assert torch.equal(outs[i], fq.moe_layer(X, ex, w, Wu, su, Wd, sd, activation=act))


def test_block_of_dense_ffn_router_and_moe(fq):
    """The operators together, as a decode step of a block uses them: dense FFN
    (up + GELU, down + residual), gate, router, MoE FFN + residual; against the
    float64 definitions fed with the device's fp16 values at each step."""
    from ffn_bounds import linear_epilogue_bound
    from oracle import linear_epilogue_ref, route_ref
    T, D, H, E, topk, F = 12, 272, 528, 16, 2, 144
    x = wl.random_f16((T, D), seed=1).cuda()
    W1, s1 = fq.quantize_weight_per_channel(wl.random_f16((H, D), seed=2, std=0.06).cuda())
    W2, s2 = fq.quantize_weight_per_channel(wl.random_f16((D, H), seed=3, std=0.06).cuda())
    b1, b2 = wl.random_f16((H,), seed=4).cuda(), wl.random_f16((D,), seed=5).cuda()
    gate = wl.random_f16((E, D), seed=6, std=0.1).cuda()
    Wu, su, Wd, sd = layer(fq, E, D, F, D, True, 7)

    q1 = fq.quantize_rows_dynamic(x)
    h = fq.linear_epilogue(*q1, W1, s1, bias=b1, activation="gelu")
    q2 = fq.quantize_rows_dynamic(h)
    y = fq.linear_epilogue(*q2, W2, s2, bias=b2, residual=x)
    logits = y @ gate.t()
    r = fq.moe_route(logits, topk)
    ws = fq.moe_layer_workspace(T, topk, F, D, "cuda")
    out = fq.moe_layer(y, r.experts, r.weights, Wu, su, Wd, sd, gated=True, residual=y, workspace=ws)
    assert_no_device_error()

    n = to_np
    ref, terms = linear_epilogue_ref(n(q1[0]), n(q1[1]), n(W1), n(s1), n(b1), "gelu")
    assert_within(n(h), ref, linear_epilogue_bound(D, ref, terms + np.abs(n(b1).astype(np.float64))), "up")
    ref, terms = linear_epilogue_ref(n(q2[0]), n(q2[1]), n(W2), n(s2), n(b2), None, n(x))
    assert_within(n(y), ref, linear_epilogue_bound(H, ref, terms + np.abs(n(b2).astype(np.float64)), n(x)), "down")
    rr = route_ref(n(logits), topk)
    assert np.array_equal(n(r.experts), rr["experts"])
    hidden = n(ws[:T * topk * F * 2].view(torch.float16)).reshape(T * topk, F)
    ht, z, terms = moe_hidden_ref(n(y), n(r.experts), n(Wu), n(su), "silu", True)
    assert_within(hidden, ht, moe_hidden_bound(D, ht, z, terms, True), "hidden")
    ref, terms = moe_out_ref(hidden, n(r.experts), n(r.weights), n(Wd), n(sd), n(y))
    assert_within(n(out), ref, moe_out_bound(F, ref, terms, n(y)), "out")


def test_agrees_with_the_grouped_path(fq):
    """Without activation the layer is the grouped chain (dispatch, up, quantize, down + combine):
    the same codes, so the difference is the chain's fp16 rounding of each contribution."""
    T, E, topk, K, F, N = 32, 8, 2, 256, 128, 264
    Wu, su, Wd, sd = layer(fq, E, K, F, N, False, 3)
    X = wl.random_f16((T, K), seed=8).cuda()
    r = fq.moe_route(wl.random_f16((T, E), seed=9).cuda(), topk)
    a = fq.moe_layer(X, r.experts, r.weights, Wu, su, Wd, sd, activation=None)
    Xg, sg = fq.quantize_rows_dispatch(X, r.token_rows, T * topk)
    H = fq.moe_grouped_linear(Xg, sg, r.offsets, Wu, su)
    Hq, sh = fq.quantize_rows_dynamic(H)
    b = fq.moe_grouped_linear_combine(Hq, sh, r.offsets, Wd, sd, r.row_token, r.row_weight, T)
    a, b = to_np(a).astype(np.float64), to_np(b).astype(np.float64)
    assert np.linalg.norm(a - b) <= 2.0 ** -9 * np.linalg.norm(b)
