"""moe_route on the GPU against the plain router of oracle.ffn: every index
equal, weights within the rounding of their formula."""
import numpy as np
import pytest
import torch

from oracle import route_ref
from fp8_quantized_generative_b200 import _lib
from fp8_quantized_generative_b200 import workloads as wl

from parity import Guards, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


def check(fq, logits, topk, renormalize=True):
    r = fq.moe_route(logits.cuda(), topk, renormalize=renormalize)
    L = logits.numpy()
    ref = route_ref(L, topk, renormalize)
    for name in ("experts", "offsets", "row_token", "token_rows"):
        got = to_np(getattr(r, name))
        assert got.dtype == np.int32 and np.array_equal(got, ref[name]), name
    # exp within 2 steps (2^-22), its argument rounded by 2^-24 |d|, at most 64 half steps of the sum and division
    top = np.where(np.isnan(L), -np.inf, L.astype(np.float64)).max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        d = np.abs(np.take_along_axis(L.astype(np.float64), ref["experts"].astype(np.int64), 1) - top)
    d = np.where(np.isfinite(d), d, 0.0)
    bound = (2.0 ** -24 * (80 + d)) * ref["weights"] + 2.0 ** -126
    assert np.all(np.abs(to_np(r.weights).astype(np.float64) - ref["weights"]) <= bound)
    # the grouped copy is the same fp32 value
    tr = to_np(r.token_rows).reshape(-1)
    assert np.array_equal(to_np(r.row_weight)[tr], to_np(r.weights).reshape(-1))
    return r


@pytest.mark.parametrize("T,E,topk", [(1, 1, 1), (1, 64, 2), (2, 3, 3), (7, 8, 8), (33, 65, 4), (64, 160, 6),
                                      (65, 64, 2), (100, 1024, 8), (300, 129, 1), (1000, 160, 6), (4099, 30, 3),
                                      (257, 513, 7), (64, 1000, 8)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_shapes(fq, T, E, topk, renormalize):
    check(fq, wl.random_f16((T, E), seed=T + E + topk), topk, renormalize)


def test_full_size_matches_the_host_grouping(fq):
    m = wl.moe(with_weights=False)
    r = check(fq, m.logits, wl.MOE_TOPK)
    assert np.array_equal(to_np(r.offsets), m.offsets)
    assert np.array_equal(to_np(r.row_token), m.token_of_row)
    assert np.allclose(to_np(r.row_weight), m.row_weight, rtol=1e-6, atol=0)


@pytest.mark.parametrize("T", [50, 500])
def test_ties(fq, T):
    g = torch.Generator().manual_seed(T)
    logits = torch.randint(-2, 3, (T, 96), generator=g).half()
    logits[logits == 0] = -0.0   # both zeros, equal in rank
    logits[::3][logits[::3] == 0] = 0.0
    check(fq, logits, 5)


@pytest.mark.parametrize("T", [40, 200])
@pytest.mark.parametrize("renormalize", [True, False])
def test_masks_infinities_and_nan(fq, T, renormalize):
    logits = wl.random_f16((T, 40), seed=T)
    logits[:, 5:25] = float("-inf")
    logits[0] = float("-inf")                 # nothing left
    logits[1] = float("nan")
    logits[2, 3:] = float("-inf")             # fewer than topk
    logits[3] = -65504.0                      # the type's lowest value everywhere
    logits[4, 7] = 65504.0
    logits[5, [2, 30]] = float("inf")
    logits[6, ::2] = float("nan")
    logits[7] = torch.tensor([float("nan"), float("-inf")] * 20).half()
    check(fq, logits, 4, renormalize)


def test_every_token_to_the_same_experts(fq):
    logits = torch.full((3000, 64), -1.0).half()
    logits[:, 9] = 2.0
    logits[:, 63] = 1.0
    r = check(fq, logits, 2)
    assert to_np(r.offsets)[10] - to_np(r.offsets)[9] == 3000


def test_no_tokens(fq):
    r = fq.moe_route(torch.empty((0, 16), dtype=torch.float16, device="cuda"), 2)
    assert r.experts.shape == (0, 2) and np.array_equal(to_np(r.offsets), np.zeros(17, np.int32))


@pytest.mark.parametrize("T,E,topk", [(3, 5, 2), (500, 70, 3)])
def test_guarded_outputs(fq, T, E, topk):
    logits = wl.random_f16((T, E), seed=3).cuda()
    g = Guards()
    i32, f32 = torch.int32, torch.float32
    ex, tr = g((T, topk), i32, -7, "experts"), g((T, topk), i32, -7, "token_rows")
    w, rw = g((T, topk), f32, float("nan"), "weights"), g((T * topk,), f32, float("nan"), "row_weight")
    off, rt = g((E + 1,), i32, -7, "offsets"), g((T * topk,), i32, -7, "row_token")
    ws = g((max(1, _lib.fp8q_moe_route_workspace_words(T, E)),), i32, -7, "workspace")
    st = _lib.fp8q_moe_route(logits.data_ptr(), T, E, topk, 1, ex.data_ptr(), w.data_ptr(), off.data_ptr(),
                             rt.data_ptr(), rw.data_ptr(), tr.data_ptr(), ws.data_ptr(),
                             torch.cuda.current_stream().cuda_stream)
    assert st == _lib.FP8Q_OK
    g.check("route")
    ref = route_ref(logits.cpu().numpy(), topk)
    assert np.array_equal(to_np(tr), ref["token_rows"]) and np.array_equal(to_np(off), ref["offsets"])
    assert bool(torch.isfinite(w).all()) and bool(torch.isfinite(rw).all())


def test_captured_and_replayed_with_new_logits(fq):
    T, E, topk = 200, 64, 2
    logits = wl.random_f16((T, E), seed=1).cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            r = fq.moe_route(logits, topk)
        for seed in (2, 3):
            new = wl.random_f16((T, E), seed=seed)
            logits.copy_(new)
            graph.replay()
            s.synchronize()
            ref = route_ref(new.numpy(), topk)
            assert np.array_equal(to_np(r.token_rows), ref["token_rows"])
            assert np.array_equal(to_np(r.row_token), ref["row_token"])


def test_feeds_the_grouped_path(fq):
    """logits -> moe_route -> dispatch -> grouped linear + combine equals the host-routed path bit for bit."""
    T, E, topk, K, N = 300, 16, 2, 256, 264
    logits = wl.random_f16((T, E), seed=11)
    X = wl.random_f16((T, K), seed=12).cuda()
    Wq, s_w = fq.quantize_weight_per_channel(wl.random_f16((E, N, K), seed=13, std=0.05).cuda())
    r = fq.moe_route(logits.cuda(), topk)
    Xg, sg = fq.quantize_rows_dispatch(X, r.token_rows, T * topk)
    got = fq.moe_grouped_linear_combine(Xg, sg, r.offsets, Wq, s_w, r.row_token, r.row_weight, T)
    row_token, offsets = wl.group_by_expert(wl.route_top2(logits.numpy(), topk), E)
    Xq, s_x = fq.quantize_rows_dynamic(X)
    rt = torch.from_numpy(row_token).cuda()
    ref = fq.moe_grouped_linear_combine(Xq[rt].contiguous(), s_x[rt].contiguous(), torch.from_numpy(offsets).cuda(), Wq,
                                        s_w, rt.int(), r.row_weight, T)
    assert torch.equal(got.view(torch.int16), ref.view(torch.int16))
    assert fq.device_error() == 0
