"""linear_epilogue on the GPU against its float64 definition (oracle.ffn),
every output element within the bound of tests/ffn_bounds.py, in guard-banded
buffers that start as NaN."""
import numpy as np
import pytest
import torch

from oracle import linear_epilogue_ref
from fp8_quantized_generative_b200 import workloads as wl

from ffn_bounds import assert_within, linear_epilogue_bound
from parity import Guards, assert_no_device_error, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


def inputs(fq, M, N, K, seed, x_fmt="e4m3", w_std=0.05):
    Xq, s_x = fq.quantize_rows_dynamic(wl.random_f16((M, K), seed=seed).cuda(), fmt=x_fmt)
    Wq, s_w = fq.quantize_weight_per_channel(wl.random_f16((N, K), seed=seed + 1, std=w_std).cuda())
    bias = wl.random_f16((N,), seed=seed + 2, std=0.5).cuda()
    residual = wl.random_f16((M, N), seed=seed + 3).cuda()
    return Xq, s_x, Wq, s_w, bias, residual


def check(fq, M, N, K, act, use_bias, use_res, seed=0, x_fmt="e4m3", in_place=False):
    Xq, s_x, Wq, s_w, bias, residual = inputs(fq, M, N, K, seed, x_fmt)
    g = Guards()
    Y = g((M, N), torch.float16, float("nan"), "Y")
    res = residual
    if in_place:
        Y.copy_(residual)
        res = Y
    out = fq.linear_epilogue(Xq, s_x, Wq, s_w, bias=bias if use_bias else None, activation=act,
                             residual=res if use_res else None, out=Y, x_fmt=x_fmt)
    torch.cuda.synchronize()
    what = f"{M}x{N}x{K} {act} bias={use_bias} residual={use_res} {x_fmt}"
    g.check(what)
    assert out.data_ptr() == Y.data_ptr()
    rb, rr = (to_np(bias) if use_bias else None), (to_np(residual) if use_res else None)
    y, terms = linear_epilogue_ref(*(to_np(t) for t in (Xq, s_x, Wq, s_w)), rb, act, rr, x_fmt)
    if rb is not None:
        terms = terms + np.abs(rb.astype(np.float64))[None, :]   # the bias addition's rounding
    assert_within(to_np(Y), y, linear_epilogue_bound(K, y, terms, rr), what)
    assert_no_device_error()
    return Y


# one row to several tiles, sizes cut on every side, each kernel (16, 32, 64, 128 padded rows; row pairs)
SHAPES = [(1, 8, 16), (1, 4096, 4096), (5, 136, 48), (16, 1000, 272), (17, 264, 1040), (33, 520, 528),
          (65, 128, 2048), (128, 392, 656), (129, 8, 64), (300, 520, 272), (257, 1000, 1040), (1031, 776, 528)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes_with_everything(fq, M, N, K):
    check(fq, M, N, K, "silu", True, True, seed=M + N + K)


@pytest.mark.parametrize("act", [None, "none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("use_bias,use_res", [(False, False), (True, False), (False, True), (True, True)])
def test_parts(fq, act, M, use_bias, use_res):
    check(fq, M, 328, 272, act, use_bias, use_res, seed=7 * M)


@pytest.mark.parametrize("M", [2, 130])
def test_e5m2(fq, M):
    check(fq, M, 264, 528, "gelu", True, True, seed=M, x_fmt="e5m2")


@pytest.mark.parametrize("M", [1, 64, 128, 700])
def test_residual_in_place(fq, M):
    check(fq, M, 520, 272, "gelu", True, True, seed=M, in_place=True)


@pytest.mark.parametrize("family,bn,ksplit", [(1, 0, 0), (2, 128, 0), (2, 192, 0), (2, 256, 0), (2, 512, 0), (3, 0, 1),
                                              (3, 0, 2), (3, 0, 4), (3, 0, 8)])
def test_kernel_choices(fq, family, bn, ksplit):
    fq.set_gemm_tuning(family, bn, ksplit)
    try:
        check(fq, 100 if family == 3 else 300, 520, 1040, "gelu_tanh", True, True, seed=bn + ksplit)
    finally:
        fq.set_gemm_tuning(0, 0, 0)


@pytest.mark.parametrize("M", [1, 32, 128, 500])
@pytest.mark.parametrize("x_fmt", ["e4m3", "e5m2"])
def test_without_parts_equals_linear_bitwise(fq, M, x_fmt):
    Xq, s_x, Wq, s_w, _, _ = inputs(fq, M, 520, 528, M, x_fmt)
    a = fq.linear(Xq, s_x, Wq, s_w, x_fmt=x_fmt)
    b = fq.linear_epilogue(Xq, s_x, Wq, s_w, x_fmt=x_fmt)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activation_over_its_range(fq, act):
    """z runs over [-20, 20) through the bias (all products are zero), tails and signs included."""
    N = 8192
    z = ((torch.arange(N, dtype=torch.float32) - N // 2) / (N // 40)).half()
    Xq = torch.zeros((1, 16), dtype=torch.uint8, device="cuda")
    Wq = torch.zeros((N, 16), dtype=torch.uint8, device="cuda")
    one = torch.ones(1, device="cuda")
    y = fq.linear_epilogue(Xq, one, Wq, torch.ones(N, device="cuda"), bias=z.cuda(), activation=act)
    ref, terms = linear_epilogue_ref(to_np(Xq), np.ones(1), to_np(Wq), np.ones(N), z.numpy(), act)
    assert_within(to_np(y), ref, linear_epilogue_bound(16, ref, terms), act)


def test_zero_rows(fq):
    Xq, s_x, Wq, s_w, bias, _ = inputs(fq, 4, 64, 128, 1)
    Y = fq.linear_epilogue(Xq[:0], s_x[:0], Wq, s_w, bias=bias, activation="gelu")
    assert Y.shape == (0, 64)


def test_captured_and_replayed_on_another_stream(fq):
    M, N, K = 40, 264, 272
    Xq, s_x, Wq, s_w, bias, residual = inputs(fq, M, N, K, 5)
    expect = fq.linear_epilogue(Xq, s_x, Wq, s_w, bias=bias, activation="silu", residual=residual)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = torch.zeros((M, N), dtype=torch.float16, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            fq.linear_epilogue(Xq, s_x, Wq, s_w, bias=bias, activation="silu", residual=residual, out=out)
        for _ in range(3):
            out.zero_()
            graph.replay()
            s.synchronize()
            assert torch.equal(out, expect)


def test_ffn_pair_full(fq):
    """The dense FFN pair at full size: bias + GELU up, bias + residual down."""
    rows = slice(0, 8192, 97)   # the float64 product of a spread of rows; every row was written (no NaN)
    for (M, N, K, act, use_res) in ((8192, 8192, 2048, "gelu", False), (8192, 2048, 8192, None, True)):
        Xq, s_x, Wq, s_w, bias, residual = inputs(fq, M, N, K, K, w_std=0.02)
        g = Guards()
        Y = g((M, N), torch.float16, float("nan"), "Y")
        fq.linear_epilogue(Xq, s_x, Wq, s_w, bias=bias, activation=act, residual=residual if use_res else None, out=Y)
        g.check(f"{M}x{N}x{K}")
        assert bool(torch.isfinite(Y).all())
        rr = to_np(residual)[rows] if use_res else None
        y, terms = linear_epilogue_ref(to_np(Xq)[rows], to_np(s_x)[rows], to_np(Wq), to_np(s_w), to_np(bias), act, rr)
        terms = terms + np.abs(to_np(bias).astype(np.float64))[None, :]
        assert_within(to_np(Y)[rows], y, linear_epilogue_bound(K, y, terms, rr), f"{M}x{N}x{K}")
    assert_no_device_error()


@pytest.mark.parametrize("M", [2, 100, 200])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_activations_of_large_values(fq, act, M):
    """Products +-2^j up to 2^124: the activation is z (rounded to fp16) or, exactly, zero.
    From |z| = 128 on that is every formula's fp16 value: z's own tail, z e^z, is below 2^-170."""
    K, powers = 16, np.arange(3, 121)
    N = 240
    one = torch.tensor([1.0]).to(torch.float8_e4m3fn).view(torch.uint8).item()
    Xq = torch.full((M, K), one, dtype=torch.uint8, device="cuda")
    Wq = torch.full((N, K), one, dtype=torch.uint8, device="cuda")
    Wq[1::2] |= 0x80
    j = np.resize(np.repeat(powers, 2), N)
    s_w = torch.from_numpy(np.exp2(j).astype(np.float32)).cuda()
    out = fq.linear_epilogue(Xq, torch.ones(M, device="cuda"), Wq, s_w, activation=act)
    got = to_np(out).astype(np.float64)
    with np.errstate(over="ignore"):
        want = np.where(np.arange(N) % 2 == 0, (K * np.exp2(j)).astype(np.float16), 0).astype(np.float64)
    assert np.array_equal(got, np.broadcast_to(want, got.shape))
    assert_no_device_error()
