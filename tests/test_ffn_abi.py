"""linear_epilogue, moe_route and moe_layer: arguments refused on the host
(no GPU needed; a refused call enqueues nothing), and calls with nothing to do."""
import pytest
import torch

from fp8_quantized_generative_b200 import _lib

A = 0x10000      # aligned
BAD = 0x10008    # 8-byte aligned, not 16
FAR = 0x900000   # another buffer
INVALID = _lib.FP8Q_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from fp8_quantized_generative_b200 import build
        build.build()
    return _lib.lib()


def epilogue(Xq=A, fmt=0, s_x=A, Wq=A, s_w=A, M=4, N=16, K=32, bias=A, act=2, residual=FAR, Y=A):
    return _lib.fp8q_linear_epilogue(Xq, fmt, s_x, Wq, s_w, M, N, K, bias, act, residual, Y, 0)


@pytest.mark.parametrize("bad", [
    dict(act=5), dict(act=-1), dict(fmt=2), dict(M=-1), dict(N=0), dict(N=12), dict(K=0), dict(K=24), dict(Xq=0),
    dict(s_x=BAD), dict(Wq=0), dict(s_w=0), dict(Y=0), dict(Y=BAD), dict(bias=BAD), dict(residual=BAD),
    dict(residual=A + 16, Y=A), dict(residual=A, Y=A + 64),
])
def test_epilogue_refuses(bad):
    assert epilogue(**bad) == INVALID
    assert _lib.last_error_message() != ""


def test_epilogue_without_rows():
    assert epilogue(Xq=0, s_x=0, M=0, Y=0, residual=0) == _lib.FP8Q_OK


def route(logits=A, T=4, E=16, topk=2, experts=A, weights=A, offsets=A, row_token=A, row_weight=A, token_rows=A, ws=A):
    return _lib.fp8q_moe_route(logits, T, E, topk, 1, experts, weights, offsets, row_token, row_weight, token_rows, ws, 0)


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=1025), dict(topk=0), dict(topk=9), dict(E=4, topk=5), dict(T=-1), dict(T=(1 << 22) + 1),
    dict(logits=0), dict(logits=A + 1), dict(experts=0), dict(weights=A + 2), dict(offsets=0), dict(offsets=A + 2),
    dict(row_token=0), dict(row_weight=0), dict(token_rows=A + 2), dict(T=65, ws=0), dict(T=65, ws=A + 2),
])
def test_route_refuses(bad):
    assert route(**bad) == INVALID
    assert _lib.last_error_message() != ""


def test_route_workspace():
    w = _lib.fp8q_moe_route_workspace_words
    assert [w(0, 64), w(64, 64), w(65, 64), w(4096, 64), w(8192, 64), w(1 << 22, 8)] == [0, 0, 3 * 64, 8192, 8192, 1024]


def layer(X=A, T=4, experts=A, weights=A, topk=2, E=8, Wu=A, su=A, Wd=A, sd=A, K=32, F=48, N=40, act=4, gated=0,
          residual=FAR, out=A, ws=A):
    return _lib.fp8q_moe_layer(X, T, experts, weights, topk, E, Wu, su, Wd, sd, K, F, N, act, gated, residual, out, ws, 0)


@pytest.mark.parametrize("bad", [
    dict(act=5), dict(E=0), dict(E=1025), dict(topk=0), dict(topk=9), dict(T=-1), dict(T=129), dict(K=0), dict(K=24),
    dict(K=8208), dict(F=0), dict(F=40), dict(F=8208), dict(N=0), dict(N=12), dict(N=(1 << 20) + 8), dict(X=0),
    dict(X=BAD), dict(Wu=0), dict(su=BAD), dict(Wd=BAD), dict(sd=0), dict(out=0), dict(ws=0), dict(ws=BAD),
    dict(experts=0), dict(experts=A + 2), dict(weights=0), dict(weights=A + 2), dict(residual=BAD),
    dict(residual=A + 16, out=A),
])
def test_layer_refuses(bad):
    assert layer(**bad) == INVALID
    assert _lib.last_error_message() != ""


def test_layer_without_tokens():
    assert layer(X=0, T=0, experts=0, weights=0, out=0, ws=0) == _lib.FP8Q_OK


def test_layer_workspace_holds_hidden_rows_and_sums():
    b = _lib.fp8q_moe_layer_workspace_bytes
    assert b(0, 2, 64, 64) == 0
    assert b(3, 2, 16, 8) >= 6 * 16 * 2 + 6 * 8 * 4
    assert b(128, 8, 8192, 1 << 20) >= 1024 * (8192 * 2 + (1 << 22))


def test_python_wrappers_refuse_cpu_tensors_and_unknown_names():
    import fp8_quantized_generative_b200 as fq
    u8, f32 = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros(4)
    with pytest.raises(ValueError, match="activation"):
        fq.linear_epilogue(u8, f32, u8, f32, activation="tanh")
    with pytest.raises(ValueError, match="activation"):
        fq.linear_epilogue(u8, f32, u8, f32, activation=["relu"])
    with pytest.raises(ValueError, match="format"):
        fq.linear_epilogue(u8, f32, u8, f32, x_fmt="e3m4")
    with pytest.raises(ValueError, match="CUDA"):
        fq.linear_epilogue(u8, f32, u8, f32)
    with pytest.raises(ValueError, match="CUDA"):
        fq.moe_route(torch.zeros((4, 8), dtype=torch.float16), 2)
    with pytest.raises(ValueError, match="CUDA"):
        fq.moe_layer(torch.zeros((4, 32), dtype=torch.float16), None, None, None, None, None, None)
    with pytest.raises(ValueError, match="activation"):
        fq.moe_layer(None, None, None, None, None, None, None, activation="swish")
    with pytest.raises(TypeError, match="Xq"):
        fq.linear_epilogue(None, f32, u8, f32)
    with pytest.raises(TypeError, match="X must"):
        fq.moe_layer(None, None, None, None, None, None, None)
