"""linear_epilogue, moe_route and moe_layer refuse wrong tensors with an error
that names the argument, and take what fits (one GPU: another device is a CPU
tensor here)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


def t(dtype, *shape):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


u8, f16, f32, i32 = torch.uint8, torch.float16, torch.float32, torch.int32


def epilogue_args():
    return dict(Xq=t(u8, 4, 32), s_x=t(f32, 4), Wq=t(u8, 16, 32), s_w=t(f32, 16), bias=t(f16, 16),
                residual=t(f16, 4, 16), out=t(f16, 4, 16))


def layer_args():
    return dict(X=t(f16, 4, 32), experts=t(i32, 4, 2), weights=t(f32, 4, 2), Wq_up=t(u8, 3, 48, 32), s_up=t(f32, 3, 48),
                Wq_down=t(u8, 3, 40, 48), s_down=t(f32, 3, 40), residual=t(f16, 4, 40), out=t(f16, 4, 40),
                workspace=t(u8, 1 << 16))


def wrong(x):
    """Variants of a tensor that are to be refused: type, device, rank, strides, shape."""
    other = f32 if x.dtype != f32 else f16
    yield "dtype", x.to(other)
    yield "device", x.cpu()
    yield "none", "not a tensor"
    if x.numel() < 1 << 16:
        yield "rank", x[None]
        yield "shape", torch.cat([x, x])
    yield "strides", torch.stack([x, x], -1)[..., 0]


@pytest.mark.parametrize("op", ["linear_epilogue", "moe_layer"])
def test_wrong_tensors(fq, op):
    fn, make = getattr(fq, op), epilogue_args if op == "linear_epilogue" else layer_args
    fn(**make())
    for name in make():
        for kind, bad in wrong(make()[name]):
            args = make()
            args[name] = bad
            with pytest.raises((ValueError, TypeError, AttributeError)):
                fn(**args)
                pytest.fail(f"{op}: {name} with a wrong {kind} went through")
    assert fq.device_error() == 0


def test_workspace_that_is_no_tensor(fq):
    with pytest.raises(TypeError, match="workspace"):
        fq.moe_layer(**{**layer_args(), "workspace": "not a tensor"})


def test_small_workspace_and_missing_arguments(fq):
    args = layer_args()
    args["workspace"] = t(u8, 16)
    with pytest.raises(ValueError, match="workspace"):
        fq.moe_layer(**args)
    args = layer_args()
    with pytest.raises(ValueError):
        fq.moe_layer(**{**args, "gated": True})
    with pytest.raises(ValueError, match="bias"):
        fq.linear_epilogue(**{**epilogue_args(), "bias": t(f16, 8)})
    with pytest.raises(ValueError, match="residual"):
        fq.linear_epilogue(**{**epilogue_args(), "residual": t(f16, 4, 8)})


def test_route_refusals(fq):
    with pytest.raises(TypeError, match="logits"):
        fq.moe_route(t(f32, 4, 8), 2)
    with pytest.raises(ValueError, match="contiguous"):
        fq.moe_route(t(f16, 8, 4).t(), 2)
    for k in (0, 9, 5):
        with pytest.raises(ValueError, match="topk"):
            fq.moe_route(t(f16, 4, 4 if k == 5 else 16), k)
    with pytest.raises(fq.Fp8qError):
        fq.moe_route(t(f16, 2, 1032), 2)


def test_too_many_tokens_names_the_grouped_path(fq):
    X = t(f16, 129, 32)
    a = layer_args()
    with pytest.raises(fq.Fp8qError, match="grouped"):
        fq.moe_layer(X, t(i32, 129, 2), t(f32, 129, 2), a["Wq_up"], a["s_up"], a["Wq_down"], a["s_down"])
