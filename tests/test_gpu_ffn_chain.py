"""Router and MoE layer back to back without waiting, many steps through the same
buffers, eagerly and in a graph: every step reads what the launch just before it wrote."""
import pytest
import torch

from fp8_quantized_generative_b200 import workloads as wl

from parity import assert_no_device_error

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    import fp8_quantized_generative_b200 as m
    assert torch.cuda.is_available()
    return m


@pytest.mark.parametrize("T,E,topk,gated", [(1, 64, 2, False), (7, 16, 4, True), (16, 40, 2, False), (60, 24, 3, True),
                                            (128, 64, 2, False)])
def test_steps_through_the_same_buffers(fq, T, E, topk, gated):
    K, F, steps = 528, 272, 40
    Wu, su = fq.quantize_weight_per_channel(wl.random_f16((E, 2 * F if gated else F, K), seed=1, std=0.08).cuda())
    Wd, sd = fq.quantize_weight_per_channel(wl.random_f16((E, K, F), seed=2, std=0.08).cuda())
    gate = wl.random_f16((E, K), seed=3, std=0.2).cuda()
    x0 = wl.random_f16((T, K), seed=4).cuda()
    logits = [wl.random_f16((T, E), seed=10 + i).cuda() for i in range(steps)]
    ws = fq.moe_layer_workspace(T, topk, F, K, "cuda")

    def step(x, bias, workspace, wait):
        x = x * (2.0 / x.abs().amax())   # (gated, the rows' squares grow past fp16 within eight steps otherwise)
        l = x @ gate.t() + bias
        if wait:
            torch.cuda.synchronize()
        r = fq.moe_route(l, topk)   # (freed after the step: the next one's lies in the same place)
        if wait:
            torch.cuda.synchronize()
        return fq.moe_layer(x, r.experts, r.weights, Wu, su, Wd, sd, gated=gated, residual=x0, workspace=workspace)

    def run(workspace, wait=False):
        x, seen = x0, []
        for bias in logits:
            x = step(x, bias, workspace, wait)
            seen.append(x)
        return seen

    expect = run(None, wait=True)   # a fresh workspace a call, the GPU idle before each
    assert all(bool(torch.isfinite(x).all()) for x in expect)
    for _ in range(3):
        for a, b in zip(run(ws), expect):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = run(ws)
        for _ in range(3):
            graph.replay()
        s.synchronize()
        for a, b in zip(got, expect):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert_no_device_error()
