"""The layer operators on torch's current stream, without naming it."""
from __future__ import annotations

import pytest
import torch

import mixed_precision_partial_amd as ar
import test_layer_gpu as base
from gpu_util import log_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    c = ar.ar_init(0)
    yield c
    torch.cuda.synchronize()
    ar.ar_free(c)


def test_inputs_and_outputs_on_a_side_stream(ctx):
    """The input is made on a side stream after milliseconds of other work there, and the output is read there."""
    log_case("side stream")
    g = base.gen(3)
    x = torch.randn(64, 4096, generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn(512, 4096, generator=g) * 50).to(torch.float8_e4m3fn).cuda()
    ws = torch.rand(4, 32, generator=g).cuda()
    codes, scales = torch.empty(64, 4096, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(64, 32, device="cuda")
    out = torch.empty(64, 512, dtype=torch.bfloat16, device="cuda")

    def enqueue(y):
        ar.ar_fp8_quantize(ctx, codes, scales, y)
        ar.ar_fp8_matmul(ctx, out, codes, scales, w, ws)
        return codes.view(torch.uint8).clone(), scales.clone(), out.clone()
    want = enqueue(x)
    torch.cuda.synchronize()
    late, busy = torch.zeros_like(x), torch.randn(8192, 8192, device="cuda")
    for y in (codes.view(torch.uint8), scales, out):
        y.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(8):
            busy = busy @ busy * 1e-4
        late.copy_(x)
        got = enqueue(late)
    torch.cuda.synchronize()
    for i, (y, z) in enumerate(zip(got, want)):
        assert torch.equal(y, z), f"output {i}"


def test_graph_of_the_current_stream(ctx):
    """A captured graph takes all four operators without a stream named, and runs none of them while it is captured."""
    log_case("graph without a stream")
    enqueue, outs = base.layer_calls(ctx)
    enqueue(None)
    torch.cuda.synchronize()
    want = [x.clone() for x in outs]
    for x in outs[3:]:
        x.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        enqueue(None)
    torch.cuda.synchronize()
    assert not any(bool(x.any()) for x in outs[3:])
    for _ in range(4):
        for x in outs[3:]:
            x.zero_()
        torch.randn(1 << 16, device="cuda").sum().item()    # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(outs, want)):
            assert torch.equal(x, y), f"output {i}"
        enqueue(None)
        torch.cuda.synchronize()
