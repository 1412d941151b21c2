"""The quantisers on another stream than the current one: what they return belongs to the current stream, so the two
are ordered both ways."""
from __future__ import annotations

import pytest
import torch

import mixture_experts_layer_37_b200 as M

pytestmark = pytest.mark.gpu

E, K, N = 4, 512, 1024
CFG = M.MoEConfig(T=4, d=K, ffn=N, E=E, k=1, weights="int8")
CALLS = {
    "int4": lambda w, s: M.moe_quantize_int4(w, 64, stream=s),
    "int8": lambda w, s: M.moe_quantize_int8(CFG, w, stream=s),
    "pack": lambda w, s: (M.moe_pack_int4((w.float() * 40).round().clamp(-8, 7).to(torch.int8), stream=s),),
}


def weights():
    return (torch.randn((E, K, N), generator=torch.Generator().manual_seed(1)) * 0.05).bfloat16().cuda()


@pytest.mark.parametrize("handle", ["stream", "address", "default"])
@pytest.mark.parametrize("call", CALLS)
def test_outputs_are_ordered_with_the_current_stream(call, handle):
    f, w = CALLS[call], weights()
    want = [t.clone() for t in f(w, None)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    current = torch.cuda.Stream() if handle == "default" else torch.cuda.current_stream()
    stream = {"stream": side, "address": side.cuda_stream, "default": 0}[handle]
    with torch.cuda.stream(current):
        late = torch.zeros_like(w)
        old = [torch.empty_like(t) for t in want]
        torch.cuda._sleep(20_000_000)               # about 10 ms
        for t in old:
            t.view(torch.uint8).fill_(255)          # still to come when the memory below is handed out again
        late.copy_(w)                               # and so are the weights
        del old, t
        got = [t.clone() for t in f(late, stream)]  # read on the current stream, without further ado
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_quantised_inside_a_captured_graph():
    """Captured with a stream of its own beside the capturing one: part of the graph, replayed with new weights."""
    w = weights()
    want = [t.clone() for t in M.moe_quantize_int4(w, 32)]
    fixed, side = torch.zeros_like(w), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = M.moe_quantize_int4(fixed, 32, stream=side)
    fixed.copy_(w)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)
