"""The linear layer and the scored routing on another stream than the current one: memory that either stream still
uses is not handed to the other.  Each test keeps one stream busy (100 ms), so that what reuses a block too early
overwrites it, or reads what is written later."""
import pytest
import torch

import moe_expert_gemm_mxfp4_b200 as mx

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BUSY = 200_000_000     # cycles


def _linear():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(2048, 512, generator=g).to(torch.bfloat16).to(DEV)
    codes, scales = mx.mxfp4_quantize(torch.randn(1024, 512, generator=g).to(DEV))
    return x, lambda a, stream=None: {"y": mx.mxfp4_linear(a, codes, scales, act=mx.ACT_SILU, stream=stream)}


def _route():
    logits = torch.randn(40000, 64, generator=torch.Generator().manual_seed(4)).to(DEV)
    return logits, lambda a, stream=None: mx.moe_mxfp4_route_scored(a, 4, n_groups=8, top_groups=4, stream=stream)


@pytest.fixture(params=[_linear, _route], ids=["linear", "route"])
def op(request):
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    a, call = request.param()
    want = {k: v.clone() for k, v in call(a).items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call(a, side)                     # both pools hold blocks of the call's sizes from here on
    torch.cuda.synchronize()
    yield a, call, want, side
    torch.cuda.synchronize()
    assert mx.mxfp4_get_device_status() == 0


def _equal(got, want):
    torch.cuda.synchronize()
    return all(torch.equal(got[k], want[k]) for k in want)


def _sizes(want):
    """Bytes of blocks like those of the call: the outputs', alone and together."""
    each = [v.numel() * v.element_size() for v in want.values()]
    return each + [sum(each) + 4096]


def test_blocks_that_the_current_stream_still_writes(op):
    a, call, want, side = op
    for _ in range(3):
        blocks = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in _sizes(want)]
        torch.cuda._sleep(BUSY)
        for b in blocks:
            b.fill_(0x5A)             # after the pause
        del b, blocks
        got = call(a, side)
        assert _equal(got, want)


def test_operands_freed_while_the_other_stream_still_reads(op):
    a, call, want, side = op
    for _ in range(3):
        copy = a.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(BUSY)
        got = call(copy, side)
        del copy
        other = torch.full_like(a, -3.0)   # at once, on the current stream
        assert _equal(got, want)
        del other


def test_results_freed_while_the_current_stream_still_reads(op):
    a, call, want, side = op
    for _ in range(3):
        got = call(a, side)
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        seen = {k: v.clone() for k, v in got.items()}   # after the pause
        del got
        call(torch.flip(a, [0]), torch.cuda.current_stream())
        with torch.cuda.stream(side):
            blocks = [torch.full((n,), 0x5A, dtype=torch.uint8, device=DEV) for n in _sizes(want)]
        assert _equal(seen, want)
        del blocks


def test_captured_with_a_fork_to_the_other_stream(op):
    a, call, want, side = op
    buf = torch.empty_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = call(buf, side)
        here.wait_stream(side)
    buf.copy_(a)
    for _ in range(2):
        graph.replay()
    assert _equal(got, want)


def test_the_current_stream_itself(op):
    a, call, want, side = op
    assert _equal(call(a, torch.cuda.current_stream()), want)
    with torch.cuda.stream(side):
        got = call(a, side)
    assert _equal(got, want)


def test_routing_beside_itself_on_streams_of_two_priorities():
    """Large calls on a stream of high and one of low priority, beside linear layers that take whole SMs: no CTA of
    a call waits for one that another call keeps off the GPU."""
    logits, route = _route()
    x, linear = _linear()
    want, y = route(logits), linear(x)["y"]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1), torch.cuda.Stream(priority=0)]
    got = []
    for _ in range(12):
        got.append((route(logits, streams[0]), linear(x, streams[2])["y"], route(logits, streams[1])))
    torch.cuda.synchronize()
    assert mx.mxfp4_get_device_status() == 0
    for a, z, b in got:
        assert all(torch.equal(a[k], want[k]) and torch.equal(b[k], want[k]) for k in want)
        assert torch.equal(z, y)


def test_routing_beside_itself_in_one_graph():
    logits, route = _route()
    want = {k: v.clone() for k, v in route(logits).items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        a = route(logits, side)
        b = route(logits)
        here.wait_stream(side)
    for _ in range(4):
        graph.replay()
    assert _equal(a, want) and _equal(b, want)
