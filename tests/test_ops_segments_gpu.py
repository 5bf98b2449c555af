"""The gated recurrence where few columns of many steps are cut into segments: two launches, the second
of which may start while the first ends, with the segments' maps in the workspace -- on another
stream, in captured graphs, and several at once."""

import pytest
import torch

from selective_state_space_13_b200 import ops, scan

pytestmark = pytest.mark.gpu

B_, L, D = 1, 9000, 72


def calls(io, form):
    """(forward, backward) calls with states carried in and out, all seeded."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dout = rand(B_, L, D).to(io), rand(B_, L, D).to(io)
    gate = rand(B_, L, D).to(io) if form == "sigmoid" else (-rand(B_, L, D).exp() / 50).to(io)
    bias = rand(D) + 3 if form == "sigmoid" else None
    h0, dlast = rand(B_, D), rand(B_, D)
    kept = ops.gated_recurrence_fwd(x, gate, gate_bias=bias, initial_state=h0, form=form)

    def forward():
        return list(ops.gated_recurrence_fwd(x, gate, gate_bias=bias, initial_state=h0, form=form,
                                             return_last_state=True))

    def backward():
        return [v for v in ops.gated_recurrence_bwd(dout, x, gate, kept, gate_bias=bias,
                                                    initial_state=h0, dlast_state=dlast,
                                                    form=form) if v is not None]

    return forward, backward


CASES = [(io, form, k) for io in (torch.float32, torch.bfloat16) for form in ("sigmoid", "exp")
         for k in (0, 1)]


def test_these_sizes_are_split(cuda_device):
    for io in (scan.SS_F32, scan.SS_BF16):
        for form in (0, 1):
            opts = ops.SsRecurrenceOpts(form, 0, 0, 0)
            size = lambda length, k: ops.gated_recurrence_workspace_size(  # noqa: E731
                scan.make_shape(B_, length, D, 1, io), opts, k)
            # maps of two segments of two columns at least: 32 float4 each
            assert size(L, False) >= 2 * 2 * 512
            assert size(L, True) >= 2 * 2 * 512 + size(64, True) * (form == 0)


@pytest.mark.parametrize("io,form,k", CASES)
def test_segments_on_another_stream(cuda_device, io, form, k):
    call = calls(io, form)[k]
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [call() for _ in range(20)]
    torch.cuda.synchronize()
    for vs in got:
        for a, b in zip(vs, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("io,form,k", CASES)
def test_segments_captured(cuda_device, io, form, k):
    call = calls(io, form)[k]
    want = call()
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call() + call())
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(3):
        for v in outs[0] + outs[1]:
            v.zero_()
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):  # at the same time
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for out in outs:
            for a, b in zip(out, want + want):
                assert torch.equal(a, b)


def test_segments_at_once(cuda_device):
    todo = [calls(io, form)[k] for io, form, k in CASES]
    want = [c() for c in todo]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append([c() for c in todo])
    torch.cuda.synchronize()
    for one in got:
        for vs, ws in zip(one, want):
            for a, b in zip(vs, ws):
                assert torch.equal(a, b)
