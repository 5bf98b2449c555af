"""The forward scan's scratch belongs to one call: two calls in flight -- of two host threads, on two
streams, in a captured graph -- never work on the same bytes.  On the host with the C call replaced;
on a GPU with split, two-direction scans (carries and per-direction outputs in the scratch)."""

import contextlib
import threading
import types

import pytest
import torch

from selective_state_space_13_b200 import scan

F32, BF16 = torch.float32, torch.bfloat16


class FakeCuda:
    """Just enough of torch.cuda for the binding's host side: a current stream, capture states, and
    the stream that every scratch allocation was made on."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.made, self.keep = 7, set(), {}, []
        empty = torch.empty

        def make(n, dtype=None, device=None, **kw):
            t = empty(n, dtype=dtype)
            if dtype is torch.uint8:
                self.made[t.data_ptr()] = self.current
                self.keep.append(t)  # an address is never handed out twice
            return t

        @contextlib.contextmanager
        def on(stream):
            before, self.current = self.current, stream.cuda_stream
            yield
            self.current = before

        stream_of = lambda handle: types.SimpleNamespace(cuda_stream=handle)  # noqa: E731
        monkeypatch.setattr(torch, "empty", make)
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream_of(self.current))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: stream_of(0))
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a, **k: stream_of(h))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                            lambda: self.current in self.capturing)
        monkeypatch.setattr(scan, "_check", lambda *a: None)


def split_call(**kw):
    u = torch.zeros(2, 64, 8)
    B = torch.zeros(1, 2, 64, 4)
    return scan.selective_scan_fwd(u, u, torch.zeros(8, 4), B, B, segments=4, **kw)


def test_two_host_threads_on_one_stream(monkeypatch):
    # the C call lets another thread run; what that thread enqueues lies between this call's launches
    FakeCuda(monkeypatch)
    seen = []

    def raw(*a):
        seen.append(a[13])
        if len(seen) == 1:
            split_call()
        return scan.SS_OK

    monkeypatch.setattr(scan, "selective_scan_fwd_raw", raw)
    split_call()
    assert len(seen) == 2 and 0 not in seen and seen[0] != seen[1]


@pytest.mark.parametrize("as_handle", [False, True])
def test_explicit_streams(monkeypatch, as_handle):
    # scratch of a call on stream s is the allocator's for s, whatever stream is current
    fake, seen = FakeCuda(monkeypatch), []
    monkeypatch.setattr(scan, "selective_scan_fwd_raw",
                        lambda *a: seen.append((a[13], a[15])) or scan.SS_OK)
    for handle in (21, 22, 0, 21):
        split_call(stream=handle if as_handle else types.SimpleNamespace(cuda_stream=handle))
    split_call()
    assert [s for _, s in seen] == [21, 22, 0, 21, 7]
    assert [fake.made[w] for w, _ in seen] == [21, 22, 0, 21, 7]
    assert fake.current == 7


def test_host_buffer_call_on_an_explicit_stream(monkeypatch):
    fake, seen = FakeCuda(monkeypatch), []
    monkeypatch.setattr(scan, "selective_scan_fwd_host_raw",
                        lambda *a: seen.append((a[13], a[16])) or scan.SS_OK)
    u, B = torch.zeros(2, 64, 8), torch.zeros(1, 2, 64, 4)
    out = torch.zeros(2, 64, 8)
    for stream in (21, 22, None):
        scan.selective_scan_fwd_host(u, u[None], torch.zeros(8, 4), B, B, out=out, stream=stream,
                                     device=torch.device("cuda", 0))
    assert [s for _, s in seen] == [21, 22, 7]
    assert [fake.made[w] for w, _ in seen] == [21, 22, 7]


# ----------------------------------------------------------------------------- on a GPU

def problem(seed, io=BF16, b=2, L=700, D=40, N=16, dirs=(0, 1)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    K = len(dirs)
    return dict(u=rand(b, L, D).to(io), delta=rand(K, b, L, D).to(io),
                A=-torch.rand(D, N, generator=g, device="cuda") - 0.1, B=rand(K, b, L, N).to(io),
                C=rand(K, b, L, N).to(io), dirs=dirs, segments=5)


@pytest.mark.gpu
def test_threads_on_one_stream_gpu(cuda_device):
    problems = [problem(s, L=700 + 100 * s) for s in range(4)]
    want = [scan.selective_scan_fwd(**p).clone() for p in problems]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [[] for _ in problems]

    def work(i):
        with torch.cuda.stream(side):
            for _ in range(40):
                got[i].append(scan.selective_scan_fwd(**problems[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert len(outs) == 40
        for o in outs:
            assert torch.equal(o, w)


@pytest.mark.gpu
def test_explicit_streams_gpu(cuda_device):
    problems = [problem(10 + s, L=900 + 300 * s) for s in range(3)]
    want = [scan.selective_scan_fwd(**p).clone() for p in problems]
    outs = [[torch.empty_like(w) for _ in range(10)] for w in want]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    for r in range(10):
        for i, (p, s) in enumerate(zip(problems, streams)):
            stream = s if r % 2 else s.cuda_stream
            scan.selective_scan_fwd(**p, out=outs[i][r], stream=stream)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for v in o:
            assert torch.equal(v, w)


@pytest.mark.gpu
def test_explicit_capturing_stream_gpu(cuda_device):
    # two graphs hold calls on a stream that is given, not current; each keeps its own scratch
    p = problem(20)
    want = scan.selective_scan_fwd(**p).clone()
    graphs, outs = [], []
    for _ in range(2):
        out = torch.zeros_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            handle = torch.cuda.current_stream().cuda_stream
            scan.selective_scan_fwd(**p, out=out, stream=handle)
        graphs.append(graph)
        outs.append(out)
    for _ in range(3):
        scan.selective_scan_fwd(**problem(21, L=1500))
        for graph, out in zip(graphs, outs):
            out.zero_()
            graph.replay()
            assert torch.equal(out, want)


@pytest.mark.gpu
def test_host_buffer_calls_on_streams_and_threads_gpu(cuda_device):
    problems = [problem(30 + s, b=4, L=300 + 200 * s) for s in range(3)]
    want = [scan.selective_scan_fwd(**p).cpu() for p in problems]
    host = []
    for p in problems:
        q = {k: v for k, v in p.items() if k != "segments"}
        q.update({k: p[k].cpu().pin_memory() for k in ("u", "delta", "B", "C")})
        host.append(q)
    streams = [torch.cuda.Stream() for _ in problems]
    outs = [[torch.empty(w.shape, dtype=w.dtype, pin_memory=True) for _ in range(6)] for w in want]
    torch.cuda.synchronize()

    def work(i):
        for r in range(6):
            stream = streams[i] if r % 2 else streams[i].cuda_stream
            scan.selective_scan_fwd_host(**host[i], out=outs[i][r], stream=stream, chunks=2)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        for v in o:
            # pieces of whole rows, other segments: a rounding of the output apart
            assert ((v.float() - w.float()).abs() <= 2.0 ** -7 * w.float().abs() + 1e-3).all()
            assert torch.equal(v, o[0])
