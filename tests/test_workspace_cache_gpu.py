"""The backward workspaces that the binding keeps (GPU): one per stream, so autograd on two streams
at once shares none, and one of its own for every captured call, so a graph keeps its results
whatever runs or grows beside it.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn
    from gated_norm_b200 import gnorm


def case(M, N, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, g, dy = (torch.randn(M, N, generator=gen, device="cuda").bfloat16() for _ in range(3))
    w = 1 + 0.1 * torch.randn(N, generator=gen, device="cuda")
    return x, g, w, dy


def backward(c, **kw):
    """The gradients of gated_rmsnorm, through autograd."""
    x, g, w, dy = c
    leaves = [t.detach().requires_grad_() for t in (x, g, w)]
    return torch.autograd.grad(gn.gated_rmsnorm(*leaves, **kw), leaves, dy)


def assert_same(got, want):
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_buffer_for_each_stream():
    s = torch.cuda.Stream()
    here = gn.workspace(1000, 128, True, "cuda")
    assert gn.workspace(500, 128, True, "cuda").data_ptr() == here.data_ptr()
    there = gn.workspace(1000, 128, True, "cuda", s)
    assert there.data_ptr() != here.data_ptr()
    with torch.cuda.stream(s):
        assert gn.workspace(1000, 128, True, "cuda").data_ptr() == there.data_ptr()
    torch.cuda.synchronize()
    assert not here[:256].any() and not there[:256].any()


@pytest.mark.parametrize("det", [True, False])
def test_two_streams_at_once(det):
    cases = [case(20000, 128, 1), case(20000, 128, 2)]
    want = [backward(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(backward(c, deterministic=det))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert_same(a[:2], b[:2])
            if det:
                assert torch.equal(a[2], b[2])
            else:  # sums of 20000 terms in another order: 2^-24 each, a random walk
                lim = 20000 ** 0.5 * 2.0 ** -24 * float(b[2].abs().max())
                assert float((a[2] - b[2]).abs().max()) <= lim
    assert gn.gnorm_device_error(reset=True) == 0


def captured(c, stream):
    graph = torch.cuda.CUDAGraph()
    x, g, w, dy = c
    with torch.cuda.graph(graph, stream=stream):
        y, rstd = gn.gnorm_fwd(x, g, w)
        out = gn.gnorm_bwd(dy, x, g, w, rstd, dw_fp32=True, deterministic=False)
    return graph, out


def test_captured_before_anything_is_cached():
    """The graph's buffer stays out of the cache; eager calls are right before its first replay."""
    c = case(20000, 128, 3)
    want = backward(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kept = dict(gnorm._ws_cache)
    graph, out = captured(c, s)
    assert gnorm._ws_cache.keys() == kept.keys()
    with torch.cuda.stream(s):
        got = backward(c)
    torch.cuda.synchronize()
    assert_same(got, want)
    graph.replay()
    torch.cuda.synchronize()
    assert_same(out[:2], want[:2])


def test_two_graphs_at_once_and_a_growing_cache():
    cases = [case(20000, 128, 4), case(20000, 128, 5)]
    want = [backward(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    made = [captured(c, s) for c, s in zip(cases, streams)]
    torch.cuda.synchronize()
    lim = [20000 ** 0.5 * 2.0 ** -24 * float(w[2].abs().max()) for w in want]
    for i in range(4):
        if i == 2:  # every cached buffer is replaced by a larger one, its memory used again
            for s in [torch.cuda.current_stream()] + streams:
                with torch.cuda.stream(s):
                    backward(case(4000, 4096, 6))
            fill = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(64)]
        for _, out in made:
            for t in out:
                t.fill_(7)
        torch.cuda.synchronize()
        for (graph, _), s in zip(made, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out), w, most in zip(made, want, lim):
            assert_same(out[:2], w[:2])
            assert float((out[2] - w[2]).abs().max()) <= most
    assert all(bool((t == 3.0).all()) for t in fill)
    assert gn.gnorm_device_error(reset=True) == 0


def test_threads_on_one_stream():
    """The kernels of two threads' calls may mingle on the stream; their workspaces differ."""
    import threading

    cases = [case(3000, 256, 7), case(5000, 256, 8)]
    want = [backward(c) for c in cases]
    torch.cuda.synchronize()
    got, places, errors = [None, None], [None, None], []
    start = threading.Barrier(2)

    def work(i):
        try:
            x, g, w, dy = cases[i]
            _, rstd = gn.gnorm_fwd(x, g, w)
            places[i] = gn.workspace(5000, 256, True, "cuda").data_ptr()
            start.wait()
            got[i] = [gn.gnorm_bwd(dy, x, g, w, rstd, dw_fp32=True) for _ in range(200)]
        except Exception as e:  # shown below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and places[0] != places[1]
    for i in range(2):
        for out in got[i]:
            assert_same(out, want[i])
    assert gn.gnorm_device_error(reset=True) == 0


def test_a_stream_that_is_not_torchs():
    """Anything with a cuda_stream names the stream, as in the other calls."""
    from types import SimpleNamespace

    x, g, w, dy = case(300, 128, 9)
    want = backward((x, g, w, dy))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = SimpleNamespace(cuda_stream=s.cuda_stream)
    _, rstd = gn.gnorm_fwd(x, g, w, stream=other)
    got = gn.gnorm_bwd(dy, x, g, w, rstd, dw_fp32=True, stream=other)
    s.synchronize()
    assert_same(got, want)
    assert gn.workspace(300, 128, True, "cuda", other).data_ptr() == gn.workspace(300, 128, True, "cuda", s).data_ptr()
