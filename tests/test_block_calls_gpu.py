"""How the block norm's calls may be made: on a stream of the caller's, with one workspace for
calls in a row, from two streams at once, in a thread of its own (GPU).  Every result is bitwise
that of the plain call."""
from __future__ import annotations

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import gated_norm_b200 as gn
    from test_block_gpu import make


def run(x, **kw):
    h, z, r1, r2 = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], g=x["g"], alpha=x["alpha"],
                                      stream=kw.get("stream"))
    return (h, z, r1, r2) + gn.gnorm_block_bwd(x["dh"], x["dz"], x["a"], x["r"], x["w1"], x["w2"], r1,
                                               r2, g=x["g"], alpha=x["alpha"], dw_fp32=True, **kw)


@pytest.mark.parametrize("M,N", [(500, 256), (70, 4096)])
def test_a_stream_and_a_workspace_of_the_caller(M, N):
    x = make(M, N, gate=True, res=torch.bfloat16)
    want = run(x)
    s = torch.cuda.Stream()
    ws = torch.empty(gn.gnorm_block_bwd_workspace_bytes(M, N), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    got = [run(x, stream=s, workspace_buf=ws) for _ in range(3)]
    s.synchronize()
    for g in got:
        for p, q in zip(want, g):
            assert torch.equal(p, q)


def test_two_streams_at_once():
    xs = [make(3000, 1024, gate=True, res=torch.bfloat16, seed=i) for i in range(2)]
    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(3):
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(run(x))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for p, q in zip(want[i % 2], g):
            assert torch.equal(p, q)


def test_in_a_thread_of_its_own():
    x = make(200, 512, gate=False, res=torch.float32)
    want = run(x)
    torch.cuda.synchronize()
    out = []
    t = threading.Thread(target=lambda: out.append(run(x)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    for p, q in zip(want, out[0]):
        assert p is None and q is None or torch.equal(p, q)


def test_given_outputs_come_back():
    x = make(64, 256, gate=True, res=torch.bfloat16)
    h, z = torch.empty_like(x["a"]), torch.empty_like(x["a"])
    out = gn.gnorm_block_fwd(x["a"], x["r"], x["w1"], x["w2"], g=x["g"], alpha=x["alpha"], h=h, z=z)
    assert out[0].data_ptr() == h.data_ptr() and out[1].data_ptr() == z.data_ptr()
    for p, q in zip(out, run(x)):
        assert torch.equal(p, q)
