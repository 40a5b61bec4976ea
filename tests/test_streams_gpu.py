"""Calls of one shape back to back, the first on the current stream and the second on another one that does not wait for
it, with workspaces that the binding allocates: each has the bits of the call made alone."""
import pytest
import torch

from causal_prefix_scan_hla2_amd import hla2 as H

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=gen, device=DEV).to(dtype)


def scan(seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    B, Hh, n, d = 2, 8, 6000, 64
    x, g, dout = (randn(gen, B, Hh, n, d) for _ in range(3))
    out, dx, dg = (torch.zeros_like(x) for _ in range(3))
    marks = torch.zeros(B, Hh, (n + 255) // 256, d, device=DEV)

    def run(stream):
        H.hla2_gated_scan_forward(x, g, out, gate=H.HLA2_GATE_SIGMOID, marks=marks, stream=stream)
        H.hla2_gated_scan_backward(x, g, dout, dx, dg, gate=H.HLA2_GATE_SIGMOID, marks=marks, stream=stream)
    return run, (out, marks, dx, dg)


def window(seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    B, Hh, Hkv, n, d = 2, 8, 2, 1500, 64
    q, dout = (randn(gen, B, Hh, n, d) for _ in range(2))
    k, v = (randn(gen, B, Hkv, n, d) for _ in range(2))
    out, dq, dk, dv = (torch.zeros_like(t) for t in (q, q, k, v))
    lse = torch.zeros(B, Hh, n, device=DEV)

    def run(stream):
        H.hla2_window_forward(q, k, v, out, 200, 4, lse=lse, stream=stream)
        H.hla2_window_backward(q, k, v, out, lse, dout, dq, dk, dv, 200, 4, stream=stream)
    return run, (out, lse, dq, dk, dv)


def step(seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    N, Hkv, G, d, window = 2, 2, 4, 64, 16000
    ck, cv = (randn(gen, N, Hkv, window, d) for _ in range(2))
    q, k, v = randn(gen, N, Hkv * G, d), randn(gen, N, Hkv, d), randn(gen, N, Hkv, d)
    out, pos = torch.zeros_like(q), torch.full((N,), 40000, dtype=torch.int64, device=DEV)
    assert H.hla2_window_step_workspace_bytes(N, Hkv * G, Hkv, d, d, window, 0, H.HLA2_BF16) > 0
    return lambda stream: H.hla2_window_step(ck, cv, pos, q, k, v, out, window, stream=stream), (out, ck, cv)


def linear(seed):
    """The linear forms' entry points."""
    gen = torch.Generator(DEV).manual_seed(seed)
    q, k, v, dout = (randn(gen, 2, 8, 4096, 64) / 8 for _ in range(4))
    outs = [torch.zeros_like(q) for _ in range(7)]
    state = torch.zeros(2, 8, H.hla2_state_floats(64, 64), device=DEV)

    def run(stream):
        H.hla2_forward(q, k, v, outs[0], decay=0.98, stream=stream)
        H.hla2_forward_state(q, k, v, outs[1], state, decay=0.98, stream=stream)
        H.hla2_backward(q, k, v, dout, outs[2], outs[3], outs[4], decay=0.98, stream=stream)
        H.hla2_ahla_forward(q, k, v, outs[5], decay=0.98, stream=stream)
        H.hla2_ho3_forward(q, k, v, outs[6], decay=0.98, stream=stream)
    return run, (*outs, state)


def check(make, other):
    first, second, alone = make(1), make(2), make(2)
    alone[0](None)
    torch.cuda.synchronize()
    assert not torch.equal(second[1][0], alone[1][0])  # not written yet
    first[0](None)
    second[0](other)
    torch.cuda.synchronize()
    for got, want in zip(second[1], alone[1]):
        assert torch.equal(got, want)
    again = make(1)
    again[0](None)
    torch.cuda.synchronize()
    for got, want in zip(first[1], again[1]):
        assert torch.equal(got, want)


@pytest.mark.parametrize("make", [scan, window, step, linear])
@pytest.mark.parametrize("handle", ["stream", "int"])
def test_back_to_back_on_two_streams(make, handle):
    s = torch.cuda.Stream(DEV)
    check(make, s if handle == "stream" else s.cuda_stream)


def test_the_default_stream_by_its_handle():
    """0 is a stream like others: the calls' results are those without a stream."""
    for make in (scan, window, step, linear):
        (run, got), (alone, want) = make(3), make(3)
        alone(None)
        run(0)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("make", [scan, window, step, linear])
def test_captured_with_the_stream_named(make):
    """A capture in which the call names the capturing stream takes its workspace from the graph's own memory; replays
    between eager calls of the same shape on another stream keep their bits."""
    (run, got), (alone, want), (other, _) = make(5), make(5), make(6)
    alone(None)
    run(None)  # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        for t in got[:1] if make is step else got:  # the step's caches are inputs too
            t.zero_()
        graph.replay()
        other(None)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
