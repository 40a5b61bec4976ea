"""Many rows: B H n of 2^28 and more."""
import pytest
import torch

from causal_prefix_scan_hla2_amd import hla2 as H

pytestmark = pytest.mark.gpu


def test_window_of_many_rows():
    """A sequence does not depend on the batch around it: the last of a large batch, which is zero but for it, has the
    bits of a call on it alone."""
    dev, B, Hh, n, d, window = torch.device("cuda:0"), 257, 16, 65536, 16, 200
    assert B * Hh * n > 2 ** 28
    gen = torch.Generator(dev).manual_seed(7)
    ones = [torch.randn(1, Hh, n, d, device=dev, generator=gen).bfloat16() for _ in range(4)]
    results = []
    for batch in (1, B):
        q, k, v, dout = (torch.zeros(batch, Hh, n, d, dtype=torch.bfloat16, device=dev) for _ in range(4))
        for t, one in zip((q, k, v, dout), ones):
            t[-1] = one[0]
        out, dq, dk, dv = (torch.zeros_like(q) for _ in range(4))
        lse = torch.empty(batch, Hh, n, device=dev)
        H.hla2_window_forward(q, k, v, out, window, lse=lse)
        H.hla2_window_backward(q, k, v, out, lse, dout, dq, dk, dv, window)
        ck, cv = (torch.zeros(batch, Hh, window, d, dtype=q.dtype, device=dev) for _ in range(2))
        H.hla2_window_cache(k, v, ck, cv, window)
        results.append([t[-1].clone() for t in (out, lse, dq, dk, dv, ck, cv)])
        del q, k, v, dout, out, dq, dk, dv, lse, ck, cv
    for a, b in zip(*results):
        assert torch.equal(a, b) and a.abs().max() > 0
