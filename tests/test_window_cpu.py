"""Windowed attention without a GPU: its refusals (every check runs before the first HIP call), the
workspace queries, and the fp64 definition's gradients against differences."""
import ctypes
import os

import numpy as np
import pytest
import torch

from causal_prefix_scan_hla2_amd import build as B
from causal_prefix_scan_hla2_amd import hla2 as H
from oracle import mixers as M

P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 8)
INV, UNS, WSP = H.HLA2_ERR_INVALID, H.HLA2_ERR_UNSUPPORTED, H.HLA2_ERR_WORKSPACE


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(H.LIB_PATH):
        B.build()
    return H.lib()


SHAPE = [
    (dict(B=0), INV), (dict(H=0), INV), (dict(Hkv=0), INV), (dict(n=0), INV), (dict(d=0), INV), (dict(dv=-16), INV),
    (dict(window=0), INV), (dict(window=-4), INV), (dict(sinks=-1), INV), (dict(dtype=2), INV), (dict(H=3, Hkv=2), INV),
    (dict(H=2, Hkv=4), INV), (dict(d=24), UNS), (dict(d=144), UNS), (dict(dv=144), UNS), (dict(dtype=0, d=80), UNS),
    (dict(dtype=0, dv=128), UNS), (dict(sinks=65), UNS), (dict(B=1 << 13, H=1 << 12), UNS), (dict(n=1 << 24, d=128), UNS),
    (dict(B=1 << 12, H=1 << 6, n=1 << 12), UNS),
]
SCALE = [(dict(scale=3e38), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV)]


def ints(kw, *names):
    full = dict(dict(B=2, H=4, Hkv=2, n=100, d=64, dv=64, window=32, sinks=4), **kw)
    return [full[x] for x in names]


ALL = ("B", "H", "Hkv", "n", "d", "dv", "window", "sinks")


@pytest.mark.parametrize("kw,code", SHAPE + SCALE + [
    (dict(q=None), INV), (dict(out=None), INV), (dict(q=ODD), INV), (dict(out=ODD), INV),
    (dict(lse=ctypes.c_void_p(4098)), INV), (dict(lens=ctypes.c_void_p(4098)), INV)])
def test_forward_rejects(L, kw, code):
    assert L.hla2_window_forward(kw.get("q", P), P, P, kw.get("out", P), kw.get("lse"), kw.get("lens"), *ints(kw, *ALL),
                                 kw.get("scale", 1.0), kw.get("dtype", 1), None) == code


@pytest.mark.parametrize("kw,code", SHAPE + SCALE + [
    (dict(lse=None), INV), (dict(dout=None), INV), (dict(dq=None), INV), (dict(dq=ODD), INV), (dict(dout=ODD), INV),
    (dict(ws=None), WSP), (dict(ws=ctypes.c_void_p(4096 + 64)), WSP), (dict(short=1), WSP),
    (dict(B=1 << 12, H=1 << 6, Hkv=1 << 6, n=40), UNS)])
def test_backward_rejects(L, kw, code):
    dt = kw.get("dtype", 1)
    need = H.hla2_window_backward_workspace_bytes(*ints(kw, *ALL), dt)
    assert (need == 0) == (code in (INV, UNS) and any(k in kw for k in ALL + ("dtype",)))
    assert L.hla2_window_backward(P, P, P, P, kw.get("lse", P), kw.get("dout", P), kw.get("dq", P), P, P, None,
                                  *ints(kw, *ALL), kw.get("scale", 1.0), dt, kw.get("ws", P),
                                  need - kw.get("short", 0), None) == code


@pytest.mark.parametrize("kw,code", [c for c in SHAPE if "H" not in c[0]] + [
    (dict(k=None), INV), (dict(cache_k=None), INV), (dict(cache_k=ODD), INV), (dict(window=1 << 24), UNS),
    (dict(window=1 << 22, d=128), UNS)])
def test_cache_rejects(L, kw, code):
    assert L.hla2_window_cache(kw.get("k", P), P, kw.get("cache_k", P), P, None,
                               *ints(kw, "B", "Hkv", "n", "d", "dv", "window", "sinks"), kw.get("dtype", 1), None) == code


@pytest.mark.parametrize("kw,code", [c for c in SHAPE if "n" not in c[0]] + SCALE + [
    (dict(pos=None), INV), (dict(pos=ctypes.c_void_p(4100)), INV), (dict(cache_k=ODD), INV), (dict(q=ODD), INV),
    (dict(H=34, Hkv=2), UNS), (dict(window=1 << 24), UNS), (dict(B=1 << 12, Hkv=64, H=64), UNS),
    (dict(window=4096, ws=None), WSP), (dict(window=4096, ws=ctypes.c_void_p(4096 + 64)), WSP),
    (dict(window=4096, short=1), WSP)])
def test_step_rejects(L, kw, code):
    dt, names = kw.get("dtype", 1), [x for x in ALL if x != "n"]
    need = H.hla2_window_step_workspace_bytes(*ints(kw, *names), dt)
    assert L.hla2_window_step(kw.get("cache_k", P), P, kw.get("pos", P), kw.get("q", P), P, P, P, *ints(kw, *names),
                              kw.get("scale", 1.0), dt, kw.get("ws", P), need - kw.get("short", 0), None) == code


def test_binding_rejects_what_the_c_side_cannot_see():
    q, k, v = torch.zeros(2, 4, 10, 16), torch.zeros(2, 2, 10, 16), torch.zeros(2, 2, 10, 32)
    out, lse = torch.zeros(2, 4, 10, 32), torch.zeros(2, 4, 10)
    with pytest.raises(ValueError, match="GPU"):
        H.hla2_window_forward(q, k, v, out, 4)
    for bad in (dict(k=k[:, :, :9]), dict(v=v.bfloat16()), dict(out=torch.zeros(2, 4, 10, 16)),
                dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=lse.double()), dict(lse=lse[:1]),
                dict(lens=torch.zeros(2)), dict(q=q[0])):
        with pytest.raises(ValueError):
            H.hla2_window_forward(**{**dict(q=q, k=k, v=v, out=out, window=4), **bad})
    with pytest.raises(ValueError):
        H.hla2_window_backward(q, k, v, out, lse, out, q, k, k, 4)  # dv has k's shape
    with pytest.raises(ValueError):
        H.hla2_window_cache(k, v, torch.zeros(2, 2, 5, 16), torch.zeros(2, 2, 6, 32), 4, 2)
    ck, cv = torch.zeros(2, 2, 6, 16), torch.zeros(2, 2, 6, 32)
    step = dict(cache_k=ck, cache_v=cv, pos=torch.zeros(2, dtype=torch.int32), q=q[:, :, 0].contiguous(),
                k=k[:, :, 0].contiguous(), v=v[:, :, 0].contiguous(), out=out[:, :, 0].contiguous(), window=4, sinks=2)
    with pytest.raises(ValueError, match="pos"):
        H.hla2_window_step(**step)
    with pytest.raises(ValueError, match="cache_k"):
        H.hla2_window_step(**{**step, "window": 5})


def test_integers_that_would_be_cut_off():
    q, out = torch.zeros(1, 1, 4, 16), torch.zeros(1, 1, 4, 16)
    for bad in (dict(window=2 ** 32 + 4), dict(window=4, sinks=2 ** 33)):
        with pytest.raises(ValueError, match="32 bits"):
            H.hla2_window_forward(q, q, q, out, **bad)


def test_oracle_gradients_against_differences():
    r = np.random.default_rng(5)
    q, k, v = r.standard_normal((2, 4, 9, 3)), r.standard_normal((2, 2, 9, 3)), r.standard_normal((2, 2, 9, 2))
    dout, lens, args = r.standard_normal((2, 4, 9, 2)), [9, 5], (3, 2, 0.6)

    def loss(q, k, v):
        return float((M.window_attention(q, k, v, *args, lens)[0] * dout).sum())

    got = M.window_attention_backward(q, k, v, dout, *args, lens)
    for i, arr in enumerate((q, k, v)):
        num = np.zeros_like(arr)
        for at in np.ndindex(arr.shape):
            pair = []
            for sign in (1, -1):
                xs = [q.copy(), k.copy(), v.copy()]
                xs[i][at] += sign * 1e-5
                pair.append(loss(*xs))
            num[at] = (pair[0] - pair[1]) / 2e-5
        # central differences: the third derivative times h^2 / 6, and cancellation of 1e-16 / h
        np.testing.assert_allclose(got[i], num, atol=1e-8)


def test_oracle_ring_holds_what_the_next_query_sees():
    for window, sinks in ((1, 0), (3, 2), (5, 1), (4, 7)):
        ring = {}
        for p in range(30):
            ring[M.cache_slot(p, window, sinks)] = p
            assert sorted(ring.values()) == sorted(np.flatnonzero(M.visible(p + 1, window, sinks)[p]))
            assert sorted(ring) == list(range(min(p + 1, window + sinks)))


def test_backward_launch_limit(L):
    """The keys' walk and the far runs share a launch: what the forward call takes can pass its limit."""
    kw = dict(B=1000, H=12000, Hkv=1, n=20, window=10)
    assert H.hla2_window_backward_workspace_bytes(*ints(kw, *ALL), 1) == 0
    assert H.hla2_window_backward_workspace_bytes(*ints(dict(kw, window=20), *ALL), 1) > 0  # no far queries
    assert L.hla2_window_backward(P, P, P, P, P, P, P, P, P, None, *ints(kw, *ALL), 1.0, 1, P, 1 << 40, None) == UNS


def test_launch_limits_are_those_of_64_rows(L):
    """B H ceil(n / 64) below 2^24 - 8, whatever B H n: the shape passes where the next check, of alignment, is what
    refuses the call."""
    def code(call, **kw):
        if call == "cache":
            return L.hla2_window_cache(ODD, P, P, P, None, *ints(kw, "B", "Hkv", "n", "d", "dv", "window", "sinks"), 1, None)
        if call == "forward":
            return L.hla2_window_forward(ODD, P, P, P, None, None, *ints(kw, *ALL), 1.0, 1, None)
        return L.hla2_window_backward(ODD, P, P, P, P, P, P, P, P, None, *ints(kw, *ALL), 1.0, 1, None, 0, None)

    small = dict(d=16, dv=16, window=8, sinks=0)
    for call in ("forward", "cache", "backward"):
        for good in (dict(B=1 << 9, H=8, Hkv=8, n=1 << 16), dict(B=1 << 9, H=32, Hkv=32, n=1 << 15),
                     dict(B=1, H=(1 << 18) - 1, Hkv=(1 << 18) - 1, n=1 << 12)):
            assert good["B"] * good["H"] * good["n"] >= 1 << 28
            assert code(call, **small, **good) == INV
        assert code(call, **small, B=1, H=1 << 18, Hkv=1 << 18, n=1 << 12) == UNS
    assert H.hla2_window_backward_workspace_bytes(*ints(dict(small, B=1 << 9, H=8, Hkv=8, n=1 << 16), *ALL), 1) == 4 << 28
