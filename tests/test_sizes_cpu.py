"""Sizes that do not fit the C side's 32-bit integers are refused by the binding and not cut off; the tensors here
have shapes and no memory."""
import pytest
import torch

from causal_prefix_scan_hla2_amd import hla2 as H

BIG = 2 ** 32 + 5  # cut to 32 bits: 5


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("shape", [(BIG, 1, 1, 1), (1, BIG, 1, 1), (1, 1, BIG, 1), (1, 1, 1, BIG), (1, BIG, 1), (2 ** 31, 1, 1)])
def test_scan(shape):
    x = meta(*shape)
    marks = torch.zeros(1)
    with pytest.raises(ValueError, match="32 bits"):
        H.hla2_gated_scan_forward(x, x, x)
    with pytest.raises(ValueError, match="32 bits"):
        H.hla2_gated_scan_backward(x, x, x, x, x, marks=marks)


@pytest.mark.parametrize("shape", [(BIG, 1, 1), (1, BIG, 1), (1, 1, BIG), (BIG, 1), (1, BIG)])
def test_scan_step(shape):
    x = meta(*shape)
    with pytest.raises(ValueError, match="32 bits"):
        H.hla2_gated_scan_step(meta(*shape, dtype=torch.float32), x, x, x)


FULL = dict(B=1, H=2, Hkv=1, n=4, d=16, dv=16)


@pytest.mark.parametrize("big", [dict(B=BIG), dict(H=2 * BIG), dict(H=2 * BIG, Hkv=BIG), dict(n=BIG), dict(d=BIG), dict(dv=BIG)])
def test_window(big):
    s = {**FULL, **big}
    q, k = meta(s["B"], s["H"], s["n"], s["d"]), meta(s["B"], s["Hkv"], s["n"], s["d"])
    v, out = meta(s["B"], s["Hkv"], s["n"], s["dv"]), meta(s["B"], s["H"], s["n"], s["dv"])
    lse = meta(s["B"], s["H"], s["n"], dtype=torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        H.hla2_window_forward(q, k, v, out, 4)
    with pytest.raises(ValueError, match="32 bits"):
        H.hla2_window_backward(q, k, v, out, lse, out, q, k, v, 4)
    if big.get("Hkv") or "H" not in big:
        with pytest.raises(ValueError, match="32 bits"):
            H.hla2_window_cache(k, v, meta(s["B"], s["Hkv"], 4, s["d"]), meta(s["B"], s["Hkv"], 4, s["dv"]), 4)
    if "n" not in big:
        cache = [meta(s["B"], s["Hkv"], 4, s[x]) for x in ("d", "dv")]
        with pytest.raises(ValueError, match="32 bits"):
            H.hla2_window_step(*cache, meta(s["B"], dtype=torch.int64), q[:, :, 0].contiguous(), k[:, :, 0].contiguous(),
                               v[:, :, 0].contiguous(), out[:, :, 0].contiguous(), 4)


def test_workspace_queries():
    for sizes in ((BIG, 1, 600, 4), (1, BIG, 600, 4), (1, 1, BIG + 600, 4), (1, 1, 600, BIG)):
        with pytest.raises(ValueError, match="32 bits"):
            H.hla2_gated_scan_workspace_bytes(*sizes, H.HLA2_F32)
    good = [1, 2, 1, 4, 16, 16, 4, 0]
    for i in range(len(good)):
        bad = [x + (i == j) * 2 ** 32 for j, x in enumerate(good)]
        with pytest.raises(ValueError, match="32 bits"):
            H.hla2_window_backward_workspace_bytes(*bad, H.HLA2_BF16)
        if i != 3:
            with pytest.raises(ValueError, match="32 bits"):
                H.hla2_window_step_workspace_bytes(*(bad[:3] + bad[4:]), H.HLA2_BF16)


def test_large_tensors_of_ordinary_sizes_pass_this_check():
    x = meta(17, 16, 65536, 128)  # 2.3e9 elements: refused only for having no memory
    with pytest.raises(ValueError, match="GPU"):
        H.hla2_gated_scan_forward(x, x, x)


@pytest.mark.parametrize("shape", [(BIG, 1, 64, 64), (1, BIG, 64, 64), (1, 1, BIG, 64)])
def test_linear_forms(shape):
    x = meta(*shape)
    for call in (H.hla2_forward, H.hla2_forward_noalloc, H.hla2_ahla_forward, H.hla2_ho3_forward):
        with pytest.raises(ValueError, match="32 bits"):
            call(x, x, x, x)
    with pytest.raises(ValueError, match="32 bits"):
        H.hla2_forward_state(x, x, x, x, x)
    with pytest.raises(ValueError, match="32 bits"):
        H.hla2_backward(x, x, x, x, x, x, x)
    if shape[2] == 64:
        t = meta(shape[0], shape[1], 64)
        with pytest.raises(ValueError, match="32 bits"):
            H.hla2_decode_step(t, t, t, t, t)
