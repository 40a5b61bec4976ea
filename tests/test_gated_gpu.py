"""The gated linear recurrence on the GPU against its fp64 definition.

Bounds, elementwise.  u = 2^-24 is fp32's half step.  With M_t = a_t M_{t-1} + |b_t| the state computed in
fp32 is off by at most E_t = a_t E_{t-1} + c u M_t: c counts, per token, the gate's rounding (exp and its
argument, division, and one product where gates are multiplied up: 6), the multiply-add and its operand (3),
and one rounding each where the token's result passes a thread's, a wave's and a tile's end (3); c = 12.
The sigmoid gate is applied as x + a (s - x): with the gate off by a relative e and the difference by u the
token's error is at most a |s - x| (e + u) + u |s_t| <= c u (a |s| + a |x|) + u |s_t|, so its source term is
c u (M_t + a_t |x_t|).
The adjoint is the same recurrence backwards.  A product of computed factors adds the factors' errors and
4 roundings.  An output in `dtype` adds its half step, finfo.eps / 2 relative to the value.
"""
import numpy as np
import pytest
import torch

from causal_prefix_scan_hla2_amd import hla2 as H
from oracle import mixers as M
from tests.parity import TOL_BF16, TOL_F32, rel_l2

pytestmark = pytest.mark.gpu

U, C = 2.0 ** -24, 12.0
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def draw(B, Hh, n, d, dtype, gate, seed=0, slow=False):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    g = -torch.nn.functional.softplus(1.5 * r(B, Hh, n, d) - (7.0 if slow else 2.0))
    if gate == M.SIGMOID:
        g = 1.5 * r(B, Hh, n, d) + (6.0 if slow else 2.0)
    t = DT[dtype]
    return dict(x=r(B, Hh, n, d).to(t), g=g.to(t), s0=r(B, Hh, d), dout=r(B, Hh, n, d).to(t), ds_last=r(B, Hh, d))


def scan_error(a, b, m0, lens, mixed):
    """E_t of the module docstring, and M_t; m0: magnitudes of the first state; mixed: a |x| for the sigmoid
    gate, 0 for the log gate."""
    B, _, n, _ = a.shape
    M_, E = np.zeros_like(a), np.zeros_like(a)
    m, e = np.abs(m0).copy(), np.zeros_like(m0)
    for i, end in enumerate(lens):
        for t in range(end):
            m[i] = a[i, :, t] * m[i] + np.abs(b[i, :, t])
            e[i] = a[i, :, t] * e[i] + C * U * (m[i] + mixed[i, :, t])
            M_[i, :, t], E[i, :, t] = m[i], e[i]
    return M_, E, m, e


def near(got, ref, err, dtype, what):
    half = torch.finfo(DT[dtype]).eps / 2
    bad = np.abs(got - ref) > err * (1 + half) + half * np.abs(ref) + 1e-37
    assert not bad.any(), "%s: %d off, worst %.3g at ref %.3g" % (
        what, bad.sum(), np.abs(got - ref)[bad].max(), ref[bad][0])


def call(c, gate, lens=None, use_s0=True, train=True, stream=None, aligned=True):
    dev = torch.device("cuda:0")
    D = {k: v.to(dev) for k, v in c.items()}
    if not aligned:  # every 16-byte vector starts one element late
        for k in ("x", "g", "dout"):
            buf = torch.empty(D[k].numel() + 1, dtype=D[k].dtype, device=dev)
            buf[1:] = D[k].reshape(-1)
            D[k] = buf[1:].view(D[k].shape)
    B, Hh, n, d = D["x"].shape
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=dev)
    poison = lambda *s, dtype=torch.float32: torch.full(s, 7.0, dtype=dtype, device=dev)  # noqa: E731
    t = D["x"].dtype
    out, last = poison(B, Hh, n, d, dtype=t), poison(B, Hh, d)
    marks = poison(B, Hh, (n + 255) // 256, d)
    s0 = D["s0"] if use_s0 else None
    H.hla2_gated_scan_forward(D["x"], D["g"], out, gate=gate, s0=s0, s_last=last, marks=marks if train else None,
                              lens=lt, stream=stream)
    got = dict(out=out, last=last)
    if train:
        dx, dg, ds0 = poison(B, Hh, n, d, dtype=t), poison(B, Hh, n, d, dtype=t), poison(B, Hh, d)
        H.hla2_gated_scan_backward(D["x"], D["g"], D["dout"], dx, dg, gate=gate, s0=s0, marks=marks,
                                   ds_last=D["ds_last"] if use_s0 else None, ds0=ds0, lens=lt, stream=stream)
        got |= dict(dx=dx, dg=dg, ds0=ds0)
    return got


def check(c, gate, dtype, lens=None, use_s0=True, got=None, aligned=True):
    got = got or call(c, gate, lens, use_s0, aligned=aligned)
    torch.cuda.synchronize()
    B, Hh, n, d = c["x"].shape
    ends = M._lens(lens, B, n)
    x, g, dout = f64(c["x"]), f64(c["g"]), f64(c["dout"])
    zero = np.zeros((B, Hh, d))
    s0, dl = (f64(c["s0"]), f64(c["ds_last"])) if use_s0 else (zero, zero)
    a, b, z = M.gates(x, g, gate)
    s, last = M.gated_scan(x, g, gate, s0, lens)
    mag, E, _, e_last = scan_error(a, z * np.abs(x), s0, ends, (1 - z if gate == M.SIGMOID else 0 * a) * np.abs(x))
    live = np.zeros((B, 1, n, 1), bool)
    for i, m in enumerate(ends):
        live[i, :, :m] = True
    L = np.broadcast_to(live, x.shape)
    for k in ("out", "dx", "dg"):
        v = f64(got[k])
        assert (v[~L] == 7.0).all(), "%s written behind a sequence's end" % k
    near(f64(got["out"])[L], s[L], E[L], dtype, "out")
    near(f64(got["last"]), last, e_last, "f32", "s_last")
    dx, dg, ds0 = M.gated_scan_backward(x, g, gate, dout, s0, dl, lens)
    # magnitudes and errors of r_t: the recurrence reversed, within each sequence
    R, Er = np.zeros_like(x), np.zeros_like(x)
    m0, e0 = np.abs(dl).copy(), np.zeros_like(dl)
    for i, end in enumerate(ends):
        for t in range(end - 1, -1, -1):
            r = np.abs(dout[i, :, t]) + m0[i]
            er = e0[i] + C * U * r
            R[i, :, t], Er[i, :, t] = r, er
            m0[i], e0[i] = a[i, :, t] * r, a[i, :, t] * er
    Mb = np.concatenate([np.abs(s0)[:, :, None], mag[:, :, :-1]], 2)
    Eb = np.concatenate([np.zeros_like(s0)[:, :, None], E[:, :, :-1]], 2)
    if gate == M.SIGMOID:
        Mb = Mb + np.abs(x)
        Eb = Eb + U * Mb
    near(f64(got["dx"])[L], dx[L], (z * (Er + C * U * R))[L], dtype, "dx")
    near(f64(got["dg"])[L], dg[L], (a * z * (Er * Mb + R * Eb + C * U * R * Mb))[L], dtype, "dg")
    near(f64(got["ds0"]), ds0, e0 + C * U * m0, "f32", "ds0")
    return got


SHAPES = [  # B, H, n, d
    (1, 1, 1, 1), (2, 3, 1, 64), (1, 2, 2, 3), (2, 2, 7, 8), (1, 1, 255, 33), (1, 1, 256, 64), (1, 2, 257, 40),
    (3, 1, 300, 130), (1, 1, 1025, 17), (2, 2, 777, 128), (1, 1, 4099, 8),
]


@pytest.mark.parametrize("gate", [M.LOG, M.SIGMOID])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype, gate):
    check(draw(*shape, dtype, gate, seed=sum(shape)), gate, dtype)


@pytest.mark.parametrize("gate", [M.LOG, M.SIGMOID])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 37])
def test_ragged_lengths(dtype, gate, d):
    # an empty sequence, one token, a whole tile, one more, a negative and a too large length
    c = draw(7, 2, 600, d, dtype, gate, seed=4)
    check(c, gate, dtype, lens=[600, 0, 1, 256, 257, -3, 9999])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_padding_is_not_read(dtype):
    c = draw(2, 1, 520, 16, dtype, M.LOG, seed=9)
    want = check(c, M.LOG, dtype, lens=[300, 513])
    bad = {k: v.clone() for k, v in c.items()}
    for k in ("x", "g", "dout"):
        bad[k][0, :, 300:], bad[k][1, :, 513:] = float("nan"), float("inf")
    got = call(bad, M.LOG, lens=[300, 513])
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_no_first_state_and_odd_alignment():
    for dtype in ("f32", "bf16"):
        check(draw(2, 2, 530, 64, dtype, M.SIGMOID, seed=5), M.SIGMOID, dtype, use_s0=False)
        check(draw(2, 2, 530, 64, dtype, M.LOG, seed=6), M.LOG, dtype, aligned=False)


@pytest.mark.parametrize("gate", [M.LOG, M.SIGMOID])
def test_slow_gates_over_many_tiles(gate):
    check(draw(1, 2, 9000, 72, "f32", gate, seed=8, slow=True), gate, "f32")


def test_gate_edges():
    """-inf resets, gates above 0 count as 0 with no gradient, large logits saturate without NaN."""
    c = draw(1, 1, 600, 8, "f32", M.LOG, seed=2)
    c["g"][:, :, 100], c["g"][:, :, 300:310], c["g"][:, :, 400] = -float("inf"), 0.5, 0.0
    c["g"][:, :, 500] = -200.0
    got = check(c, M.LOG, "f32")
    assert torch.equal(got["out"][:, :, 100].cpu(), c["x"][:, :, 100])
    assert (got["dg"][:, :, 300:310] == 0).all() and (got["dg"][:, :, 400] != 0).all()
    c = draw(1, 1, 600, 8, "f32", M.SIGMOID, seed=3)
    c["g"][:, :, 50], c["g"][:, :, 70], c["g"][:, :, 90], c["g"][:, :, 95] = 200.0, -200.0, float("inf"), -float("inf")
    check(c, M.SIGMOID, "f32")


def test_nan_stays_in_its_channel_and_after_its_token():
    c = draw(1, 1, 700, 64, "bf16", M.LOG, seed=12)
    c["x"][0, 0, 350, 5] = float("nan")
    out = call(c, M.LOG, train=False)["out"].float().cpu()
    nan = torch.isnan(out[0, 0])
    assert nan[350:, 5].all() and nan.sum() == 350


@pytest.mark.parametrize("gate", [M.LOG, M.SIGMOID])
def test_last_state_may_be_the_first_states_buffer(gate):
    c = draw(2, 2, 1000, 64, "bf16", gate, seed=7)
    want = call(c, gate)
    dev = torch.device("cuda:0")
    D = {k: v.to(dev) for k, v in c.items()}
    state, out = D["s0"].clone(), torch.empty_like(D["x"])
    H.hla2_gated_scan_forward(D["x"], D["g"], out, gate=gate, s0=state, s_last=state)
    assert torch.equal(state, want["last"]) and torch.equal(out, want["out"])


@pytest.mark.parametrize("gate", [M.LOG, M.SIGMOID])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_prefill_then_steps_equal_the_whole(dtype, gate):
    c = draw(3, 2, 300, 72, dtype, gate, seed=10)
    dev = torch.device("cuda:0")
    D = {k: v.to(dev) for k, v in c.items()}
    whole = check(c, gate, dtype)
    n0 = 280
    state, out = torch.empty_like(D["s0"]), torch.empty_like(D["x"][:, :, :n0])
    H.hla2_gated_scan_forward(D["x"][:, :, :n0].contiguous(), D["g"][:, :, :n0].contiguous(), out, gate=gate,
                              s0=D["s0"], s_last=state)
    a, b, z = M.gates(f64(c["x"]), f64(c["g"]), gate)
    mixed = (1 - z if gate == M.SIGMOID else 0 * a) * np.abs(f64(c["x"]))
    _, E, _, _ = scan_error(a, z * np.abs(f64(c["x"])), f64(c["s0"]), [300] * 3, mixed)
    ref, _ = M.gated_scan(f64(c["x"]), f64(c["g"]), gate, f64(c["s0"]))
    for t in range(n0, 300):
        o = torch.empty_like(D["x"][:, :, 0])
        H.hla2_gated_scan_step(state, D["x"][:, :, t].contiguous(), D["g"][:, :, t].contiguous(), o, gate=gate)
        near(f64(o), ref[:, :, t], E[:, :, t], dtype, "step %d" % t)
    near(f64(state), f64(whole["last"]), 2 * E[:, :, -1], "f32", "state")


def test_step_leaves_idle_sequences():
    dev = torch.device("cuda:0")
    gen = torch.Generator().manual_seed(1)
    x, g, st = (torch.randn(5, 3, 9, generator=gen).to(dev) for _ in range(3))
    pos = torch.tensor([0, -1, 1 << 33, -(1 << 40), 4], device=dev)
    out, state = torch.full_like(x, 7.0), st.clone()
    H.hla2_gated_scan_step(state, x, g, out, gate=H.HLA2_GATE_SIGMOID, pos=pos)
    idle = torch.tensor([1, 3], device=dev)
    assert torch.equal(state[idle], st[idle]) and (out[idle] == 7).all()
    a, b, _ = M.gates(f64(x), f64(g), M.SIGMOID)
    live = [0, 2, 4]
    ref = (a * f64(st) + b)[live]
    near(f64(out)[live], ref, C * U * (np.abs(f64(st)) + np.abs(f64(x)))[live], "f32", "out")


def test_captured_and_replayed():
    """Forward and backward in one graph, replayed with eager work between, each replay on new inputs."""
    dev = torch.device("cuda:0")
    c = draw(2, 2, 1500, 64, "bf16", M.SIGMOID, seed=21)
    D = {k: v.to(dev) for k, v in c.items()}
    out, dx, dg = (torch.empty_like(D["x"]) for _ in range(3))
    last, ds0 = torch.empty_like(D["s0"]), torch.empty_like(D["s0"])
    marks = torch.empty(2, 2, 6, 64, device=dev)
    ws = torch.empty(max(1, H.hla2_gated_scan_workspace_bytes(2, 2, 1500, 64, H.HLA2_BF16)), dtype=torch.uint8, device=dev)

    def both():
        H.hla2_gated_scan_forward(D["x"], D["g"], out, gate=M.SIGMOID, s0=D["s0"], s_last=last, marks=marks, workspace=ws)
        H.hla2_gated_scan_backward(D["x"], D["g"], D["dout"], dx, dg, gate=M.SIGMOID, s0=D["s0"], marks=marks,
                                   ds_last=D["ds_last"], ds0=ds0, workspace=ws)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for k in range(4):
        new = draw(2, 2, 1500, 64, "bf16", M.SIGMOID, seed=30 + k)
        for name, v in new.items():
            D[name].copy_(v.to(dev))
        for t in (out, dx, dg, last, ds0):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        check(new, M.SIGMOID, "bf16", got=dict(out=out, last=last, dx=dx, dg=dg, ds0=ds0))
        want = call(new, M.SIGMOID)
        for name, t in (("out", out), ("last", last), ("dx", dx), ("dg", dg), ("ds0", ds0)):
            assert torch.equal(want[name], t), name


def test_two_streams_at_once():
    """Two calls in flight on two streams, each with its own workspace, equal the calls alone."""
    dev = torch.device("cuda:0")
    cs = [draw(2, 4, 3000, 64, "bf16", M.LOG, seed=s) for s in (40, 41)]
    want = [call(c, M.LOG) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in cs]
    got = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append(call(c, M.LOG))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for k in w:
            assert torch.equal(w[k], g[k]), k


@pytest.mark.parametrize("shape", [(1, 1, 600, 20), (1, 3, 600, 64), (1, 7, 257, 33), (1, 8, 513, 8), (1, 9, 600, 64), (1, 40, 300, 8),
                                   (1, 2, 2049, 64)])
def test_few_slabs(shape):
    """Fewer and more slabs than XCDs, few and many tiles to a slab."""
    check(draw(*shape, "f32", M.LOG, seed=sum(shape)), M.LOG, "f32")
    check(draw(*shape, "bf16", M.SIGMOID, seed=sum(shape)), M.SIGMOID, "bf16")


@pytest.mark.parametrize("gate", [M.LOG, M.SIGMOID])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_gate_of_any_payload(dtype, gate):
    """A NaN gate, here all bits set, passes the tiles after it (before it, backward) in its channel alone."""
    c = draw(1, 1, 1100, 64, dtype, gate, seed=60)
    c["g"].view(torch.int32 if dtype == "f32" else torch.int16)[0, 0, 300, 5] = -1
    got = call(c, gate)
    out, dx = torch.isnan(got["out"][0, 0]), torch.isnan(got["dx"][0, 0])
    assert out[300:, 5].all() and out.sum() == 800
    assert dx[:300, 5].all() and not dx[301:].any() and not dx[:, torch.arange(64, device=dx.device) != 5].any()


# Gates that hold: 1 - a far below a's own rounding step.  What counts there is the relative error of 1 - a, so
# the results meet the bars of tests/parity.py in the 2-norm: 1e-4 for all results of fp32 inputs and for the fp32
# states of bf16 ones, 2e-2 for bf16 outputs.  (A token rounds the state by at most u; over the 9000 tokens here
# that adds up to sqrt(9000) u = 6e-6 in the root mean square, and to a few times that with the tiles' own.)
def gates_that_hold(gate, mean, constant, n, seed, dtype):
    c = draw(1, 2, n, 24, dtype, gate, seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    r = torch.randn(1, 2, 1 if constant else n, 24, generator=gen)
    g = mean + r if gate == M.SIGMOID else -mean * torch.exp(r)
    c["g"] = g.expand(1, 2, n, 24).to(DT[dtype]).contiguous()
    return c


def norms(c, gate, use_s0, dtype):
    got = call(c, gate, use_s0=use_s0)
    x, g, dout = f64(c["x"]), f64(c["g"]), f64(c["dout"])
    s0, dl = (f64(c["s0"]), f64(c["ds_last"])) if use_s0 else (None, None)
    s, last = M.gated_scan(x, g, gate, s0)
    dx, dg, ds0 = M.gated_scan_backward(x, g, gate, dout, s0, dl)
    err = {}
    for k, ref in dict(out=s, last=last, dx=dx, dg=dg, ds0=ds0).items():
        err[k] = rel_l2(f64(got[k]), ref)
    print(gate, err)
    assert all(e <= (TOL_F32 if dtype == "f32" or k in ("last", "ds0") else TOL_BF16) for k, e in err.items()), err


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("use_s0", [False, True])
@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("mean", [8, 10, 12, 14, 16, 18])
def test_sigmoid_gates_that_hold(mean, constant, use_s0, dtype):
    norms(gates_that_hold(M.SIGMOID, mean, constant, 9000, 70 + mean, dtype), M.SIGMOID, use_s0, dtype)


def test_one_token_of_a_sigmoid_gate_that_holds():
    """s = (1 - a) x from a zero state: 1 - a to a few roundings (exp with its argument rounded by |g| u, the sum, the
    division, two products: (8 + |g|) u), in the forward call and in the step."""
    g = torch.tensor([3.0, 9.0, 14.0, 17.0, 20.0, 40.0, 80.0])
    want = 1 / (1 + np.exp(f64(g)))
    dev = torch.device("cuda:0")
    for dtype in ("f32", "bf16"):
        gd = g.to(DT[dtype]).to(dev).view(1, 7)  # every value is one of bf16
        x, st, out = torch.ones_like(gd), torch.zeros(1, 7, device=dev), torch.empty_like(gd)
        H.hla2_gated_scan_step(st, x, gd, out, gate=M.SIGMOID)
        last, o = torch.empty(1, 7, device=dev), torch.empty(1, 1, 7, dtype=DT[dtype], device=dev)
        H.hla2_gated_scan_forward(x.view(1, 1, 7), gd.view(1, 1, 7), o, gate=M.SIGMOID, s_last=last)
        for s in (st, last):
            assert (np.abs(f64(s)[0] - want) <= (8 + f64(g)) * U * want).all()


def test_an_open_sigmoid_gate_holds_its_state():
    """a = 1 to fp32 and 1 - a = 0: the state keeps its bits, whatever the inputs."""
    dev = torch.device("cuda:0")
    for dtype in ("f32", "bf16"):
        c = draw(1, 1, 1500, 40, dtype, M.SIGMOID, seed=77)
        c["g"].fill_(200.0)
        c["x"].mul_(1000.0)
        got = call(c, M.SIGMOID)
        assert torch.equal(got["last"].cpu(), c["s0"])
        assert torch.equal(got["out"].cpu(), c["s0"][:, :, None].to(DT[dtype]).expand_as(c["x"]))
        st, o = c["s0"].to(dev).clone(), torch.empty(1, 1, 40, dtype=DT[dtype], device=dev)
        H.hla2_gated_scan_step(st, c["x"][:, :, 0].contiguous().to(dev), c["g"][:, :, 0].contiguous().to(dev), o, gate=M.SIGMOID)
        assert torch.equal(st.cpu(), c["s0"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("use_s0", [False, True])
@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("size", [1e-2, 1e-3, 1e-4, 1e-5, 1e-6])
def test_log_gates_that_hold(size, constant, use_s0, dtype):
    """Constant decays over 40000 tokens: sqrt(40000) u = 1.2e-5 in the root mean square."""
    norms(gates_that_hold(M.LOG, size, constant, 40000, 90, dtype), M.LOG, use_s0, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_of_a_state_by_a_log_gate(dtype):
    """n tokens of one gate and no input: s = exp(n g) s0.  A token's factor is off by at most 4 u of 1 - a (the
    series' rest, three multiply-adds and one product) or 4 u of a, and its product by u; so 4 u n |g| + u n in
    all, and 12 u for the tiles' maps of each 256 tokens."""
    n, g = 5000, torch.tensor([-2.0 ** -k for k in range(2, 24)])
    c = dict(x=torch.zeros(1, 1, n, 22), g=g.expand(1, 1, n, 22).contiguous(), s0=torch.ones(1, 1, 22),
             dout=torch.zeros(1, 1, n, 22), ds_last=torch.ones(1, 1, 22))
    for k in ("x", "g", "dout"):
        c[k] = c[k].to(DT[dtype])
    got = call(c, M.LOG)
    t = np.arange(1, n + 1)[:, None]
    want = np.exp(t * f64(g)[None])
    err = U * (4 * t * np.abs(f64(g)) + t + 12 * (t // 256 + 1)) * want
    near(f64(got["out"])[0, 0], want, err, dtype, "out")
    for k in ("last", "ds0"):
        near(f64(got[k])[0, 0], want[-1], err[-1], "f32", k)
