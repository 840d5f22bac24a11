"""GPU parity of linear attention with a decay for each head (forward,
backward, single-token step) against the float64 oracle
``oracle.linattn_decay``.

Bounds, from the roundings each path makes:
* bfloat16: the masked scores, the copy of the state that the queries meet and
  the result are rounded once each, by at most half a step (2^-8 of the
  value).  Elementwise the error is at most 2^-8 (A + |ref|) with A the same
  sums over absolute values, plus float32's share; over a tensor the three
  errors are independent and each has an rms of at most 2^-8 / sqrt(3), so
  the relative 2-norm stays below 2^-8 (3.9e-3); the bound is 5e-3.
* float32, and float32 states of both: sums of at most T + D terms with
  relative roundings of 2^-24, rms below sqrt(T + D) 2^-24 < 1e-5 up to the
  lengths here.  On the tensor cores a state's keys are two bfloat16 terms: the
  weight is cut at 2^-18 of it and the second term, at most 2^-8 of the
  product, rounded by at most 2^-9 of itself: 2^-18 + 2^-17 = 1.2e-5 of a product at
  most, and an rms of at most 1 / sqrt(3) of that, 6.6e-6, over independent
  products.
"""
import numpy as np
import pytest
import torch

import rwkv_linear_rnn_b200 as W
from oracle import linattn_decay as ld

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
REL = {"f32": 1e-5, "bf16": 5e-3}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
STATE_REL = 1e-5


def rel(x, ref):
    x, ref = np.asarray(x, np.float64).ravel(), np.asarray(ref, np.float64).ravel()
    assert np.all(np.isfinite(x))
    return np.linalg.norm(x - ref) / max(np.linalg.norm(ref), 1e-30)


def host(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Random inputs on the device and, rounded to the element type, on the host."""

    def __init__(self, seed, B, T, H, D, M, dtype, layout="bthd", state=False, lengths=None, decay=None, fused=False):
        rng = np.random.default_rng(seed)
        self.shape = B, T, H, D, M
        self.dtype = dtype

        def tensor(width):
            t = torch.from_numpy(rng.normal(size=(B, T, H, width)).astype(np.float32)).cuda().to(TYPES[dtype])
            if layout == "bhtd":  # heads outside positions
                t = t.transpose(1, 2).contiguous().transpose(1, 2)
            elif layout == "fused":  # a slice of a wider row
                wide = torch.zeros(B, T, H, width + 16, dtype=t.dtype, device="cuda")
                wide[..., 8:8 + width] = t
                t = wide[..., 8:8 + width]
            elif layout == "odd":  # off every vector alignment
                flat = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
                flat[1:] = t.reshape(-1)
                t = flat[1:].view(B, T, H, width)
            return t

        self.q, self.k, self.v, self.go = tensor(D), tensor(D), tensor(M), tensor(M)
        if decay is None:
            decay = -np.exp2(-8.0 * np.arange(1, H + 1) / H) * rng.uniform(0.5, 1.5, H)
        self.decay = np.asarray(decay, np.float32)
        self.g = torch.from_numpy(self.decay).cuda()
        self.state = self.gs = None
        if state:
            self.state, self.gs = (torch.from_numpy(rng.normal(size=(B, H, D, M)).astype(np.float32)).cuda()
                                   for _ in range(2))
        self.lengths = None
        if lengths is not None:
            self.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
            # what lies behind a row's length is not used, whatever it holds
            for b, n in enumerate(lengths):
                for t in (self.q, self.k, self.v, self.go):
                    t[b, min(max(n, 0), T):] = float("nan")
        self.scale = D ** -0.5

    def host(self, *names):
        got = []
        for n in names:
            t = getattr(self, n)
            if t is None or n == "decay":
                got.append(t)
                continue
            x = host(t)
            got.append(np.nan_to_num(x) if n in ("q", "k", "v", "go") else x)
        return got

    def n(self):
        return None if self.lengths is None else self.lengths.tolist()


def check_forward(c):
    q, k, v, state = c.host("q", "k", "v", "state")
    out, s = W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, scale=c.scale, lengths=c.lengths, want_state=True)
    ref, s_ref = ld.fwd_recur(q, k, v, c.decay, state, c.scale, c.n())
    assert out.shape == ref.shape and out.dtype == c.q.dtype
    assert rel(host(out), ref) <= REL[c.dtype]
    big = np.abs(ld.fwd_recur(*(np.abs(x) for x in (q, k, v)), c.decay, None if state is None else np.abs(state),
                              c.scale, c.n())[0])
    slack = (c.shape[1] + c.shape[3] + 16) * 2.0 ** -24
    assert np.all(np.abs(host(out) - ref) <= HALF_STEP[c.dtype] * (big + np.abs(ref)) + slack * big + 1e-30)
    assert rel(host(s), s_ref) <= STATE_REL
    # without the state asked for, the same outputs to the same bounds
    out2, none = W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, scale=c.scale, lengths=c.lengths)
    assert none is None
    assert rel(host(out2), ref) <= REL[c.dtype]
    return out


def check_backward(c):
    q, k, v, go, state, gs = c.host("q", "k", "v", "go", "state", "gs")
    got = W.linattn_decay_backward(c.q, c.k, c.v, c.g, c.go, c.state, scale=c.scale, lengths=c.lengths,
                                   grad_state_out=c.gs, want_grad_state=True)
    ref = ld.bwd_recur(q, k, v, c.decay, go, state, c.scale, c.n(), gs)
    for name, a, b in zip(("gq", "gk", "gv"), got, ref):
        assert a.shape == b.shape and a.dtype == c.q.dtype
        assert rel(host(a), b) <= REL[c.dtype], name
    assert rel(host(got[3]), ref[3]) <= STATE_REL


SIZES = [1, 2, 15, 16, 17, 31, 33, 64, 127, 128, 129, 200, 256, 257, 300, 511]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", SIZES)
def test_lengths_from_one_token_up(T, dtype):
    c = Case(T, 2, T, 3, 64, 64, dtype, state=T % 2 == 0)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,M", [(1, 1), (3, 5), (8, 8), (8, 128), (17, 33), (32, 32), (40, 72), (64, 128), (72, 40),
                                 (128, 64), (96, 96), (120, 8), (127, 101), (128, 128)])
def test_head_sizes(D, M, dtype):
    c = Case(D * M, 1, 161, 2, D, M, dtype, state=True)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["bhtd", "fused", "odd"])
def test_layouts(layout, dtype):
    for D, M in ((64, 64), (128, 96)):
        c = Case(7, 2, 150, 3, D, M, dtype, layout=layout, state=True)
        check_forward(c)
        check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_padded_rows(D, dtype):
    """Rows of every length, none included; NaN behind them; zeros come out there."""
    lengths = [0, 1, 128, 129, 300, 257, -5, 1000]
    c = Case(11, len(lengths), 300, 2, D, D, dtype, state=True, lengths=lengths)
    out = check_forward(c)
    check_backward(c)
    for b, n in enumerate(lengths):
        assert not host(out)[b, min(max(n, 0), 300):].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_empty_rows_pass_the_state(dtype):
    c = Case(12, 2, 200, 2, 64, 64, dtype, state=True, lengths=[0, 0])
    out, s = W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, lengths=c.lengths, want_state=True)
    assert not out.any() and torch.equal(s, c.state)
    *grads, gs = W.linattn_decay_backward(c.q, c.k, c.v, c.g, c.go, c.state, lengths=c.lengths, grad_state_out=c.gs,
                                          want_grad_state=True)
    assert not any(x.any() for x in grads) and torch.equal(gs, c.gs)
    _, s = W.linattn_decay_forward(c.q, c.k, c.v, c.g, lengths=c.lengths, want_state=True)
    assert not s.any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_positions(dtype):
    z = torch.empty(2, 0, 3, 32, dtype=TYPES[dtype], device="cuda")
    g = torch.full((3,), -0.1, device="cuda")
    s = torch.randn(2, 3, 32, 32, device="cuda")
    out, s1 = W.linattn_decay_forward(z, z, z, g, s, want_state=True)
    assert out.shape == z.shape and torch.equal(s, s1)
    _, s1 = W.linattn_decay_forward(z, z, z, g, want_state=True)
    assert not s1.any()
    *_, gs = W.linattn_decay_backward(z, z, z, g, z, s, grad_state_out=s, want_grad_state=True)
    assert torch.equal(gs, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [[0.0, -1e-7, -1e-4], [-0.5, -2.0, -5.0], [-30.0, -200.0, float("-inf")]])
def test_slow_and_fast_decays(decay, dtype):
    c = Case(13, 1, 700, 3, 64, 64, dtype, state=True, decay=decay)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,M,lengths", [(64, 64, None), (128, 128, [5000, 3333]), (32, 96, [4097, 1])])
def test_long_rows_in_segments(D, M, lengths, dtype):
    """Few heads and many positions: every head is cut into segments."""
    c = Case(14, 2, 5000, 1, D, M, dtype, state=True, lengths=lengths, decay=[-0.004])
    assert W.linattn_decay_workspace_size(0, 2, 5000, 1, D, M, W.WKV_F32 if dtype == "f32" else W.WKV_BF16) > 0
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_more_heads_than_multiprocessors(dtype):
    c = Case(15, 12, 140, 26, 32, 32, dtype)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,M", [(64, 64), (128, 128), (5, 3), (72, 40)])
def test_steps_continue_a_prompt(D, M, dtype):
    """A prompt and then single tokens give what the whole sequence gives."""
    c = Case(16, 3, 150, 2, D, M, dtype)
    q, k, v = c.host("q", "k", "v")
    ref, s_ref = ld.fwd_recur(q, k, v, c.decay, None, c.scale)
    _, s = W.linattn_decay_forward(c.q[:, :130], c.k[:, :130], c.v[:, :130], c.g, scale=c.scale, want_state=True)
    got = []
    for t in range(130, 150):
        y, s2 = W.linattn_decay_step(c.q[:, t], c.k[:, t], c.v[:, t], c.g, s, scale=c.scale)
        assert s2 is s
        got.append(host(y))
    assert rel(np.stack(got, 1), ref[:, 130:]) <= REL[dtype]
    assert rel(host(s), s_ref) <= STATE_REL


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,H,D,M", [(1, 1, 1, 1), (5, 3, 64, 64), (300, 2, 128, 128), (2, 40, 33, 7), (7, 2, 16, 128)])
def test_step(N, H, D, M, dtype):
    rng = np.random.default_rng(N)
    q, k = (torch.from_numpy(rng.normal(size=(N, H, D)).astype(np.float32)).cuda().to(TYPES[dtype]) for _ in range(2))
    v = torch.from_numpy(rng.normal(size=(N, H, M)).astype(np.float32)).cuda().to(TYPES[dtype])
    s = torch.from_numpy(rng.normal(size=(N, H, D, M)).astype(np.float32)).cuda()
    g = -torch.rand(H, device="cuda")
    g[0] = float("-inf") if N == 5 else g[0]
    ref, s_ref = ld.step(*(host(x) for x in (q, k, v, g, s)), 0.25)
    before = s.clone()
    y, s2 = W.linattn_decay_step(q, k, v, g, s, scale=0.25, state_out=torch.empty_like(s))
    assert torch.equal(s, before)
    assert rel(host(y), ref) <= (1e-6 if dtype == "f32" else 2.0 ** -8)
    assert rel(host(s2), s_ref) <= 1e-6
    y2, _ = W.linattn_decay_step(q, k, v, g, s, scale=0.25)  # in place
    assert torch.equal(y, y2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [20, 300])
def test_outputs_given_by_the_caller(T, dtype):
    """Strided outputs are written at their positions and nowhere else; the
    state may be updated in place."""
    c = Case(17, 2, T, 3, 64, 64, dtype, state=True)
    wide = torch.full((2, T + 2, 3, 96), 7.0, dtype=c.q.dtype, device="cuda")
    out = wide[:, 1:T + 1, :, 16:80]
    ref, s_ref = W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, want_state=True)
    got, _ = W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, out=out)
    assert got is out and torch.equal(out, ref)
    assert (wide[:, 0] == 7).all() and (wide[:, -1] == 7).all()
    assert (wide[..., :16] == 7).all() and (wide[..., 80:] == 7).all()
    grads = W.linattn_decay_backward(c.q, c.k, c.v, c.g, c.go, c.state)
    wides = [torch.full((2, T + 2, 3, 96), 7.0, dtype=c.q.dtype, device="cuda") for _ in range(3)]
    W.linattn_decay_backward(c.q, c.k, c.v, c.g, c.go, c.state,
                             **{n: w[:, 1:T + 1, :, 16:80] for n, w in zip(("grad_q", "grad_k", "grad_v"), wides)})
    for w, x in zip(wides, grads):
        assert torch.equal(w[:, 1:T + 1, :, 16:80], x)
        assert (w[:, 0] == 7).all() and (w[:, -1] == 7).all() and (w[..., 80:] == 7).all() and (w[..., :16] == 7).all()
    # the C call with one state buffer for both
    o = torch.empty_like(ref)
    abi, v4 = W.abi, lambda t: W.abi.View(t.data_ptr(), *t.stride()[:3])  # noqa: E731
    dt = W.WKV_F32 if dtype == "f32" else W.WKV_BF16
    need = W.linattn_decay_workspace_size(0, 2, T, 3, 64, 64, dt)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    assert abi.linattn_decay_forward(2, T, 3, 64, 64, dt, v4(c.q), v4(c.k), v4(c.v), c.g.data_ptr(), 1.0, 0,
                                     c.state.data_ptr(), v4(o), c.state.data_ptr(), ws.data_ptr(), need, 0,
                                     torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(o, ref) and torch.equal(c.state, s_ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [40, 300])
def test_autograd(T, dtype):
    """Gradients through the wrapper, a row split in two calls included: they
    equal those of the whole row, to the roundings of the type."""
    c = Case(18, 2, T, 2, 64, 64, dtype, state=True)
    q, k, v, go, state, gs = c.host("q", "k", "v", "go", "state", "gs")
    ref = ld.bwd_recur(q, k, v, c.decay, go, state, c.scale, None, gs)
    x = [t.detach().clone().requires_grad_() for t in (c.q, c.k, c.v, c.state)]
    out, s = W.linattn_decay_state(x[0], x[1], x[2], c.g, x[3], scale=c.scale)
    torch.autograd.backward([out, s], [c.go, c.gs])
    for t, r, tol in zip(x, ref, (REL[dtype],) * 3 + (STATE_REL,)):
        assert rel(host(t.grad), r) <= tol
    y = [t.detach().clone().requires_grad_() for t in (c.q, c.k, c.v, c.state)]
    cut = T // 3
    o1, s1 = W.linattn_decay_state(*(t[:, :cut] for t in y[:3]), c.g, y[3], scale=c.scale)
    o2, s2 = W.linattn_decay_state(*(t[:, cut:] for t in y[:3]), c.g, s1, scale=c.scale)
    torch.autograd.backward([o1, o2, s2], [c.go[:, :cut], c.go[:, cut:], c.gs])
    for t, r, tol in zip(y, ref, (REL[dtype],) * 3 + (STATE_REL,)):
        assert rel(host(t.grad), r) <= tol
    # an expanded gradient, no state, and a gradient for one input alone
    q1 = c.q.detach().clone().requires_grad_()
    W.linattn_decay(q1, c.k, c.v, c.g, scale=c.scale).sum().backward()
    ones = ld.bwd_recur(q, k, v, c.decay, np.ones_like(go), None, c.scale)
    assert rel(host(q1.grad), ones[0]) <= REL[dtype]


def test_broadcast_inputs():
    """Keys shared by all heads through an expanded view; their gradient is
    the heads' sum."""
    torch.manual_seed(3)
    k = torch.randn(2, 100, 1, 64, device="cuda", requires_grad=True)
    q, v, go = (torch.randn(2, 100, 4, 64, device="cuda") for _ in range(3))
    g = torch.tensor([-0.1, -0.2, -0.01, -0.5], device="cuda")
    W.linattn_decay(q, k.expand(2, 100, 4, 64), v, g).backward(go)
    ref = ld.bwd_recur(host(q), np.repeat(host(k), 4, 2), host(v), host(g), host(go))[1].sum(2, keepdims=True)
    assert rel(host(k.grad), ref) <= 1e-5
    # the library itself reads strides of zero
    out, _ = W.linattn_decay_forward(q, k.detach().expand(2, 100, 4, 64), v, g)
    assert rel(host(out), ld.fwd_recur(host(q), np.repeat(host(k), 4, 2), host(v), host(g))[0]) <= 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_same_bits_every_time(dtype):
    c = Case(19, 2, 2500, 2, 64, 128, dtype, state=True)
    runs = []
    for _ in range(3):
        out, s = W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, want_state=True)
        runs.append([out, s, *W.linattn_decay_backward(c.q, c.k, c.v, c.g, c.go, c.state, grad_state_out=c.gs,
                                                       want_grad_state=True)])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_streams_and_graphs(dtype):
    """Calls on two streams at once, and two graphs captured and replayed in
    turn, give what one call alone gives."""
    cs = [Case(20 + i, 1, 3000, 2, 64, 64, dtype, state=True) for i in range(2)]

    def run(c, **kw):
        out, s = W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, want_state=True, **kw)
        return [out, s, *W.linattn_decay_backward(c.q, c.k, c.v, c.g, c.go, c.state, grad_state_out=c.gs,
                                                  want_grad_state=True, **kw)]

    ref = [run(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = [[run(c, stream=s) for _ in range(4)] for c, s in zip(cs, streams)]
    torch.cuda.synchronize()
    for r, g in zip(ref, got):
        for x in g:
            assert all(torch.equal(a, b) for a, b in zip(r, x))
    graphs, outs = [], []
    for c in cs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(run(c))
        graphs.append(graph)
    for s, graph in zip(streams, graphs):
        with torch.cuda.stream(s):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    for r, o in zip(ref, outs):
        assert all(torch.equal(a, b) for a, b in zip(r, o))
    assert W.linattn_decay_status() == 0


def test_a_nan_stays_in_its_head():
    c = Case(22, 2, 300, 2, 64, 64, "bf16")
    c.v[0, 150, 0, 3] = float("nan")
    out, _ = W.linattn_decay_forward(c.q, c.k, c.v, c.g)
    assert out[0, 150:, 0, 3].isnan().all()
    assert not out[0, :128, 0].isnan().any()       # chunks before it
    assert not out[0, :, 1].isnan().any() and not out[1].isnan().any()


def test_wrapper_refusals():
    c = Case(23, 1, 4, 2, 32, 32, "f32")
    q, k, v, g = c.q, c.k, c.v, c.g
    f = W.linattn_decay_forward
    for args, err in [((q.cpu(), k, v, g), ValueError), ((q.half(), k.half(), v.half(), g), TypeError),
                      ((q, k.bfloat16(), v, g), TypeError), ((q, k[:, :3], v, g), ValueError),
                      ((q, k, v, g.double()), ValueError), ((q, k, v, g[:1]), ValueError),
                      ((q[0], k[0], v[0], g), ValueError), ((q.transpose(2, 3), k, v, g), ValueError)]:
        with pytest.raises(err):
            f(*args)
    with pytest.raises(ValueError):
        f(q, k, v, g, lengths=torch.ones(1, device="cuda"))
    with pytest.raises(ValueError):
        f(q, k, v, g, torch.zeros(1, 2, 32, 31, device="cuda"))
    with pytest.raises(W.WKVError):
        f(q, k, v, g, out=q)
    with pytest.raises(W.WKVError):
        big = torch.zeros(1, 4, 2, 160, device="cuda")
        f(big, big, v, g)
