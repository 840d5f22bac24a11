"""Linear attention with a decay for each head and rotary positions where calls
can go wrong: both together as a model runs them, broadcast views, offsets that
pass 32 bits, heads of two sizes with padded rows, threads, and gradients
against differences.

Bounds are those of test_gpu_linattn_decay.py; differences are exact up to
rounding, because the output is linear in each of its inputs.
"""
import threading

import numpy as np
import pytest
import torch

import rwkv_linear_rnn_b200 as W
from oracle import linattn_decay as ld
from rwkv_linear_rnn_b200.constants import WKV_ERR_TIMEOUT
from test_gpu_linattn_decay import REL, STATE_REL, TYPES, Case, check_backward, check_forward, host, rel

pytestmark = pytest.mark.gpu


def rounded(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[dtype]).double().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
def test_a_batch_of_prompts_and_its_next_tokens(D, dtype):
    """Padded prompts with rotary positions, then one token a row at each row's
    own position: what the oracle gives row by row."""
    torch.manual_seed(D)
    lengths = [300, 1, 257, 40]
    B, T, H, new = len(lengths), 300, 3, 4
    qkv = torch.randn(B, T + new, 3, H, D, device="cuda").to(TYPES[dtype])
    q, k, v = (qkv[:, :, i] for i in range(3))
    g = torch.tensor([-0.01, -0.3, -0.002], device="cuda")
    f, m = W.rotary_frequencies(D // 2, scaling="linear", factor=2.0)
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    pos = torch.arange(T, device="cuda")
    a, b = W.linattn_rotary(q[:, :T], k[:, :T], pos, f, mscale=m)
    out, s = W.linattn_decay_forward(a, b, v[:, :T], g, scale=D ** -0.5, lengths=n, want_state=True)
    for r, length in enumerate(lengths):
        row = [host(x[r:r + 1]) for x in (q, k, v)]
        at = list(range(length)) + list(range(T, T + new))  # the row's tokens: its prompt, then the new ones
        p = np.arange(length + new)
        rq, rk = (rounded(ld.rotary(x[:, at], p, host(f), m), dtype) for x in row[:2])
        ref, s_ref = ld.fwd_recur(rq, rk, row[2][:, at], host(g), None, D ** -0.5)
        # bfloat16: the rotated rows differ from the oracle's by a step here and there
        assert rel(host(out[r:r + 1, :length]), ref[:, :length]) <= (1e-5 if dtype == "f32" else 8e-3)
        if r == 0:
            last, last_s = ref, s_ref
    got = []
    for t in range(T, T + new):
        p = (n + (t - T)).long()[:, None]
        a, b = W.linattn_rotary(q[:, t:t + 1], k[:, t:t + 1], p, f, mscale=m)
        y, s = W.linattn_decay_step(a[:, 0], b[:, 0], v[:, t], g, s, scale=D ** -0.5)
        got.append(host(y[:1]))
    assert rel(np.stack(got, 1), last[:, lengths[0]:]) <= (1e-5 if dtype == "f32" else 8e-3)
    assert rel(host(s[:1]), last_s) <= (1e-5 if dtype == "f32" else 4e-3)


@pytest.mark.parametrize("T", [20, 300])
def test_broadcast_bfloat16_keys(T):
    """Keys and values shared by heads through strides of zero."""
    torch.manual_seed(T)
    k, v = (torch.randn(2, T, 1, 64, device="cuda").bfloat16().expand(2, T, 4, 64) for _ in range(2))
    q = torch.randn(2, T, 4, 64, device="cuda").bfloat16()
    g = torch.tensor([-0.1, -0.2, -0.01, -0.5], device="cuda")
    out, s = W.linattn_decay_forward(q, k, v, g, scale=0.125, want_state=True)
    ref, s_ref = ld.fwd_recur(host(q), host(k), host(v), host(g), None, 0.125)
    assert rel(host(out), ref) <= REL["bf16"] and rel(host(s), s_ref) <= STATE_REL


@pytest.mark.parametrize("T", [7, 200])
def test_offsets_beyond_32_bits(T):
    """Batch rows 2^31 elements and more apart, inputs and outputs."""
    far = (1 << 31) + 4096
    B, H, D = 2, 2, 64
    torch.manual_seed(T)
    base = torch.empty(far * (B - 1) + 4 * T * H * D, dtype=torch.bfloat16, device="cuda")

    def view(i):
        return base.as_strided((B, T, H, D), (far, H * D, D, 1), i * T * H * D)

    for i in range(3):
        view(i).copy_(torch.randn(B, T, H, D, device="cuda"))
    q, k, v, out = (view(i) for i in range(4))
    g = torch.tensor([-0.1, -0.02], device="cuda")
    near = [x.contiguous() for x in (q, k, v)]
    ref, s_ref = W.linattn_decay_forward(*near, g, want_state=True)
    got, s = W.linattn_decay_forward(q, k, v, g, want_state=True, out=out)
    assert torch.equal(out, ref) and torch.equal(s, s_ref)
    go = torch.randn_like(ref)
    for x, y in zip(W.linattn_decay_backward(q, k, v, g, go), W.linattn_decay_backward(*near, g, go)):
        assert x is None or torch.equal(x, y)
    y, _ = W.linattn_decay_step(q[:, 0], k[:, 0], v[:, 0], g, s.clone(), out=out[:, 0])
    z, _ = W.linattn_decay_step(*(x[:, 0] for x in near), g, s.clone())
    assert torch.equal(y, z)
    f, _ = W.rotary_frequencies(D)
    pos = torch.arange(T, device="cuda")
    a, b = W.linattn_rotary(q, k, pos, f, out_q=out)
    c, d = W.linattn_rotary(near[0], near[1], pos, f)
    assert torch.equal(a, c) and torch.equal(b, d)


@pytest.mark.parametrize("D,M", [(64, 128), (128, 64), (72, 40), (32, 128)])
def test_padded_rows_with_heads_of_two_sizes(D, M):
    lengths = [0, 129, 300, 1, 128]
    c = Case(D + M, len(lengths), 300, 2, D, M, "bf16", state=True, lengths=lengths, layout="fused")
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,M", [(64, 128), (128, 72)])
def test_segments_with_heads_of_two_sizes(D, M, dtype):
    c = Case(31, 1, 3000, 2, D, M, dtype, state=True, decay=[-0.003, -0.2], lengths=[2900])
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("D,M", [(64, 64), (40, 24), (8, 64)])
def test_two_heads_on_a_multiprocessor(D, M):
    """More heads of up to 64 than multiprocessors (forward 180 of them, backward 540), with every kind of
    decay and padded rows."""
    H = 36
    decay = -np.exp2(-9.0 * np.arange(H) / H)
    decay[:8] = 0.0, -1e-7, -0.5, -2.0, -5.0, -30.0, -200.0, float("-inf")
    lengths = [300, 0, 129, 256, 1]
    c = Case(33, len(lengths), 300, H, D, M, "bf16", state=True, decay=decay, lengths=lengths, layout="fused")
    out = check_forward(c)
    check_backward(c)
    for b, n in enumerate(lengths):
        assert not host(out)[b, n:].any()


def test_two_heads_on_a_multiprocessor_over_many_chunks():
    c = Case(34, 8, 1500, 20, 16, 16, "bf16", state=True)
    check_forward(c)
    check_backward(c)


@pytest.mark.parametrize("T", [3, 90])
def test_gradients_against_differences(T):
    c = Case(32, 2, T, 2, 40, 24, "f32", state=True)
    x = dict(q=c.q, k=c.k, v=c.v, state=c.state)

    def loss(**kw):
        a = x | kw
        out, s = W.linattn_decay_forward(a["q"], a["k"], a["v"], c.g, a["state"], scale=c.scale, want_state=True)
        return (out.double() * c.go.double()).sum() + (s.double() * c.gs.double()).sum()

    grads = W.linattn_decay_backward(c.q, c.k, c.v, c.g, c.go, c.state, scale=c.scale, grad_state_out=c.gs,
                                     want_grad_state=True)
    torch.manual_seed(3)
    for (name, t), grad in zip(x.items(), grads):
        d = torch.randn_like(t)
        diff = float(loss(**{name: t + d}) - loss(**{name: t - d})) / 2
        terms = grad.double() * d.double()
        # float32 roundings of the inputs and sums, against the terms' absolute sum
        assert abs(diff - float(terms.sum())) <= 1e-4 * float(terms.abs().sum()), name


def test_calls_from_two_threads():
    cs = [Case(40 + i, 1, 700, 4, 64, 64, "bf16", state=True) for i in range(2)]
    ref = [W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, want_state=True) for c in cs]
    torch.cuda.synchronize()
    got = [[] for _ in cs]

    def work(i):
        s = torch.cuda.Stream()
        c = cs[i]
        for _ in range(20):
            got[i].append(W.linattn_decay_forward(c.q, c.k, c.v, c.g, c.state, want_state=True, stream=s))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for r, runs in zip(ref, got):
        assert len(runs) == 20 and all(torch.equal(a, b) for x in runs for a, b in zip(x, r))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", [(2, 40, 1, 0, 1024, 1024), (1, 3, 1, 1, 1000, 998), (600, 1, 1, 1, 32, 32),
                                           (1, 2, 70, 3, 128, 48), (3, 2, 2, 2, 80, 40), (20, 1, 1, 0, 8, 2)])
def test_rotary_block_shapes(B, T, Hq, Hk, D, R, interleaved):
    """Many positions to a block, many blocks to a position, several rows to a block."""
    torch.manual_seed(D)
    q = torch.randn(B, T, Hq, D, device="cuda").bfloat16()
    k = torch.randn(B, T, Hk, D, device="cuda").bfloat16() if Hk else None
    pos = torch.randint(0, 10000, (B, T), device="cuda")
    f, _ = W.rotary_frequencies(R)
    oq, ok = W.linattn_rotary(q, k, pos, f, interleaved=interleaved)
    for x, y in ((q, oq), (k, ok)):
        if x is None:
            continue
        ref = ld.rotary(host(x), host(pos), host(f), 1.0, interleaved)
        # half a step of the result, and the pair's float32 roundings (elements are below 8)
        assert np.all(np.abs(host(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -21 * 12)
        assert torch.equal(y[..., R:], x[..., R:])


def test_the_status_word_of_every_way_to_name_the_device():
    q = torch.randn(1, 40, 2, 64, device="cuda").bfloat16()
    W.linattn_decay_forward(q, q, q, torch.zeros(2, device="cuda"))
    here = torch.cuda.current_device()
    word = W._decay_status[here][0]
    for name in (None, "cuda", f"cuda:{here}", torch.device("cuda"), q.device):
        assert W.linattn_decay_status(name) == 0
        word.fill_(WKV_ERR_TIMEOUT)
        assert W.linattn_decay_status(name) == WKV_ERR_TIMEOUT, name
        assert W.linattn_decay_status(name) == 0
