"""GPU parity of the rotary positions (``linattn_rotary``) against float64.

Bounds: float32 results carry the roundings of cos, sin (2^-24 of the angle's
reduced value each, and sincospi's own few units) and of two products and a
sum, below 2^-21 of the pair's length; bfloat16 adds half a step, 2^-8 of the
value.
"""
import numpy as np
import pytest
import torch

import rwkv_linear_rnn_b200 as W
from oracle import linattn_decay as ld

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def host(t):
    return t.detach().double().cpu().numpy()


def check(got, x, positions, freq, R, dtype, mscale, interleaved, inverse):
    ref = ld.rotary(host(x), positions, freq, mscale, interleaved, inverse)
    y = host(got)
    assert y.shape == ref.shape and got.dtype == x.dtype
    np.testing.assert_array_equal(y[..., R:], host(x)[..., R:])
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    pair = np.hypot(ref[..., a], ref[..., b])
    for s in (a, b):
        bound = 2.0 ** -21 * pair + (2.0 ** -8 * np.abs(ref[..., s]) if dtype == "bf16" else 0.0)
        assert np.all(np.abs(y[..., s] - ref[..., s]) <= bound + 1e-38)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (128, 64), (64, 16), (80, 40), (96, 80), (10, 6), (3, 2), (64, 62)])
def test_layouts_and_parts_of_the_head(D, R, interleaved, dtype):
    torch.manual_seed(D + R)
    B, T, Hq, Hk = 2, 37, 3, 1
    qkv = torch.randn(B, T, Hq + Hk + 1, D, device="cuda").to(TYPES[dtype])
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    pos = torch.randint(0, 5000, (B, T), device="cuda")
    f, m = W.rotary_frequencies(R, scaling="by_parts", factor=4.0, trained_length=512)
    for inverse in (False, True):
        oq, ok = W.linattn_rotary(q, k, pos, f, mscale=m, interleaved=interleaved, inverse=inverse)
        check(oq, q, host(pos), host(f), R, dtype, m, interleaved, inverse)
        check(ok, k, host(pos), host(f), R, dtype, m, interleaved, inverse)
    keep = qkv.clone()  # in place: neighbours in the fused rows stay
    W.linattn_rotary(q, k, pos, f, mscale=m, interleaved=interleaved, out_q=q, out_k=k)
    fq, fk = W.linattn_rotary(keep[:, :, :Hq], keep[:, :, Hq:Hq + Hk], pos, f, mscale=m, interleaved=interleaved)
    assert torch.equal(q, fq) and torch.equal(k, fk) and torch.equal(qkv[:, :, -1], keep[:, :, -1])


@pytest.mark.parametrize("far", [0, 1 << 20, (1 << 40) + 12345, -(1 << 21)])
def test_far_positions(far):
    """Float32 angles would be off by whole radians from 2^20 positions on."""
    torch.manual_seed(1)
    q = torch.randn(1, 9, 2, 64, device="cuda")
    pos = far + torch.arange(9, device="cuda")
    f, _ = W.rotary_frequencies(64)
    oq, ok = W.linattn_rotary(q, None, pos, f)
    assert ok is None
    if abs(far) <= 1 << 21:  # where float64's product of the oracle is exact to 2^-31
        check(oq, q, host(pos), host(f), 64, "f32", 1.0, False, False)
    else:  # the same angles with Python's integers and a rational period
        from fractions import Fraction
        two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572")
        turns = [[float(Fraction(int(p)) * Fraction(float(w)) / two_pi % 1) for w in f.cpu()] for p in pos.cpu()]
        z = np.exp(2j * np.pi * np.array(turns))[None, :, None]
        x = host(q)
        w = (x[..., :32] + 1j * x[..., 32:]) * z
        # 2^40 positions leave float64 2^-53 2^40 radians: 1.3e-4 at most
        np.testing.assert_allclose(host(oq), np.concatenate([w.real, w.imag], -1), atol=2e-3)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (300, 1, 40, 8), (1, 4097, 2, 1), (3, 65, 12, 12)])
def test_sizes_and_position_types(B, T, Hq, Hk, dtype):
    torch.manual_seed(T)
    q = torch.randn(B, Hq, T, 64, device="cuda").to(TYPES[dtype]).transpose(1, 2)
    k = torch.randn(B, T, Hk, 64, device="cuda").to(TYPES[dtype])
    f, _ = W.rotary_frequencies(64)
    pos = torch.arange(T, device="cuda") * 3
    oq, ok = W.linattn_rotary(q, k, pos, f)
    check(oq, q, host(pos), host(f), 64, dtype, 1.0, False, False)
    check(ok, k, host(pos), host(f), 64, dtype, 1.0, False, False)
    for p in (pos.int(), pos.expand(B, T), pos.int().repeat(B, 1)):
        a, b = W.linattn_rotary(q, k, p, f)
        assert torch.equal(a, oq) and torch.equal(b, ok)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient(interleaved):
    torch.manual_seed(2)
    q, k = (torch.randn(2, 20, 3, 32, device="cuda", requires_grad=True) for _ in range(2))
    gq, gk = (torch.randn(2, 20, 3, 32, device="cuda") for _ in range(2))
    pos = torch.arange(20, device="cuda") + 1000
    f, _ = W.rotary_frequencies(24)
    oq, ok = W.rotary(q, k, pos, f, mscale=1.25, interleaved=interleaved)
    torch.autograd.backward([oq, ok], [gq, gk])
    for x, g in ((q, gq), (k, gk)):
        turned = ld.rotary(host(g)[..., :24], host(pos), host(f), 1.25, interleaved, True)
        np.testing.assert_allclose(host(x.grad)[..., :24], turned, atol=1e-5)
        np.testing.assert_array_equal(host(x.grad)[..., 24:], host(g)[..., 24:])
    # against differences: the map is linear, so a difference is exact to rounding
    d = torch.randn_like(q)
    with torch.no_grad():
        hi, lo = (W.linattn_rotary(q + s * d, None, pos, f, mscale=1.25, interleaved=interleaved)[0] for s in (1, -1))
    a = ((hi - lo).double() / 2 * gq.double()).sum()
    b = (q.grad.double() * d.double()).sum()
    assert abs(float(a - b)) <= 1e-4 * float((q.grad.double() * d.double()).abs().sum())


def test_graph_and_stream():
    torch.manual_seed(4)
    q, k = (torch.randn(4, 33, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    pos = torch.arange(33, device="cuda")
    f, _ = W.rotary_frequencies(64)
    ref = W.linattn_rotary(q, k, pos, f)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = W.linattn_rotary(q, k, pos, f)
    graph.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = W.linattn_rotary(q, k, pos, f, stream=s)
    torch.cuda.synchronize()
    for x in (got, other):
        assert torch.equal(x[0], ref[0]) and torch.equal(x[1], ref[1])


def test_refusals():
    q = torch.zeros(1, 4, 2, 32, device="cuda")
    pos = torch.arange(4, device="cuda")
    f, _ = W.rotary_frequencies(32)
    for bad in [dict(positions=pos.float()), dict(positions=pos[:3]), dict(inv_freq=f.float()),
                dict(positions=pos.cpu()), dict(k=q[..., :16]), dict(q=q[0])]:
        a = dict(q=q, k=q.clone(), positions=pos, inv_freq=f) | bad
        with pytest.raises(ValueError):
            W.linattn_rotary(a["q"], a["k"], a["positions"], a["inv_freq"])
    with pytest.raises(W.WKVError):  # more pairs than the head has
        W.linattn_rotary(q, None, pos, W.rotary_frequencies(34)[0])


def test_with_the_attention():
    """Rotary positions, a prompt in two calls, then single tokens: what the
    oracle gives for the whole row."""
    torch.manual_seed(5)
    B, T, H, D = 2, 200, 3, 64
    q, k, v = (torch.randn(B, T, H, D, device="cuda") for _ in range(3))
    g = torch.tensor([-0.02, -0.2, -0.005], device="cuda")
    f, _ = W.rotary_frequencies(D)
    pos = torch.arange(T, device="cuda")
    rq, rk = (ld.rotary(host(x), np.arange(T), host(f)) for x in (q, k))
    ref, s_ref = ld.fwd_recur(rq, rk, host(v), host(g), None, D ** -0.5)
    outs, s = [], None
    for lo, hi in ((0, 150), (150, 190)):
        a, b = W.linattn_rotary(q[:, lo:hi], k[:, lo:hi], pos[lo:hi], f)
        o, s = W.linattn_decay_forward(a, b, v[:, lo:hi], g, s, scale=D ** -0.5, want_state=True)
        outs.append(host(o))
    for t in range(190, T):
        a, b = W.linattn_rotary(q[:, t:t + 1], k[:, t:t + 1], pos[t:t + 1], f)
        o, s = W.linattn_decay_step(a[:, 0], b[:, 0], v[:, t], g, s, scale=D ** -0.5)
        outs.append(host(o)[:, None])
    got = np.concatenate(outs, 1)
    assert np.linalg.norm(got - ref) <= 1e-5 * np.linalg.norm(ref)
    assert np.linalg.norm(host(s) - s_ref) <= 1e-5 * np.linalg.norm(s_ref)
