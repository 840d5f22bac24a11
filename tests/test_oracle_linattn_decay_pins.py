"""Pins for the oracle of linear attention with a decay for each head and of
rotary positions (``oracle.linattn_decay``): the recurrence against the direct
sum, gradients against finite differences and against autograd of the direct
form, states carried across a split, limits, and the rotation's identities."""
import numpy as np
import pytest
import torch

from oracle import linattn_decay as ld


def case(seed, B=2, T=7, H=3, D=4, M=5, lengths=False):
    rng = np.random.default_rng(seed)
    q, k = rng.normal(size=(2, B, T, H, D))
    v, g = rng.normal(size=(2, B, T, H, M))
    decay = -rng.uniform(0.01, 1.5, H)
    s, gs = rng.normal(size=(2, B, H, D, M))
    n = rng.integers(0, T + 1, B) if lengths else None
    return q, k, v, decay, g, s, gs, n


@pytest.mark.parametrize("lengths", [False, True])
@pytest.mark.parametrize("with_state", [False, True])
def test_recurrence_equals_direct_sum(lengths, with_state):
    q, k, v, decay, _, s, _, n = case(1, lengths=lengths)
    s = s if with_state else None
    out, _ = ld.fwd_recur(q, k, v, decay, s, 0.3, n)
    np.testing.assert_allclose(out, ld.fwd_direct(q, k, v, decay, s, 0.3, n), rtol=1e-12, atol=1e-13)


def test_limits():
    q, k, v, _, _, s, _, _ = case(2)
    # lam = 0: a position sees itself alone
    out, last = ld.fwd_recur(q, k, v, np.full(3, -np.inf), s)
    np.testing.assert_allclose(out, np.einsum("bthd,bthd->bth", q, k)[..., None] * v, rtol=1e-12)
    np.testing.assert_allclose(last, k[:, -1][..., None] * v[:, -1][..., None, :], rtol=1e-12)
    # lam = 1: plain cumulative sums
    out, last = ld.fwd_recur(q, k, v, np.zeros(3))
    np.testing.assert_allclose(last, np.einsum("bthd,bthm->bhdm", k, v), rtol=1e-12)


def test_split_sequence_carries_the_state():
    q, k, v, decay, _, s, _, _ = case(3)
    whole, last = ld.fwd_recur(q, k, v, decay, s)
    a, mid = ld.fwd_recur(q[:, :3], k[:, :3], v[:, :3], decay, s)
    b, end = ld.fwd_recur(q[:, 3:], k[:, 3:], v[:, 3:], decay, mid)
    np.testing.assert_allclose(np.concatenate([a, b], 1), whole, rtol=1e-12)
    np.testing.assert_allclose(end, last, rtol=1e-12)
    y, nxt = ld.step(q[:, 0], k[:, 0], v[:, 0], decay, s)
    np.testing.assert_allclose(y, whole[:, 0], rtol=1e-12)


@pytest.mark.parametrize("lengths", [False, True])
def test_gradients_match_finite_differences(lengths):
    q, k, v, decay, g, s, gs, n = case(4, B=2, T=4, H=2, D=3, M=2, lengths=lengths)

    def loss(q, k, v, s):
        out, last = ld.fwd_recur(q, k, v, decay, s, 0.7, n)
        return np.sum(out * g) + np.sum(last * gs)

    grads = ld.bwd_recur(q, k, v, decay, g, s, 0.7, n, gs)
    args = [q, k, v, s]
    for i, got in enumerate(grads):
        num = np.zeros_like(args[i])
        for at in np.ndindex(args[i].shape):
            d = np.zeros_like(args[i])
            d[at] = 1e-5
            hi, lo = (loss(*[x + sgn * d if j == i else x for j, x in enumerate(args)]) for sgn in (1, -1))
            num[at] = (hi - lo) / 2e-5
        np.testing.assert_allclose(got, num, rtol=1e-6, atol=1e-8)


def test_gradients_match_autograd_of_the_direct_form():
    q, k, v, decay, g, s, _, _ = case(5)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    t = torch.arange(7)
    far = (t[:, None] - t).clamp(min=0)
    w = torch.where(t[:, None] >= t, torch.exp(torch.tensor(decay)[:, None, None] * far), 0.0)
    out = torch.einsum("bihd,bjhd,hij,bjhm->bihm", tq, tk, w, tv)
    out.backward(torch.tensor(g))
    for got, ref in zip(ld.bwd_recur(q, k, v, decay, g), (tq.grad, tk.grad, tv.grad)):
        np.testing.assert_allclose(got, ref.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_identities(interleaved):
    rng = np.random.default_rng(6)
    x, y = rng.normal(size=(2, 2, 5, 3, 10))
    f = 10.0 ** -np.arange(4.0)
    how = dict(interleaved=interleaved)
    p = np.arange(5)
    # part of the head: the rest passes; lengths are kept; the inverse undoes it
    r = ld.rotary(x, p, f, **how)
    np.testing.assert_array_equal(r[..., 8:], x[..., 8:])
    np.testing.assert_allclose(np.sum(r * r, -1), np.sum(x * x, -1), rtol=1e-12)
    np.testing.assert_allclose(ld.rotary(r, p, f, inverse=True, **how), x, rtol=1e-11, atol=1e-12)
    # products depend on the distance alone
    a = np.sum(ld.rotary(x, p, f, **how) * ld.rotary(y, p + 3, f, **how), -1)
    b = np.sum(ld.rotary(x, p + 100, f, **how) * ld.rotary(y, p + 103, f, **how), -1)
    np.testing.assert_allclose(a, b, rtol=1e-9, atol=1e-10)
    # <rot(x), y> = <x, rot^-1(y)> over the rotated part: the inverse is the gradient
    lhs = np.sum((ld.rotary(x, p, f, 1.5, **how) * y)[..., :8])
    np.testing.assert_allclose(lhs, np.sum((x * ld.rotary(y, p, f, 1.5, inverse=True, **how))[..., :8]), rtol=1e-10)


def test_rotation_of_one_pair():
    x = np.array([1.0, 2.0, 3.0, 4.0]).reshape(1, 1, 1, 4)
    c, s = np.cos(0.5 * 7), np.sin(0.5 * 7)
    np.testing.assert_allclose(ld.rotary(x, [7], [0.5], interleaved=True).ravel(), [c - 2 * s, s + 2 * c, 3, 4])
    c2, s2 = np.cos(0.1 * 7), np.sin(0.1 * 7)
    np.testing.assert_allclose(ld.rotary(x, [7], [0.5, 0.1]).ravel(),
                               [c - 3 * s, 2 * c2 - 4 * s2, s + 3 * c, 2 * s2 + 4 * c2])
