"""Rotary positions up to the magnitude of 2^53 that ``linattn_rotary`` takes,
against rational arithmetic.

Bound: the reduced angle is rounded to float32 once, at most half a step of
half a turn (2 pi 2^-26 radians); sincospi adds at most 2 units of 2^-24, the
two products and their sum 3 of 2^-24: below 2^-21 of the pair's length.  The
float64 arithmetic before the rounding has to lose far less than 2^-26 of a
turn, however many turns there are.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

import rwkv_linear_rnn_b200 as W

pytestmark = pytest.mark.gpu
TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572")


def turned(x, positions, freq):
    """x [1, T, H, 2 n] float64 with its halves turned, from exact turns."""
    n = len(freq)
    turns = [[float(Fraction(p) * Fraction(w) / TWO_PI % 1) for w in freq] for p in positions]
    z = (x[..., :n] + 1j * x[..., n:]) * np.exp(2j * np.pi * np.array(turns))[None, :, None]
    return z


@pytest.mark.parametrize("first", [0, (1 << 30) + 77, 1 << 32, (1 << 36) + 1, (1 << 40) + 12345, (1 << 47) - 3,
                                   (1 << 53) - 8, -(1 << 32) - 5, -(1 << 53)])
@pytest.mark.parametrize("freq", ["usual", "unusual"])
def test_angles_of_far_positions(first, freq):
    torch.manual_seed(first % 1000)
    q = torch.randn(1, 9, 2, 64, device="cuda")
    if freq == "usual":
        f, _ = W.rotary_frequencies(64)
    else:  # up to many turns a position, and down to a turn in 2^40
        f = torch.logspace(3, -12, 32, dtype=torch.float64, device="cuda")
    pos = first + torch.arange(9, device="cuda")
    assert int(pos[0]) == first and int(pos.abs().max()) <= 1 << 53
    out, _ = W.linattn_rotary(q, None, pos, f)
    z = turned(q.double().cpu().numpy(), pos.tolist(), f.tolist())
    y = out.double().cpu().numpy()
    got = y[..., :32] + 1j * y[..., 32:]
    assert np.all(np.abs(got - z) <= 2.0 ** -21 * np.sqrt(2) * np.abs(z))


def test_inverse_undoes_a_far_turn():
    """Both ways take the same angle: back within the two calls' roundings."""
    q = torch.randn(1, 5, 1, 32, device="cuda")
    pos = (1 << 52) + 12345 + torch.arange(5, device="cuda")
    f, _ = W.rotary_frequencies(32)
    out, _ = W.linattn_rotary(q, None, pos, f)
    back, _ = W.linattn_rotary(out, None, pos, f, inverse=True)
    pair = torch.hypot(q[..., :16], q[..., 16:]).repeat(1, 1, 1, 2)
    assert bool(((back - q).abs() <= 2.0 ** -20 * pair).all())
