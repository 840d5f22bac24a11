"""float64 CPU oracle for linear attention with a decay for each head and for
rotary positions (test infrastructure).

Only the test suite may import this module; the CUDA library never does and
the two share no code.  Plain numpy in float64:

* ``fwd_direct`` -- the O(T^2) definition, out_t = scale * (sum_{j<=t}
                    lam^{t-j} (q_t . k_j) v_j + lam^{t+1} q_t^T S_{-1});
* ``fwd_recur``  -- the state form S_t = lam S_{t-1} + k_t v_t^T, out_t =
                    scale * q_t^T S_t, with the state after each row's last
                    position;
* ``bwd_recur``  -- the gradients: S_t forward in time for q, its adjoint
                    W_t = scale q_t g_t^T + lam W_{t+1} in reverse for k, v and
                    the state;
* ``rotary``     -- the rotation as products of complex numbers.

Conventions: q, k [B, T, H, D], v, out [B, T, H, M], log_decay [H], state
[B, H, D, M], lengths [B]; positions from a row's length on are not read,
outputs and gradients are zero there.

Pinned by ``tests/test_oracle_linattn_decay_pins.py``.
"""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return tuple(None if x is None else np.asarray(x, dtype=np.float64) for x in xs)


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def fwd_direct(q, k, v, log_decay, state=None, scale=1.0, lengths=None):
    """O(T^2) definition; returns out."""
    q, k, v, g, state = _f64(q, k, v, log_decay, state)
    B, T, H, D = q.shape
    out = np.zeros((B, T, H, v.shape[-1]))
    for b, n in enumerate(_lengths(lengths, B, T)):
        for h in range(H):
            with np.errstate(invalid="ignore"):
                far = np.subtract.outer(np.arange(n), np.arange(n)).astype(float)
                w = np.where(far > 0, np.exp(g[h] * np.maximum(far, 1)), np.where(far == 0, 1.0, 0.0))
            o = (q[b, :n, h] @ k[b, :n, h].T * w) @ v[b, :n, h]
            if state is not None:
                o = o + np.exp(g[h] * np.arange(1, n + 1))[:, None] * (q[b, :n, h] @ state[b, h])
            out[b, :n, h] = scale * o
    return out


def fwd_recur(q, k, v, log_decay, state=None, scale=1.0, lengths=None):
    """One position at a time; returns (out, state after the last position)."""
    q, k, v, g, state = _f64(q, k, v, log_decay, state)
    B, T, H, D = q.shape
    M = v.shape[-1]
    lam = np.exp(g)[:, None, None]
    out = np.zeros((B, T, H, M))
    S = np.zeros((B, H, D, M)) if state is None else state.copy()
    for b, n in enumerate(_lengths(lengths, B, T)):
        for t in range(n):
            S[b] = lam * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            out[b, t] = scale * np.einsum("hd,hdm->hm", q[b, t], S[b])
    return out, S


def bwd_recur(q, k, v, log_decay, grad_out, state=None, scale=1.0, lengths=None, grad_state_out=None):
    """(grad_q, grad_k, grad_v, grad_state)."""
    q, k, v, g, go, state, gs = _f64(q, k, v, log_decay, grad_out, state, grad_state_out)
    B, T, H, D = q.shape
    M = v.shape[-1]
    lam = np.exp(g)[:, None, None]
    gq, gk, gv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    S = np.zeros((B, H, D, M)) if state is None else state.copy()
    G = np.zeros((B, H, D, M)) if gs is None else gs.copy()
    for b, n in enumerate(_lengths(lengths, B, T)):
        for t in range(n):
            S[b] = lam * S[b] + k[b, t][:, :, None] * v[b, t][:, None, :]
            gq[b, t] = scale * np.einsum("hdm,hm->hd", S[b], go[b, t])
        for t in reversed(range(n)):
            W = G[b] + scale * q[b, t][:, :, None] * go[b, t][:, None, :]
            gk[b, t] = np.einsum("hdm,hm->hd", W, v[b, t])
            gv[b, t] = np.einsum("hdm,hd->hm", W, k[b, t])
            G[b] = lam * W
    return gq, gk, gv, G


def step(q, k, v, log_decay, state, scale=1.0):
    """One token for N sequences: (out [N, H, M], state)."""
    out, S = fwd_recur(np.asarray(q)[:, None], np.asarray(k)[:, None], np.asarray(v)[:, None], log_decay, state, scale)
    return out[:, 0], S


def rotary(x, positions, inv_freq, mscale=1.0, interleaved=False, inverse=False):
    """x [B, T, H, D] with its first 2 len(inv_freq) elements rotated by positions [B, T] or [T]."""
    x, f = _f64(x, inv_freq)
    B, T = x.shape[:2]
    pos = np.broadcast_to(np.asarray(positions, dtype=np.float64), (B, T))
    turn = np.exp((-1j if inverse else 1j) * pos[..., None] * f)[:, :, None] * mscale
    R = 2 * f.shape[0]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = (x[..., a] + 1j * x[..., b]) * turn
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y
