"""Host-side checks of linear attention with a decay for each head and of
rotary positions (no GPU needed): calls that are refused before any launch,
workspace sizes, and the frequency plans."""
import math

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def W():
    from rwkv_linear_rnn_b200.build import build_library
    build_library()
    import rwkv_linear_rnn_b200
    return rwkv_linear_rnn_b200


F = 1 << 20  # an aligned non-null address; refusals come before any use
INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3


def view(W, n, b=8 * 2 * 32, t=2 * 32, h=32):
    return W.abi.View(F * n, b, t, h)


def forward(W, B=1, T=8, H=2, D=32, M=32, dtype=0, q=None, k=None, v=None, g=F, lengths=0, s_in=0, out=None, s_out=0,
            ws=F * 99, ws_bytes=1 << 40, status=0, null=()):
    a = dict(q=q or view(W, 1), k=k or view(W, 2), v=v or view(W, 3), out=out or view(W, 4))
    a.update({n: None for n in null})
    return W.abi.linattn_decay_forward(B, T, H, D, M, dtype, a["q"], a["k"], a["v"], g, 1.0, lengths, s_in, a["out"],
                                       s_out, ws, ws_bytes, status, 0)


def test_forward_refusals(W):
    V = lambda **x: W.abi.View(*[x.get(n, d) for n, d in (("ptr", F), ("b", 512), ("t", 64), ("h", 32))])  # noqa: E731
    for kw, code in [
        (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
        (dict(B=1 << 23, H=2), INVALID), (dict(D=0), INVALID), (dict(M=0), INVALID), (dict(dtype=2), INVALID),
        (dict(D=129), UNSUPPORTED), (dict(M=256), UNSUPPORTED), (dict(g=0), INVALID),
        (dict(null=("q",)), INVALID), (dict(null=("out",)), INVALID), (dict(q=V(ptr=0)), INVALID),
        (dict(k=V(ptr=F * 2 + 2)), UNSUPPORTED),                 # off the element size
        (dict(v=V(ptr=F * 3, t=-64)), INVALID),                  # negative stride
        (dict(out=V(ptr=F * 4, t=0)), INVALID),                  # an output that overlaps itself
        (dict(out=V(ptr=F * 4, h=16)), INVALID),
        (dict(out=V(ptr=F * 4, b=100), B=2), INVALID),
        (dict(out=V(ptr=F)), INVALID),                           # out is q
        (dict(s_in=F * 5 + 4), UNSUPPORTED), (dict(s_out=F * 5 + 8), UNSUPPORTED),
        (dict(s_in=F * 5, s_out=F * 5 + 64), UNSUPPORTED),       # partly overlapping states
        (dict(lengths=F + 2), UNSUPPORTED), (dict(status=F + 1), UNSUPPORTED),
        (dict(T=4096, ws=0), WORKSPACE), (dict(T=4096, ws_bytes=16), WORKSPACE), (dict(T=4096, ws=F + 16), WORKSPACE),
    ]:
        assert forward(W, **kw) == code, kw
    assert forward(W, T=0, null=("q", "k", "v", "out")) == 0     # nothing to do


def test_backward_refusals(W):
    def call(**kw):
        a = dict(q=1, k=2, v=3, go=4, gq=5, gk=6, gv=7)
        for n in a:
            a[n] = kw.get(n, view(W, a[n]))
        return W.abi.linattn_decay_backward(
            kw.get("B", 1), kw.get("T", 8), 2, kw.get("D", 32), 32, kw.get("dtype", 0), a["q"], a["k"], a["v"],
            kw.get("g", F), 1.0, 0, kw.get("s_in", 0), a["go"], kw.get("gso", 0), a["gq"], a["gk"], a["gv"],
            kw.get("gs", 0), kw.get("ws", F * 99), 1 << 40, 0, 0)

    for kw, code in [
        (dict(B=0), INVALID), (dict(dtype=7), INVALID), (dict(D=200), UNSUPPORTED), (dict(g=0), INVALID),
        (dict(go=None), INVALID), (dict(gk=None), INVALID), (dict(gq=view(W, 4)), INVALID),
        (dict(gv=view(W, 6)), INVALID), (dict(gq=view(W, 7)), INVALID), (dict(gk=view(W, 6, t=0)), INVALID),
        (dict(gs=F * 8 + 4), UNSUPPORTED), (dict(gs=F * 8, s_in=F * 8), UNSUPPORTED),
        (dict(gs=F * 8, gso=F * 8 + 32), UNSUPPORTED), (dict(T=4096, ws=0), WORKSPACE),
    ]:
        assert call(**kw) == code, kw


def test_step_refusals(W):
    def call(N=4, H=2, D=32, M=32, dtype=0, g=F, s_in=F * 5, s_out=F * 5, **kw):
        a = [kw.get(n, view(W, i + 1)) for i, n in enumerate(("q", "k", "v", "out"))]
        return W.abi.linattn_decay_step(N, H, D, M, dtype, a[0], a[1], a[2], g, 1.0, s_in, a[3], s_out, 0)

    for kw, code in [
        (dict(N=0), INVALID), (dict(H=0), INVALID), (dict(N=1 << 30, H=2), INVALID), (dict(D=0), INVALID),
        (dict(dtype=5), INVALID), (dict(D=129), UNSUPPORTED), (dict(g=0), INVALID), (dict(s_in=0), INVALID),
        (dict(s_out=0), INVALID), (dict(q=None), INVALID), (dict(out=view(W, 1)), INVALID),
        (dict(out=view(W, 4, h=0)), INVALID), (dict(s_in=F * 5 + 4), UNSUPPORTED),
        (dict(s_out=F * 5 + 1024), UNSUPPORTED),
    ]:
        assert call(**kw) == code, kw


def test_rotary_refusals(W):
    def call(B=1, T=4, D=32, R=16, dtype=0, Hq=2, Hk=2, pos=F * 7, pb=8, ps=0, f=F * 8, inter=0, **kw):
        a = {n: kw.get(n, view(W, i + 1)) for i, n in enumerate(("q", "k", "oq", "ok"))}
        return W.abi.linattn_rotary(B, T, D, R, dtype, Hq, a["q"], Hk, a["k"], pos, pb, ps, f, 1.0, inter, 0, a["oq"],
                                    a["ok"], 0)

    for kw, code in [
        (dict(B=0), INVALID), (dict(T=-1), INVALID), (dict(R=15), INVALID), (dict(R=0), INVALID), (dict(R=34), INVALID),
        (dict(D=1025, R=2), INVALID), (dict(dtype=3), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID),
        (dict(k=None), INVALID), (dict(ok=None), INVALID), (dict(pb=2), INVALID), (dict(ps=-1), INVALID),
        (dict(pos=0), INVALID), (dict(f=0), INVALID), (dict(pos=F + 4), UNSUPPORTED), (dict(f=F + 4), UNSUPPORTED),
        (dict(q=W.abi.View(F + 2, 512, 64, 32)), UNSUPPORTED),
        (dict(oq=W.abi.View(F, 1024, 64, 32)), INVALID),         # in place with other strides
        (dict(oq=view(W, 2)), INVALID), (dict(ok=view(W, 3)), INVALID), (dict(oq=view(W, 3, t=32)), INVALID),
    ]:
        assert call(**kw) == code, kw
    assert call(T=0) == 0


def test_workspace_sizes(W):
    size = W.linattn_decay_workspace_size
    assert size(0, 1, 8, 2, 32, 32, 0) == 0                      # one segment per head: no states to keep
    n = size(0, 1, 65536, 2, 64, 64, 0)                          # two heads, long: cut into segments
    assert n > 0 and n % (2 * 64 * 64 * 4) == 0
    assert size(1, 1, 65536, 2, 64, 64, 0) >= n
    for bad in [(2, 1, 8, 2, 32, 32, 0), (0, 0, 8, 2, 32, 32, 0), (0, 1, -1, 2, 32, 32, 0), (0, 1, 8, 2, 129, 32, 0),
                (0, 1, 8, 2, 32, 32, 2)]:
        assert size(*bad) == 0


def test_frequency_plans(W):
    plain, m = W.rotary_frequencies(64, device="cpu")
    assert m == 1.0 and plain.dtype == torch.float64
    np.testing.assert_allclose(plain.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    lin, _ = W.rotary_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    np.testing.assert_allclose(lin, plain / 4, rtol=1e-14)
    ntk, _ = W.rotary_frequencies(64, scaling="ntk", factor=4.0, device="cpu")
    np.testing.assert_allclose([ntk[0], ntk[-1]], [1.0, plain[-1] / 4], rtol=1e-12)
    parts, m = W.rotary_frequencies(64, scaling="by_parts", factor=4.0, trained_length=4096, device="cpu")
    assert m == pytest.approx(0.1 * math.log(4.0) + 1)
    turns = 4096 * plain / (2 * math.pi)
    assert torch.equal(parts[turns > 32], plain[turns > 32])
    np.testing.assert_allclose(parts[turns < 1], plain[turns < 1] / 4, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert bool(((parts < plain) & (parts > plain / 4))[mid].all())
    for bad in [dict(rotated=5), dict(rotated=0), dict(rotated=8, scaling="other"), dict(rotated=8, factor=0.0),
                dict(rotated=8, scaling="by_parts", factor=2.0)]:
        with pytest.raises(ValueError):
            W.rotary_frequencies(bad.pop("rotated"), device="cpu", **bad)


def test_wrappers_refuse_before_the_library(W):
    z = lambda *s: torch.zeros(s)  # noqa: E731
    with pytest.raises(ValueError, match="constant"):
        W.linattn_decay(z(1, 2, 1, 4), z(1, 2, 1, 4), z(1, 2, 1, 4), z(1).requires_grad_())
