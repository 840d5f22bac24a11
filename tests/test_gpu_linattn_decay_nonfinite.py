"""Where a NaN or an infinity at one position goes, in the outputs and in every
gradient: to what depends on it, to the rest of its chunk of 128 positions on
the tensor cores, and nowhere else (other positions, heads and rows keep their
bits).
"""
import math

import pytest
import torch

import rwkv_linear_rnn_b200 as W
from test_gpu_linattn_decay import TYPES

pytestmark = pytest.mark.gpu
B, H = 2, 3
# which positions of a result depend on position p of an input
LATER, EARLIER, SAME, NONE = (lambda t, p: t >= p), (lambda t, p: t <= p), (lambda t, p: t == p), (lambda t, p: t < 0)
REACH = {  # input: (out, grad_q, grad_k, grad_v)
    "q": (SAME, NONE, EARLIER, EARLIER),
    "k": (LATER, LATER, NONE, SAME),
    "v": (LATER, LATER, SAME, NONE),
    "go": (NONE, SAME, EARLIER, EARLIER),
}


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("bad", list(REACH))
@pytest.mark.parametrize("dtype,D,M,T", [("bf16", 64, 64, 500), ("bf16", 128, 64, 3000), ("bf16", 64, 64, 30),
                                         ("f32", 64, 64, 500), ("f32", 24, 40, 3000)])
def test_reach(dtype, D, M, T, bad, value):
    torch.manual_seed(T)
    t = {n: torch.randn(B, T, H, w, device="cuda").to(TYPES[dtype]) for n, w in (("q", D), ("k", D), ("v", M), ("go", M))}
    g = torch.tensor([-0.02, -0.001, -0.3], device="cuda")
    chunk = 128 if dtype == "bf16" and T > 32 else 1

    def run():
        out, _ = W.linattn_decay_forward(t["q"], t["k"], t["v"], g)
        return [out, *W.linattn_decay_backward(t["q"], t["k"], t["v"], g, t["go"])[:3]]

    clean = run()
    for p in (0, 2 * T // 5, T - 1):
        row, head = 1, 1
        keep = t[bad][row, p, head].clone()
        t[bad][row, p, head] = value
        dirty = run()
        t[bad][row, p, head] = keep
        at = torch.arange(T, device="cuda")
        for name, reach, a, b in zip(("out", "gq", "gk", "gv"), REACH[bad], dirty, clean):
            may = reach(at, p)
            if reach is not NONE:
                assert not bool(torch.isfinite(a[row, p, head]).any()), name
                may = may | (at // chunk == p // chunk)
            same = torch.ones(B, T, H, dtype=torch.bool, device="cuda")
            same[row, :, head] = ~may
            assert torch.equal(a[same], b[same]), (name, p)
    assert W.linattn_decay_status() == 0
