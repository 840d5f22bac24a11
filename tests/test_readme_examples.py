"""The README's examples (no GPU needed): what they pass to the calls, with
stand-ins for the library's functions."""
import os
import re

import pytest
import torch

from conftest import ROOT


class Library:
    """Calls of the decayed attention: outputs of the right shapes, and every rotated tensor remembered."""

    def __init__(self):
        self.rotated = []
        self.calls = []

    def is_rotated(self, t):
        return any(t.untyped_storage().data_ptr() == r.untyped_storage().data_ptr() for r in self.rotated)

    def rotary_frequencies(self, rotated, **how):
        return torch.ones(rotated // 2, dtype=torch.float64), 1.0

    def linattn_rotary(self, q, k, positions, inv_freq, *, mscale=1.0):
        assert not self.is_rotated(q) and not self.is_rotated(k), "rotated twice"
        assert positions.shape in (q.shape[1:2], q.shape[:2])
        self.rotated += [q.clone(), k.clone()]
        self.calls.append("rotary")
        return self.rotated[-2:]

    def linattn_decay_forward(self, q, k, v, log_decay, state=None, *, scale, lengths, want_state):
        assert self.is_rotated(q) and self.is_rotated(k) and not self.is_rotated(v)
        B, T, H, D = q.shape
        self.calls.append("forward")
        return torch.zeros_like(v), torch.zeros(B, H, D, v.shape[3])

    def linattn_decay_step(self, q, k, v, log_decay, state, *, scale):
        assert self.is_rotated(q) and self.is_rotated(k) and q.dim() == v.dim() == 3
        self.calls.append("step")
        return torch.zeros_like(v), state


def test_a_prompt_and_its_next_token():
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "linattn_decay_step" in b]
    if not blocks:
        pytest.fail("no example of the decayed attention")
    for code in blocks:
        code = code.replace('"cuda"', '"cpu"').replace("T, H, D = 8, 4096, 16, 128", "T, H, D = 2, 16, 2, 8")
        lib = Library()
        names = {"torch": torch, "W": lib}
        exec(code, names)
        assert lib.calls == ["rotary", "forward", "rotary", "step"]
        token, prompt = names["v1"], names["v"]
        assert token.shape == (prompt.shape[0], 1, *prompt.shape[2:])
        assert token.untyped_storage().data_ptr() != prompt.untyped_storage().data_ptr()
