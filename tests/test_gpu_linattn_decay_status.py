"""The decayed attention's status word, whatever mode the first call runs in."""
import subprocess
import sys

import pytest
import torch

import rwkv_linear_rnn_b200 as W
from conftest import ROOT
from rwkv_linear_rnn_b200.constants import WKV_ERR_TIMEOUT

pytestmark = pytest.mark.gpu


@pytest.fixture
def fresh(monkeypatch):
    """As if no call had been made yet."""
    monkeypatch.setattr(W, "_decay_status", {})


def a_call():
    q = torch.randn(1, 40, 2, 64, device="cuda").bfloat16()
    return W.linattn_decay_forward(q, q, q, torch.zeros(2, device="cuda"))


@pytest.mark.parametrize("mode", [torch.inference_mode, torch.no_grad, torch.enable_grad])
def test_first_call_under_any_mode(fresh, mode):
    with mode():
        a_call()
    assert W.linattn_decay_status() == 0
    word = W._decay_status[torch.cuda.current_device()][0]
    for read_in in (torch.inference_mode, torch.enable_grad):
        word.fill_(WKV_ERR_TIMEOUT)
        with read_in():
            assert W.linattn_decay_status() == WKV_ERR_TIMEOUT
        assert W.linattn_decay_status() == 0


CAPTURED_FIRST = """
import torch
import rwkv_linear_rnn_b200 as W
from rwkv_linear_rnn_b200 import abi

given = []
call = abi.linattn_decay_forward_at


def spy(*args):
    given.append(args[-2])
    return call(*args)


abi.linattn_decay_forward_at = spy
q = torch.randn(1, 300, 2, 64, device="cuda").bfloat16()
g = torch.tensor([-0.1, -0.01], device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out, _ = W.linattn_decay_forward(q, q, q, g)
graph.replay()
assert given[0] != 0, "captured without a status word"
assert W.linattn_decay_status() == 0
word = W._decay_status[torch.cuda.current_device()][0]
assert word.data_ptr() == given[0]
word.fill_(-5)
assert W.linattn_decay_status() == -5 and W.linattn_decay_status() == 0
again, _ = W.linattn_decay_forward(q, q, q, g)
assert given[1] == given[0] and torch.equal(out, again)
print("captured first")
"""


def test_a_process_whose_first_call_is_captured():
    run = subprocess.run([sys.executable, "-c", CAPTURED_FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "captured first" in run.stdout, run.stdout + run.stderr
