"""The decayed attention's status word, whatever mode the first call runs in."""
import pytest
import torch

import rwkv_linear_rnn_b200 as W
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
