"""What the differentiable forms refuse (no GPU needed)."""
import pytest
import torch

from test_linattn_decay_host import W  # noqa: F401  (the fixture)


def test_a_decay_parameter_is_refused_only_where_gradients_are_recorded(W):  # noqa: F811
    """log_decay has no gradient, so asking for one is an error; a module that holds it as a parameter
    can still be evaluated.  (On the CPU that gets as far as the device check.)"""
    q = torch.zeros(1, 2, 1, 4)
    g = torch.zeros(1, requires_grad=True)
    for call in (W.linattn_decay, W.linattn_decay_state):
        with pytest.raises(ValueError, match="constant"):
            call(q, q, q, g)
        with torch.enable_grad(), pytest.raises(ValueError, match="constant"):
            call(q, q, q, g)
        for off in (torch.no_grad, torch.inference_mode):
            with off(), pytest.raises(ValueError, match="CUDA device"):
                call(q, q, q, g)
        with pytest.raises(ValueError, match="CUDA device"):
            call(q, q, q, g.detach())


def test_frequencies_that_ask_for_a_gradient_are_refused(W):  # noqa: F811
    """The rotation's frequencies are constants too: no silent missing gradient."""
    q = torch.zeros(1, 2, 1, 4, requires_grad=True)
    f = torch.ones(2, dtype=torch.float64, requires_grad=True)
    pos = torch.arange(2)
    with pytest.raises(ValueError, match="constant"):
        W.rotary(q, None, pos, f)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):
        W.rotary(q, None, pos, f)
    with pytest.raises(ValueError, match="CUDA device"):
        W.rotary(q, None, pos, f.detach())
