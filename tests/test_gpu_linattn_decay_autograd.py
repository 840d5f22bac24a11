"""Calls that write into given tensors, beside graphs that saved those tensors:
autograd has to hear of the writes, as it does of torch's own.
"""
import pytest
import torch

import rwkv_linear_rnn_b200 as W

pytestmark = pytest.mark.gpu
B, T, H, D = 2, 70, 2, 64


def tensors(n, *shape):
    return [torch.randn(*shape, device="cuda") for _ in range(n)]


@pytest.fixture
def graph():
    torch.manual_seed(0)
    t = dict(zip("qkv", (x.requires_grad_() for x in tensors(3, B, T, H, D))), state=tensors(1, B, H, D, D)[0],
             g=torch.tensor([-0.1, -0.01], device="cuda"))
    t["out"] = W.linattn_decay(t["q"], t["k"], t["v"], t["g"], t["state"])
    return t


def rows(n):
    return tensors(n, B, T, H, D)


def one():
    return tensors(3, B, H, D)


def rotate(q, k, **out):
    W.linattn_rotary(q, k, torch.arange(T, device="cuda"), W.rotary_frequencies(D)[0], **out)


WRITES = {
    "step in place": lambda t: W.linattn_decay_step(*one(), t["g"], t["state"]),
    "step's state_out": lambda t: W.linattn_decay_step(*one(), t["g"], t["state"].clone(), state_out=t["state"]),
    "step's out": lambda t: W.linattn_decay_step(*one(), t["g"], t["state"].clone(), out=t["v"][:, 0]),
    "forward's out": lambda t: W.linattn_decay_forward(*rows(3), t["g"], out=t["k"]),
    "backward's grad_q": lambda t: W.linattn_decay_backward(*rows(3), t["g"], *rows(1), grad_q=t["q"]),
    "backward's grad_k": lambda t: W.linattn_decay_backward(*rows(3), t["g"], *rows(1), grad_k=t["q"]),
    "backward's grad_v": lambda t: W.linattn_decay_backward(*rows(3), t["g"], *rows(1), grad_v=t["v"]),
    "rotary in place": lambda t: rotate(t["q"], t["k"].clone(), out_q=t["q"]),
    "rotary's out_k": lambda t: rotate(*rows(2), out_k=t["k"]),
}


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
@pytest.mark.parametrize("write", WRITES)
def test_a_write_into_a_saved_tensor_is_an_error_in_backward(graph, write, mode):
    with mode():
        WRITES[write](graph)
    with pytest.raises(RuntimeError, match="inplace operation"):
        graph["out"].sum().backward()


def test_writes_elsewhere_leave_the_graph_alone(graph):
    with torch.no_grad():
        x, k, v = tensors(3, B, H, D)
        y, s = W.linattn_decay_step(x, k, v, graph["g"], graph["state"].clone())
        W.linattn_decay_forward(graph["q"], graph["k"], graph["v"], graph["g"], graph["state"], want_state=True)
        W.linattn_decay_step(x, k, v, graph["g"], graph["state"], state_out=torch.empty_like(s))
    graph["out"].sum().backward()
    want = W.linattn_decay_backward(graph["q"].detach(), graph["k"].detach(), graph["v"].detach(), graph["g"],
                                    torch.ones_like(graph["out"]), graph["state"])
    assert all(torch.equal(graph[n].grad, w) for n, w in zip("qkv", want))


def test_evaluating_with_a_decay_parameter(graph):
    decay = torch.nn.Parameter(graph["g"].clone())
    with torch.no_grad():
        out = W.linattn_decay(graph["q"], graph["k"], graph["v"], decay, graph["state"])
    assert torch.equal(out, graph["out"].detach())


@pytest.mark.parametrize("D,M", [(3, 5), (7, 1), (64, 64)])
def test_states_that_are_slices_off_16_bytes(D, M):
    """States of odd sizes cut from a larger tensor, and their gradients cut from a larger one by cat's backward."""
    q, k = (x.requires_grad_() for x in tensors(2, 1, 9, 1, D))
    v = torch.randn(1, 9, 1, M, device="cuda", requires_grad=True)
    g = torch.tensor([-0.1], device="cuda")
    pool = torch.randn(3, 1, D, M, device="cuda", requires_grad=True)
    weight = torch.randn(2, 1, D, M, device="cuda")

    def loss(state):
        outs = [W.linattn_decay_state(q, k, v, g, state(i)) for i in (1, 2)]
        s = torch.cat([s for _, s in outs])
        return sum(o.sum() for o, _ in outs) + (s * weight).sum()

    def grads(state):
        for t in (q, k, v, pool):
            t.grad = None
        loss(state).backward()
        return [t.grad.clone() for t in (q, k, v, pool)]

    for a, b in zip(grads(lambda i: pool[i:i + 1]), grads(lambda i: pool[i:i + 1].clone())):
        assert torch.equal(a, b) and bool(a.abs().sum() > 0)
