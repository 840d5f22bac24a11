"""The tensor-core pass's waits: blocks that follow each other on a
multiprocessor leave nothing under way for the next one.
"""
import pytest
import torch

import rwkv_linear_rnn_b200 as W

pytestmark = pytest.mark.gpu


def inputs(seed, B, T, H, D, M):
    torch.manual_seed(seed)
    q, k = (torch.randn(B, T, H, D, device="cuda").bfloat16() for _ in range(2))
    v, go = (torch.randn(B, T, H, M, device="cuda").bfloat16() for _ in range(2))
    return q, k, v, -torch.rand(H, device="cuda"), go


@pytest.mark.parametrize("D,M", [(64, 64), (128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("BH", [(1, 100), (8, 100)])
def test_blocks_one_after_another(BH, D, M):
    """Many short blocks on each multiprocessor, call after call: the same bits each time, and no wait that gives up."""
    B, H = BH
    q, k, v, g, go = inputs(D + M, B, 140, H, D, M)
    n = torch.randint(0, 141, (B,), device="cuda", dtype=torch.int32)

    def calls():
        out, s = W.linattn_decay_forward(q, k, v, g, lengths=n, want_state=True)
        return [out, s, *W.linattn_decay_backward(q, k, v, g, go, lengths=n, want_grad_state=True)]

    ref = calls()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            got = calls()
    for _ in range(25):
        graph.replay()
    assert W.linattn_decay_status() == 0
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
