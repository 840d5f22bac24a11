"""The tensor-core pass's waits: blocks that follow each other on a
multiprocessor leave nothing under way for the next one, and a wait that runs
out ends its launch with a status.
"""
import time

import pytest
import torch

import rwkv_linear_rnn_b200 as W
from rwkv_linear_rnn_b200 import abi
from rwkv_linear_rnn_b200.constants import WKV_ERR_TIMEOUT

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


def view(t):
    return abi.View(t.data_ptr(), *t.stride()[:3])


# one chunk, several; two blocks on a multiprocessor (more than 148 heads of 64, 49 for the gradients); segments
@pytest.mark.parametrize("B,T,H,D,M", [(1, 100, 2, 64, 64), (1, 500, 3, 128, 128), (1, 300, 2, 128, 64), (8, 300, 50, 64, 64),
                                       (1, 4096, 2, 64, 128)])
def test_a_wait_that_runs_out_is_reported_and_the_context_survives(B, T, H, D, M):
    """The first block holds back an arrival: its roles give up within the limit that the options name, the status
    word says so, and the next call is right."""
    q, k, v, g, go = inputs(T, B, T, H, D, M)
    ref = [*W.linattn_decay_forward(q, k, v, g, want_state=True), *W.linattn_decay_backward(q, k, v, g, go)[:3]]
    out, s = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    grads = [torch.empty_like(x) for x in ref[2:]]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    sizes = [W.linattn_decay_workspace_size(op, B, T, H, D, M, W.WKV_BF16) for op in (0, 1)]
    ws = torch.empty(max(sizes) + 256, dtype=torch.uint8, device="cuda")
    opt = abi.Options(test_hold_first_chunk=1, spin_limit=2000)

    def forward(opt):
        assert 0 == abi.linattn_decay_forward_ex(
            B, T, H, D, M, W.WKV_BF16, view(q), view(k), view(v), g.data_ptr(), 1.0, 0, 0, view(out), s.data_ptr(),
            ws.data_ptr(), sizes[0], status.data_ptr(), stream, opt)

    def backward(opt):
        assert 0 == abi.linattn_decay_backward_ex(
            B, T, H, D, M, W.WKV_BF16, view(q), view(k), view(v), g.data_ptr(), 1.0, 0, 0, view(go), 0,
            *map(view, grads), 0, ws.data_ptr(), sizes[1], status.data_ptr(), stream, opt)

    for call, got, want in ((forward, (out, s), ref[:2]), (backward, grads, ref[2:])):
        torch.cuda.synchronize()
        begin = time.perf_counter()
        call(opt)
        torch.cuda.synchronize()
        took = time.perf_counter() - begin
        assert status.item() == WKV_ERR_TIMEOUT
        assert took < 0.5  # two launches, each with waits of 2 ms
        status.zero_()
        for other in (None, abi.Options(spin_limit=100000)):
            for x in got:
                x.fill_(7.0)
            call(other)
            assert status.item() == 0
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert W.linattn_decay_status() == 0


@pytest.mark.parametrize("spin_limit", [1, 1 << 31, (1 << 63) - 1])
def test_the_smallest_and_the_largest_limit(spin_limit):
    """The largest is bounded all the same and does not wrap round to none; the smallest may give up, and says so."""
    q, k, v, g, _ = inputs(5, 1, 300, 2, 64, 64)
    ref, _ = W.linattn_decay_forward(q, k, v, g)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = W.linattn_decay_workspace_size(0, 1, 300, 2, 64, 64, W.WKV_BF16)
    ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(ref)
    assert 0 == abi.linattn_decay_forward_ex(
        1, 300, 2, 64, 64, W.WKV_BF16, view(q), view(k), view(v), g.data_ptr(), 1.0, 0, 0, view(out), 0, ws.data_ptr(), need,
        status.data_ptr(), torch.cuda.current_stream().cuda_stream, abi.Options(spin_limit=spin_limit))
    if spin_limit > 1:
        assert status.item() == 0
    assert status.item() == WKV_ERR_TIMEOUT or torch.equal(out, ref)
