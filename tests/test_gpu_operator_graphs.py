"""Every operator on a stream of its own and captured into a CUDA graph gives the bits of a plain
call, with the inputs that are there when the graph is replayed."""
import pytest
import torch

import dtensor_reshard_gb300 as rs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    yield
    assert rs.reshard_device_status(clear=True) == 0


def _quantize(block_rows):
    x = torch.randn(300, 700, device="cuda")
    q = torch.empty(300, 700, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-300 // block_rows), 6, device="cuda")
    return x, (q, s), lambda st: rs.reshard_fp8_quantize(x, q, s, (300, 700), "fp32", block_rows, stream=st)


def _matmul(tokens, n, k):
    x = torch.randint(0, 127, (tokens, k), dtype=torch.uint8, device="cuda")
    w = torch.randint(0, 127, (n, k), dtype=torch.uint8, device="cuda")
    xs, ws = torch.rand(tokens, k // 128, device="cuda"), torch.rand(-(-n // 128), k // 128, device="cuda")
    y = torch.empty(tokens, n, device="cuda")
    return xs, (y,), lambda st: rs.reshard_fp8_matmul(x, xs, w, ws, y, (tokens, n, k), "fp32", stream=st)


def _sample(rows, vocab):
    x = torch.randn(rows, vocab, device="cuda") * 3
    u, p = torch.rand(rows, device="cuda"), torch.full((rows,), 0.9, device="cuda")
    k = torch.arange(rows, device="cuda", dtype=torch.int32) * 7
    token, logprob = torch.empty(rows, dtype=torch.int32, device="cuda"), torch.empty(rows, device="cuda")
    return x, (token, logprob), lambda st: rs.reshard_sample(x, (rows, vocab), "fp32", u, token, logprob,
                                                            top_k=k, top_p=p, stream=st)


def _balance(nseq, seqlen, experts):
    shape = (nseq, seqlen, experts)
    x = torch.randn(shape, device="cuda")
    choices = x.topk(2, dim=2).indices.to(torch.int32)
    workspace = torch.empty(rs.reshard_balance_loss_workspace(shape), dtype=torch.uint8, device="cuda")
    counts = torch.empty(nseq, experts, dtype=torch.int32, device="cuda")
    loss, grad = torch.empty(1, device="cuda"), torch.empty_like(x)
    return x, (counts, loss, grad), lambda st: rs.reshard_balance_loss(
        x, shape, "fp32", choices, 2, 0.1, workspace, counts, loss=loss, dlogits=grad, stream=st)


CASES = {
    "quantize 1x128": lambda: _quantize(1), "quantize 128x128": lambda: _quantize(128),
    "product of one token": lambda: _matmul(1, 1000, 2048), "product of some": lambda: _matmul(40, 1000, 2048),
    "product of many": lambda: _matmul(700, 5001, 2048), "product with k shared": lambda: _matmul(128, 3333, 2816),
    "sample": lambda: _sample(5, 3000), "sample a batch": lambda: _sample(200, 9001),
    "balance, one launch": lambda: _balance(2, 30, 9), "balance": lambda: _balance(3, 500, 64),
    "balance, counts by clusters": lambda: _balance(1, 40000, 16),
    "balance, many sequences": lambda: _balance(3000, 2, 16), "balance, many experts": lambda: _balance(1, 300, 1500),
}


@pytest.mark.parametrize("name", CASES)
def test_on_a_stream_and_in_a_graph(name):
    torch.manual_seed(5)
    changing, outputs, call = CASES[name]()

    def bits():
        torch.cuda.synchronize()
        return [o.clone().view(torch.uint8) for o in outputs]

    def spoil():
        for o in outputs:
            o.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()
    call(None)
    want = bits()
    spoil()
    side = torch.cuda.Stream()
    call(side)
    assert all(torch.equal(a, b) for a, b in zip(bits(), want))
    spoil()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(side)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(bits(), want))
        spoil()
    changing.mul_(1.25)                      # other inputs, in the same place
    call(None)
    want = bits()
    spoil()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(bits(), want))
