"""The operators that train and score on streams of their own, captured into CUDA graphs, from several
host threads and one behind another, give the bits of plain calls, with the inputs that are there when
a graph is replayed."""
import threading

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


def _score(rows, vocab, ntop, dtype=torch.float32, name="fp32"):
    x = (torch.randn(rows, vocab, device="cuda") * 3).to(dtype)
    target = torch.randint(-1, vocab, (rows,), device="cuda", dtype=torch.int32)
    t = torch.rand(rows, device="cuda") + 0.5
    lp, h = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    state = torch.empty(rows, 4, device="cuda")
    token = torch.empty(rows, ntop, dtype=torch.int32, device="cuda")
    top = torch.empty(rows, ntop, device="cuda")
    call = lambda st: rs.reshard_logprob(  # noqa: E731
        x, (rows, vocab), name, target=target, logprob=lp, entropy=h, state=state, top_token=token, top_logprob=top,
        ntop=ntop, temperature=t, stream=st)
    call.target, call.temperature = target, t
    return x, (lp, h, state, token, top), call


def _policy(rows, vocab):
    """Scores and their gradient, one call behind the other."""
    x, outs, score = _score(rows, vocab, 0, torch.bfloat16, "bf16")
    target, temperature = score.target, score.temperature
    grad, g, h = torch.empty_like(x), torch.randn(rows, device="cuda"), torch.randn(rows, device="cuda")

    def call(st):
        score(st)
        rs.reshard_logprob_grad(x, (rows, vocab), "bf16", outs[2], grad, target=target, dlogprob=g, dentropy=h,
                                temperature=temperature, stream=st)
    return x, (*outs[:3], grad), call


def _distill(rows, vocab, k, tail):
    x = torch.randn(rows, vocab, device="cuda") * 3
    y = torch.log_softmax(torch.randn(rows, vocab, device="cuda") * 3, 1).topk(k, dim=1)
    token, value = y.indices.to(torch.int32), y.values.contiguous()
    loss, grad = torch.empty(rows, device="cuda"), torch.empty_like(x)
    return x, (loss, grad), lambda st: rs.reshard_distill_loss(x, (rows, vocab), "fp32", token, value, k, loss=loss,
                                                               dlogits=grad, tail=tail, stream=st)


def _layer(tokens, topk, cols, nexperts, quantised):
    """Sorted, dispatched, combined, and both gradients: what a layer's step runs in turn."""
    x = torch.randn(tokens, cols, device="cuda")
    experts = torch.rand(tokens, nexperts, device="cuda").topk(topk, dim=1).indices.to(torch.int32)
    n = tokens * topk
    slot, offsets = torch.empty_like(experts), torch.empty(nexperts + 1, dtype=torch.int32, device="cuda")
    rows = torch.zeros(n, cols, dtype=torch.uint8 if quantised else torch.float32, device="cuda")
    scale = torch.zeros(n, -(-cols // 128), device="cuda") if quantised else None
    back = torch.randn(n, cols, device="cuda")
    w, out = torch.rand(tokens, topk, device="cuda"), torch.empty_like(x)
    drows, dw, dx = torch.empty_like(back), torch.empty_like(w), torch.empty_like(x)
    shape = (tokens, topk, cols)

    def call(st):
        rs.reshard_expert_sort(experts, (tokens, topk), nexperts, slot, offsets, stream=st)
        rs.reshard_expert_dispatch(x, shape, "fp32", slot, rows, scale=scale, stream=st)
        rs.reshard_expert_combine(back, shape, "fp32", slot, out, weight=w, stream=st)
        rs.reshard_expert_combine_grad(x, shape, "fp32", slot, rows=back, weight=w, drows=drows, dweight=dw, stream=st)
        rs.reshard_expert_combine(drows, shape, "fp32", slot, dx, stream=st)
    outs = [slot, offsets, rows, out, drows, dw, dx] + ([scale] if quantised else [])
    return x, tuple(outs), call


CASES = {
    "score a row": lambda: _score(1, 50000, 20), "score rows": lambda: _score(300, 4001, 7),
    "score with many alternatives": lambda: _score(5, 9001, 200), "policy": lambda: _policy(90, 7001),
    "policy of a row": lambda: _policy(1, 70001), "distill": lambda: _distill(200, 5001, 30, False),
    "distill with the rest": lambda: _distill(3, 50001, 256, True), "layer of a token": lambda: _layer(1, 2, 300, 8, False),
    "layer": lambda: _layer(700, 4, 1024, 60, False), "layer in 8 bits": lambda: _layer(3000, 8, 256, 300, True),
}


@pytest.mark.parametrize("name", CASES)
def test_on_a_stream_and_in_a_graph(name):
    torch.manual_seed(6)
    changing, outputs, call = CASES[name]()

    def bits():
        torch.cuda.synchronize()
        return [o.clone().view(torch.uint8) for o in outputs]

    def spoil():
        for o in outputs:
            o.view(torch.uint8).fill_(0x5A)
        torch.cuda.synchronize()

    def same(want):
        return all(torch.equal(a, b) for a, b in zip(bits(), want))
    call(None)
    want = bits()
    spoil()
    side = torch.cuda.Stream()
    call(side)
    assert same(want)
    spoil()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(side)
        call(side)                           # behind itself, with nothing between
    for _ in range(2):
        graph.replay()
        graph.replay()
        assert same(want)
        spoil()
    changing.mul_(1.25)                      # other inputs, in the same place
    call(None)
    want = bits()
    spoil()
    graph.replay()
    assert same(want)


def test_what_a_kernel_writes_is_there_for_the_next_that_starts_early():
    """Kernels may start while the one in front of them ends: chains in which each reads what the one
    before has just written, many times over, with other streams at work."""
    torch.manual_seed(7)
    t, k, c, e = 257, 4, 512, 31
    shape = (t, k, c)
    experts = torch.rand(t, e, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    slot, offsets = torch.empty_like(experts), torch.empty(e + 1, dtype=torch.int32, device="cuda")
    a, b = torch.randn(t, c, device="cuda"), torch.empty(t, c, device="cuda")
    start = a.clone()
    rows, w = torch.empty(t * k, c, device="cuda"), torch.full((t, k), 0.25, device="cuda")
    other = [torch.randn(2048, 2048, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(200):
        if i % 20 == 0:
            with torch.cuda.stream(side):
                other[0] @ other[1]
        rs.reshard_expert_sort(experts, (t, k), e, slot, offsets, stream=main)
        rs.reshard_expert_dispatch(a, shape, "fp32", slot, rows, stream=main)
        rs.reshard_expert_combine(rows, shape, "fp32", slot, b, weight=w, stream=main)
        a, b = b, a
    torch.cuda.synchronize()
    assert torch.equal(a, start)             # four quarters of a value are the value


def test_threads_with_sizes_of_their_own():
    torch.manual_seed(8)
    made = [_score(3, 20000, 20), _score(200, 900, 130), _policy(40, 3001), _distill(30, 4001, 17, True),
            _distill(7, 30001, 64, False), _layer(300, 4, 640, 40, True), _layer(5000, 2, 64, 1500, False)]
    want = []
    for _, outs, call in made:
        call(None)
        torch.cuda.synchronize()
        want.append([o.clone().view(torch.uint8) for o in outs])
    for _, outs, _ in made:
        for o in outs:
            o.view(torch.uint8).fill_(0x5A)
    streams, errors = [torch.cuda.Stream() for _ in made], []
    torch.cuda.synchronize()

    def work(call, stream):
        try:
            for _ in range(200):
                call(stream)
        except Exception as e:        # noqa: BLE001 -- reported by the test
            errors.append(str(e))
    threads = [threading.Thread(target=work, args=(m[2], s)) for m, s in zip(made, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, outs, _), bits in zip(made, want):
        assert all(torch.equal(o.view(torch.uint8), b) for o, b in zip(outs, bits))
