"""The operators from several host threads at once, each with sizes and a stream of its own."""
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


def _product(experts):
    """One token an expert, each times 2.0 over 256 values of 1.0: 512 everywhere."""
    x = torch.full((experts, 256), 0x38, dtype=torch.uint8, device="cuda")       # 1.0
    w = torch.full((experts, 128, 256), 0x40, dtype=torch.uint8, device="cuda")  # 2.0
    xs, ws = torch.ones(experts, 2, device="cuda"), torch.ones(experts, 1, 2, device="cuda")
    offsets = torch.arange(experts + 1, device="cuda", dtype=torch.int32)
    y = torch.zeros(experts, 128, device="cuda")

    def call(stream):
        rs.reshard_fp8_matmul(x, xs, w, ws, y, (experts, 128, 256), "fp32", offsets=offsets,
                              nexperts=experts, stream=stream)
    return call, lambda: bool((y == 512).all())


def _sample(vocab):
    logits = torch.zeros(152, vocab, device="cuda")
    logits[:, vocab // 2] = 100.0
    u = torch.full((152,), 0.5, device="cuda")
    token = torch.zeros(152, dtype=torch.int32, device="cuda")

    def call(stream):
        rs.reshard_sample(logits, (152, vocab), "fp32", u, token, stream=stream)
    return call, lambda: bool((token == vocab // 2).all())


def _balance(experts):
    shape = (1, 300, experts)
    logits = torch.zeros(shape, device="cuda")
    choices = torch.arange(300, device="cuda", dtype=torch.int32).view(1, 300, 1) % experts
    workspace = torch.empty(rs.reshard_balance_loss_workspace(shape), dtype=torch.uint8, device="cuda")
    counts = torch.zeros(experts, dtype=torch.int32, device="cuda")
    loss = torch.zeros(1, device="cuda")

    def call(stream):
        rs.reshard_balance_loss(logits, shape, "fp32", choices, 1, 1.0, workspace, counts, loss=loss,
                                stream=stream)
    return call, lambda: int(counts.sum()) == 300 and abs(float(loss) - 1.0) < 1e-5


def _run(jobs, calls, prepare):
    errors = []

    def work(call, stream):
        try:
            prepare()
            for _ in range(calls):
                call(stream)
        except Exception as e:        # noqa: BLE001 -- reported by the test
            errors.append(str(e))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(job[0], s)) for job, s in zip(jobs, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for _, right in jobs:
        assert right()


def test_threads_with_sizes_of_their_own():
    """A kernel's limit of shared memory belongs to the process: no call may lower it under
    another one's."""
    jobs = [_product(e) for e in (2, 900, 3000)] + [_sample(v) for v in (300, 9000, 40000)]
    jobs += [_balance(e) for e in (544, 1024)]
    _run(jobs, 2000, lambda: torch.zeros(1, device="cuda"))


def test_a_thread_that_has_not_used_the_gpu_yet():
    """No context is current on a new host thread until a call makes it so."""
    for make in (lambda: _product(2), lambda: _product(40), lambda: _sample(300), lambda: _balance(544)):
        call, right = make()
        call(None)                    # the library has met the device, the thread below has not
        assert right()
        _run([make()], 3, lambda: None)
