"""What a product gives must not depend on the calls before it: the same product in fresh
processes, after different ones."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import hashlib, sys, torch
import dtensor_reshard_gb300 as rs

def product(tokens, n, k, dtype=torch.float32, name="fp32"):
    g = torch.Generator(device="cuda").manual_seed(n)
    def values(*shape):
        return torch.randint(0, 127, shape, generator=g, device="cuda", dtype=torch.uint8)
    x, w = values(tokens, k), values(n, k)
    xs = torch.rand((tokens, k // 128), generator=g, device="cuda")
    ws = torch.rand((-(-n // 128), k // 128), generator=g, device="cuda")
    y = torch.empty(tokens, n, dtype=dtype, device="cuda")
    rs.reshard_fp8_matmul(x, xs, w, ws, y, (tokens, n, k), name)
    torch.cuda.synchronize()
    return hashlib.sha256(y.cpu().numpy().tobytes()).hexdigest()

kinds = {"one": lambda: product(1, 2688, 7168), "some": lambda: product(33, 2688, 7168),
         "more": lambda: product(20, 1000, 4096), "many": lambda: product(513, 2688, 7168)}
print({k: kinds[k]() for k in sys.argv[1:]})
print({k: kinds[k]() for k in sorted(kinds)})
"""


def test_products_do_not_depend_on_earlier_calls():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    seen = []
    for order in (["one"], ["some", "one"], ["many", "more", "one", "some"]):
        r = subprocess.run([sys.executable, "-c", PROGRAM, *order], cwd=ROOT, capture_output=True,
                           text=True, timeout=300)
        assert r.returncode == 0, r.stderr
        first, every = map(eval, r.stdout.strip().splitlines())
        assert first.items() <= every.items()
        seen.append(every)
    assert seen[0] == seen[1] == seen[2]
