"""The operators beside a refit on a GB300, against plain 64-bit forms (operator_oracles):
quantisation, the block-scaled product, sampling and the balance loss, at the sizes,
strides and masks where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import dtensor_reshard_gb300 as rs
from tests import operator_oracles as oo

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# half a unit in the last place of a result (finfo.eps / 2), and of the smallest one
EPS = {"bf16": (2.0 ** -8, 0.0), "fp16": (2.0 ** -11, 2.0 ** -25), "fp32": (2.0 ** -24, 0.0)}
E4M3 = torch.tensor(oo.e4m3_values(), dtype=torch.float64)


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required")
    yield
    assert rs.reshard_device_status(clear=True) == 0


def _f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


# --------------------------------------------------------------------------- quantize
def _quantize(x, block_rows, ldx=None, ldq=None, lds=None, shift=0, dtype="bf16"):
    """Quantise x [n, r, c] laid out with the given pitches, `shift` elements past an
    aligned address; also checks that nothing but the outputs was written."""
    n, r, c = x.shape
    ldx, ldq, lds = ldx or c, ldq or c, lds or -(-c // 128)
    buf = torch.full((shift + n * r * ldx,), 7.0, dtype=DT[dtype], device="cuda")
    buf[shift:].view(n, r, ldx)[:, :, :c] = x
    R, C = -(-r // block_rows), -(-c // 128)
    q = torch.full((n * r * ldq + shift,), 0xA5, dtype=torch.uint8, device="cuda")
    s = torch.full((n, R, lds), -5.0, device="cuda")
    rs.reshard_fp8_quantize(buf[shift:], q[shift:], s, (n, r, c), dtype, block_rows, ldx=ldx,
                            ldq=ldq, lds=lds)
    torch.cuda.synchronize()
    assert bool((q[:shift] == 0xA5).all())
    q = q[shift:].view(n, r, ldq)
    assert bool((q[:, :, c:] == 0xA5).all()) and bool((s[:, :, C:] == -5.0).all())
    return E4M3[q[:, :, :c].cpu().long()].numpy(), s[:, :, :C].cpu().numpy()


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 1, 128), (1, 3, 129), (2, 130, 257), (3, 128, 128),
                                   (2, 1, 7168), (1, 257, 1000), (1, 5, 16), (1, 300, 40),
                                   (1, 33, 2048)])
def test_quantize_is_exact(shape, dtype, block_rows):
    g = torch.Generator(device="cuda").manual_seed(sum(shape) + block_rows)
    x = torch.randn(shape, generator=g, device="cuda") * 3
    x *= 1 + 30 * (torch.rand(shape[2], generator=g, device="cuda") > 0.98)
    x = x.to(DT[dtype])
    for ldx, ldq, lds, shift in ((None, None, None, 0), (shape[2] + 8, shape[2] + 16, None, 8),
                                 (shape[2] + 3, shape[2] + 1, -(-shape[2] // 128) + 2, 1)):
        q, s = _quantize(x, block_rows, ldx, ldq, lds, shift, dtype)
        wq, ws = oo.quantize(_f64(x), block_rows)
        assert np.array_equal(s, ws)
        assert np.array_equal(q, wq)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("cols", [256, 201])
def test_quantize_of_zeros_extremes_nan_and_infinities(block_rows, cols):
    x = torch.zeros(1, 6, cols, device="cuda")
    x[0, 1, :5] = torch.tensor([3e38, -1e38, 1.0, -0.0, 1e-40])
    x[0, 2, 3] = math.nan
    x[0, 2, 4:7] = torch.tensor([1.0, -2.0, 448.0])
    x[0, 4, 0] = 1e-44                       # a scale below the smallest
    x[0, 5, 130:133] = torch.tensor([math.inf, 5.0, -math.inf])
    if block_rows == 128:                    # one kind of block at a time
        for row in range(6):
            one = x[:, row:row + 1]
            q, s = _quantize(one, 128, dtype="fp32")
            wq, ws = oo.quantize(_f64(one), 128)
            assert np.array_equal(s, ws) and np.array_equal(q, wq, equal_nan=True)
    q, s = _quantize(x, block_rows, dtype="fp32")
    wq, ws = oo.quantize(_f64(x), block_rows)
    assert np.array_equal(s, ws) and np.array_equal(q, wq, equal_nan=True)


# ----------------------------------------------------------------------------- matmul
def _operands(t, n, k, e, seed, pad=0):
    """(bytes, pitches, values, scales) of random operands; bytes beyond k are NaN's."""
    g = torch.Generator().manual_seed(seed)
    ld = -(-k // 16) * 16 + 16 * pad
    out = []
    for rows, br in (((1, t), 1), ((e, n), 128)):
        b = torch.randint(0, 256, (*rows, ld), generator=g, dtype=torch.uint8)
        b[(b & 127) == 127] -= 1             # no NaN inside the rows
        b[..., k:] = 0x7F
        s = torch.rand((rows[0], -(-rows[1] // br), -(-k // 128) + pad), generator=g) * 0.01 + 1e-4
        out += [b, s]
    return ld, out


def _product(t, n, k, dtype, experts=0, counts=None, seed=0, pad=0, rows=None, fill=None):
    e = max(1, experts)
    ld, (x, xs, w, ws) = _operands(t, n, k, e, seed, pad)
    if fill:
        fill(x, xs, w, ws)
    offsets = None
    if experts:
        offsets = torch.cat([torch.zeros(1), torch.tensor(counts).cumsum(0)]).to(torch.int32)
        offsets += rows or 0
    ldy = n + pad
    y = torch.full((t, ldy), 77.0, dtype=DT[dtype], device="cuda")
    B = -(-k // 128)
    rs.reshard_fp8_matmul(x.cuda(), xs.cuda(), w.cuda(), ws.cuda(), y, (t, n, k), dtype,
                          offsets=None if offsets is None else offsets.cuda(), nexperts=e, ldx=ld,
                          ldw=ld, ldxs=B + pad, ldws=B + pad, ldy=ldy)
    torch.cuda.synchronize()
    want, bound = oo.matmul(E4M3[x[0].long()][:, :k].numpy(), _f64(xs[0])[:, :B],
                            E4M3[w.long()][:, :, :k].numpy(), _f64(ws)[:, :, :B],
                            None if offsets is None else offsets.numpy(), EPS[dtype][0])
    y = _f64(y)
    assert np.all(y[:, n:] == 77.0)
    return y[:, :n], want, bound + EPS[dtype][1]


def _near(got, want, bound):
    untouched = np.isnan(want)
    assert np.all(got[untouched] == 77.0)
    worst = (np.abs(got - want) - bound)[~untouched]
    assert np.all(worst <= 0), (float(worst.max()), np.argwhere(np.abs(got - want) > bound)[:4])


@pytest.mark.parametrize("t", [1, 2, 7, 16, 17, 63, 64, 65, 129, 200, 300])
@pytest.mark.parametrize("n,k", [(1, 1), (8, 16), (127, 100), (128, 128), (129, 129), (257, 640),
                                 (520, 1000)])
def test_matmul(t, n, k):
    for dtype, pad in (("bf16", 0), ("fp16", 1), ("fp32", 3)):
        _near(*_product(t, n, k, dtype, seed=t * 31 + n + k, pad=pad))


@pytest.mark.parametrize("n,k", [(2048, 2048), (72, 4100), (2688, 7168)])
@pytest.mark.parametrize("t", [1, 33, 513])
def test_matmul_long(t, n, k):
    _near(*_product(t, n, k, "bf16", seed=t + n))
    _near(*_product(t, n, k, "fp32", seed=t + n + 1))


@pytest.mark.parametrize("counts", [[5], [0, 3, 0, 0, 9, 0], [128, 1, 127, 129, 0, 300],
                                    [0, 0, 0], [1] * 70, [0] * 200 + [2] + [0] * 55,
                                    [700, 13, 0, 260]])
@pytest.mark.parametrize("n,k", [(40, 100), (130, 256), (256, 777)])
def test_matmul_of_experts(counts, n, k):
    t = sum(counts) + 5                      # rows before and after every expert's stay as they were
    for dtype, pad in (("bf16", 0), ("fp32", 1)):
        _near(*_product(t, n, k, dtype, len(counts), counts, seed=len(counts) + n, pad=pad, rows=2))


def test_matmul_clamps_offsets_to_the_tokens():
    ld, (x, xs, w, ws) = _operands(20, 64, 128, 3, 5)
    x, xs, w, ws = (v.cuda() for v in (x, xs, w, ws))
    got = []
    for offsets in ([0, 7, 20, 20], [-9, 7, 10 ** 6, 10 ** 6]):
        y = torch.zeros(20, 64, device="cuda")
        rs.reshard_fp8_matmul(x, xs, w, ws, y, (20, 64, 128), "fp32",
                              offsets=torch.tensor(offsets, dtype=torch.int32).cuda(), nexperts=3,
                              ldx=ld, ldw=ld)
        got.append(y)
    torch.cuda.synchronize()
    assert torch.equal(got[0], got[1]) and bool((got[0] != 0).any())


@pytest.mark.parametrize("t", [3, 200])
def test_matmul_passes_nan_and_infinite_scales(t):
    """A NaN value or scale reaches exactly the outputs that it is a factor of."""
    def fill(x, xs, w, ws):
        x[0, 1, 5] = 0x7F
        w[0, 9, 3] = 0x7F
        xs[0, 2, 0] = math.inf
    got, want, bound = _product(t, 150, 256, "fp32", seed=3, fill=fill)
    bad = np.zeros((t, 150), bool)
    bad[1], bad[:, 9], bad[2] = True, True, True
    assert np.array_equal(np.isfinite(got), ~bad)
    ok = ~bad
    assert np.all(np.abs(got - want)[ok] <= bound[ok])


def test_matmul_without_inner_size_is_zero():
    y = torch.full((3, 5), 9.0, device="cuda")
    rs.reshard_fp8_matmul(None, None, None, None, y, (3, 5, 0), "fp32")
    torch.cuda.synchronize()
    assert bool((y == 0).all())


def test_matmul_on_a_stream_and_in_a_graph_gives_equal_bits():
    ld, (x, xs, w, ws) = _operands(300, 700, 900, 1, 8)
    x, xs, w, ws = (v.cuda() for v in (x, xs, w, ws))

    def call(y, stream):
        rs.reshard_fp8_matmul(x, xs, w, ws, y, (300, 700, 900), "fp32", ldx=ld, ldw=ld, stream=stream)
    ys = [torch.zeros(300, 700, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    call(ys[0], None)
    side = torch.cuda.Stream()
    call(ys[1], side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(ys[2], side)
    graph.replay()
    torch.cuda.synchronize()
    assert bool((ys[0] != 0).any())
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


# ----------------------------------------------------------------------------- sample
def _sample(x, dtype, temperature, top_k, top_p, min_p, u, ld=None):
    rows, v = x.shape
    ld = ld or v
    buf = torch.full((rows, ld), 1e4, dtype=DT[dtype], device="cuda")
    buf[:, :v] = x
    token = torch.full((rows,), -99, dtype=torch.int32, device="cuda")
    logprob = torch.full((rows,), 5.0, device="cuda")
    dev = [None if a is None else torch.tensor(a, dtype=t, device="cuda") for a, t in (
        (temperature, torch.float32), (top_k, torch.int32), (top_p, torch.float32),
        (min_p, torch.float32), (u, torch.float32))]
    rs.reshard_sample(buf, (rows, v), dtype, dev[4], token, logprob, *dev[:4], ld=ld)
    torch.cuda.synchronize()
    x = _f64(buf[:, :v])
    f32 = [None if d is None else _f64(d) for d in dev]
    for r in range(rows):
        args = [dflt if a is None else a[r] for a, dflt in zip(f32, (1.0, 0, 1.0, 0.0, 0.0))]
        tokens, lp = oo.sample(x[r], *args)
        got = int(token[r])
        assert got in tokens, (r, got, tokens, args)
        want = -math.inf if lp is None else float(lp[got])
        have = float(logprob[r])
        # |z| rounds twice in float32, the sum's logarithm is off by its terms' 2^-22 at most
        assert have == want or abs(have - want) <= 2.0 ** -22 * (abs(want) * 2 + 8), (r, have, want)
    return token.cpu()


VOCABS = [1, 2, 31, 257, 1000, 1025, 5003, 50021]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_sample_settings(vocab, dtype):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    settings = [(t, k, p, m) for t in (0.0, 0.3, 1.0, 2.0) for k in (0, 1, 5, 200)
                for p, m in ((1.0, 0.0), (0.9, 0.0), (0.3, 0.1), (1.0, 0.05))]
    n = len(settings)
    x = torch.randn(n, vocab, generator=g, device="cuda") * 3
    u = torch.rand(n, generator=g, device="cuda").tolist()
    _sample(x, dtype, *map(list, zip(*settings)), u)
    _sample(x, dtype, *map(list, zip(*settings)), u, ld=vocab + 3)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [9, 300, 4099])
def test_sample_of_flat_and_tied_rows(vocab, dtype):
    """Ties at every threshold go to the lowest index."""
    x = torch.zeros(24, vocab, device="cuda")
    x[8:16] = (torch.arange(vocab, device="cuda") % 3).float()
    x[16:] = -(torch.arange(vocab, device="cuda") % 2).float() * 0.0   # -0 and +0 are one value
    k = [0, 1, 2, 3, 4, 5, 7, vocab] * 3
    p = [1.0, 1.0, 0.5, 0.7, 1.0, 0.01, 0.99, 0.5] * 3
    for u in (0.0, 0.26, 0.74, 0.999):
        _sample(x, dtype, [1.0] * 24, k, p, [0.0, 0.0, 0.0, 0.4] * 6, [u] * 24)


@pytest.mark.parametrize("vocab", [5, 130, 2500])
def test_sample_of_masked_rows_infinities_and_nan(vocab):
    lowest = torch.finfo(torch.float32).min
    x = torch.randn(10, vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    x[0] = -math.inf                         # nothing left
    x[1] = math.nan
    x[2] = lowest                            # all masked with the type's lowest value: uniform
    x[3, 1:] = -math.inf                     # one left
    x[4, ::2] = -math.inf
    x[5, ::2] = lowest
    x[6, 1] = math.nan
    x[7, [1, 3]] = math.inf                  # only these two can be taken
    x[8] = lowest
    x[8, 2] = -math.inf
    x[9, 0] = 3e38                           # differences overflow
    x[9, 1:] = -3e38
    for t, k, p, u in ((1.0, 0, 1.0, 0.4), (0.5, 3, 0.9, 0.9), (0.0, 0, 1.0, 0.5), (1.0, 0, 0.5, 0.0),
                       (math.inf, 0, 1.0, 0.6), (1e-42, 0, 1.0, 0.6)):
        tok = _sample(x, "fp32", [t] * 10, [k] * 10, [p] * 10, [0.0] * 10, [u] * 10)
        assert tok[0] == -1 and tok[1] == -1 and tok[3] == 0 and int(tok[7]) in (1, 3)
        assert int(tok[4]) % 2 == 1 and tok[6] != 1 and tok[8] != 2
        # an infinite temperature makes every finite logit as likely, the lowest one too
        assert int(tok[5]) % 2 == 1 or t == math.inf


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [15, 60])        # CTAs of 512 and of 256 threads
def test_sample_wherever_the_cut_lies(dtype, rows):
    """The last kept token at several depths below the largest, alone there, among a few hundred tokens that
    are nearly alike, and among thousands; by top-p, by top-k, and by both."""
    vocab = 20011
    g = torch.Generator(device="cuda").manual_seed(rows)
    for depth in (0.5, 5.0, 10.6, 10.7, 13.25, 16.0):
        for alike in (1, 100, 300, 390, 5000):
            x = torch.full((rows, vocab), -60.0, device="cuda")
            x[:, 7::97] = -depth - 3 - torch.rand(rows, len(range(7, vocab, 97)), generator=g, device="cuda")
            x[:, 11:11 + 4 * alike:4] = -depth - 0.004 * torch.rand(rows, alike, generator=g, device="cuda")
            x[:, 13000] = 0.0
            # half of the mass of the alike tokens belongs to the nucleus
            mass = alike * math.exp(-depth)
            total = 1 + mass + (vocab // 97) * math.exp(-depth - 3.5)
            p = [(1 + 0.5 * mass) / total, 1.0, 0.999 - 0.3 * mass / total] * (rows // 3)
            k = [0, 1 + (alike + 1) // 2, 1 + alike - alike // 4] * (rows // 3)
            _sample(x, dtype, [1.0] * rows, k, p, [0.0] * rows,
                    torch.rand(rows, generator=g, device="cuda").tolist())


def test_sample_odd_settings_and_defaults():
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn(12, 700, device="cuda", generator=g) * 2
    nan, inf = math.nan, math.inf
    _sample(x, "fp32", [1.0, nan, -1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 1.0, 0.01],
            [-3, 0, 0, 10 ** 9, 700, 699, 0, 0, 0, 0, 0, 0],
            [2.0, 0.5, 0.5, 1.0, 1.0, 1.0, 0.0, -1.0, nan, 0.9, 1e-30, 0.9999],
            [0.0, 0.0, 0.0, 5.0, -1.0, nan, 0.0, 0.0, 0.0, 1.0, 0.0, 0.0],
            [0.5, 0.5, 0.5, 0.5, 1.0, 0.5, 0.9, 0.9, 0.9, inf, -2.0, nan])
    for absent in range(4):
        args = [[0.7] * 12, [20] * 12, [0.8] * 12, [0.1] * 12]
        args[absent] = None
        _sample(x, "bf16", *args, torch.rand(12, generator=g, device="cuda").tolist())
    _sample(x, "fp16", None, None, None, None, torch.rand(12, generator=g, device="cuda").tolist())
    # no log-probability asked for
    token = torch.empty(12, dtype=torch.int32, device="cuda")
    rs.reshard_sample(x, (12, 700), "fp32", torch.zeros(12, device="cuda"), token)
    torch.cuda.synchronize()
    assert bool((token == 0).all())


def test_sample_follows_the_distribution():
    """20000 draws of one row fall on its tokens as often as their probabilities say."""
    p = torch.tensor([0.5, 0.2, 0.0, 0.15, 0.1, 0.05])
    rows = 20000
    x = p.log().repeat(rows, 1).cuda()
    u = ((torch.arange(rows) + 0.5) / rows).cuda()
    token = torch.empty(rows, dtype=torch.int32, device="cuda")
    rs.reshard_sample(x, (rows, 6), "fp32", u, token)
    share = torch.bincount(token.cpu().long(), minlength=6) / rows
    assert float((share - p).abs().max()) <= 1.5 / rows      # u is a grid: one point each way


@pytest.mark.parametrize("dtype,vocab", [("bf16", 262144), ("fp32", 262144), ("fp16", 1 << 20),
                                         ("fp32", 1 << 20)])
def test_sample_large_vocabularies(dtype, vocab):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.randn(5, vocab, generator=g, device="cuda") * 2
    x[1, 1::2] = -math.inf
    x[2] = 0.5
    _sample(x, dtype, [1.0, 0.7, 1.0, 0.0, 0.8], [0, 0, 70000, 0, 50], [0.95, 0.9, 0.5, 1.0, 0.9],
            [0.0, 0.0, 0.0, 0.0, 0.02], [0.7, 0.2, 0.6, 0.1, 0.95])


# ---------------------------------------------------------------------------- balance
def _balance(x, experts, mask, topk, score, dtype, coef=0.01, grad=None, ld=None, loss=True,
             dlogits=True):
    S, T, E = x.shape
    ld = ld or E
    buf = torch.full((S, T, ld), math.nan, dtype=DT[dtype], device="cuda")
    buf[:, :, :E] = x
    out = torch.full((S, T, ld), 7.0, dtype=DT[dtype], device="cuda")
    nbytes = rs.reshard_balance_loss_workspace((S, T, E))
    ws = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    counts = torch.full((S, E), -3, dtype=torch.int32, device="cuda")
    lo = torch.full((1,), 9.0, device="cuda")
    g = None if grad is None else torch.tensor([grad], device="cuda")
    dev = [experts.to("cuda", torch.int32), None if mask is None else mask.to("cuda", torch.uint8)]
    for _ in range(2):                       # the second call finds the first one's workspace
        rs.reshard_balance_loss(buf, (S, T, E), dtype, dev[0], topk, coef, ws, counts,
                                loss=lo if loss else None, dlogits=out if dlogits else None,
                                mask=dev[1], score=score, grad=g, ld=ld)
    torch.cuda.synchronize()
    assert bool((out[:, :, E:] == 7.0).all())
    return float(lo), counts.cpu().numpy(), _f64(out[:, :, :E]), _f64(buf[:, :, :E])


def _check_balance(x, experts, mask, topk, score, dtype, coef=0.01, grad=None, **kw):
    lo, counts, got, xv = _balance(x, experts, mask, topk, score, dtype, coef, grad, **kw)
    m = None if mask is None else mask.numpy()
    want, wcounts, wgrad, tokens = oo.balance(xv, experts.numpy(), m, topk, score, coef)
    assert np.array_equal(counts, wcounts)
    S, T, E = x.shape
    # float32 scores of E terms: E / 32 + 5 additions and about 16 roundings beside them,
    # exponentials' arguments rounded at |l| <= 2^5; f and dot carry the same again
    rel = (E / 32 + 21 + 32) * 2.0 ** -23
    f = wcounts * E / (topk * np.maximum(tokens, 1))[:, None]
    if kw.get("loss", True):
        assert abs(lo - want) <= 2 * rel * max(abs(want), 1e-30), (lo, want)
    if not kw.get("dlogits", True):
        assert np.all(got == 7.0)
        return
    scale = abs(1.0 if grad is None else grad)
    live = max(1, int((tokens > 0).sum()))
    slope = np.zeros(x.shape)
    for s in range(S):
        for t in range(T):
            slope[s, t] = oo.scores(xv[s, t], score)[1]
    n = np.maximum(tokens, 1)[:, None, None]
    size = scale * coef / (live * n) * slope * (f[:, None, :] + f.max(1)[:, None, None])
    wgrad = wgrad * (1.0 if grad is None else grad)
    if m is not None:
        size = np.where(m[..., None] != 0, size, 0.0)
    eps, tiny = EPS[dtype]
    assert np.all(np.abs(got - wgrad) <= 2 * rel * np.nan_to_num(size) + eps * np.abs(wgrad) + tiny
                  + 2.0 ** -133)


def _router(S, T, E, topk, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(S, T, E, generator=g) + torch.randn(E, generator=g)
    experts = x.topk(topk, dim=2).indices.to(torch.int32)
    return x, experts, g


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("S,T,E,topk", [(1, 1, 1, 1), (1, 61, 19, 2), (3, 130, 8, 1), (2, 65, 256, 8),
                                        (4, 7, 33, 4), (1, 300, 64, 6), (2, 20, 1000, 8),
                                        (1, 5, 4096, 3), (40, 3, 16, 2)])
def test_balance(S, T, E, topk, dtype, score):
    x, experts, g = _router(S, T, E, topk, S * 7 + T + E)
    _check_balance(x, experts, None, topk, score, dtype, ld=E + 5)
    mask = torch.rand(S, T, generator=g) < 0.6
    mask[S // 2] = False                     # a sequence without tokens
    _check_balance(x, experts, mask.to(torch.uint8), topk, score, dtype, grad=-3.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_matches_differences(score):
    """The kernel's gradient against central differences of the 64-bit loss.  The step's
    error is h^2 / 6 of a third derivative below f's largest value times the slope's
    bound of 1, the kernel's own a few float32 roundings of the same size."""
    S, T, E, topk, h = 2, 5, 6, 2, 1e-4
    x, experts, _ = _router(S, T, E, topk, 5)
    mask = torch.ones(S, T, dtype=torch.uint8)
    mask[1, 3:] = 0
    lo, counts, got, xv = _balance(x, experts, mask, topk, score, "fp32", coef=1.0)
    f_most = (counts * E / (topk * np.array([[5], [3]]))).max()
    for s in range(S):
        for t in range(T):
            for e in range(E):
                d = xv.copy()
                d[s, t, e] += h
                up = oo.balance(d, experts.numpy(), mask.numpy(), topk, score, 1.0)[0]
                d[s, t, e] -= 2 * h
                dn = oo.balance(d, experts.numpy(), mask.numpy(), topk, score, 1.0)[0]
                assert abs(got[s, t, e] - (up - dn) / (2 * h)) <= f_most * (h * h + 2.0 ** -20)


def test_balance_dropped_choices_masked_logits_and_padding():
    x, experts, g = _router(2, 50, 12, 3, 9)
    experts[0, ::3, 1] = -1                  # dropped
    experts[1, 5] = 10 ** 6
    mask = torch.ones(2, 50, dtype=torch.uint8)
    mask[1, 40:] = 0
    x[1, 40:] = math.nan                     # padding holds anything
    x[0, :, 4] = -math.inf                   # an expert that is switched off
    x[0, 7] = -math.inf                      # a token with none left
    x[0, 8] = torch.finfo(torch.float32).min
    for score in ("softmax", "sigmoid"):
        _check_balance(x, experts, mask, 3, score, "fp32")
        _check_balance(x, experts, mask, 3, score, "fp32", loss=False)
        _check_balance(x, experts, mask, 3, score, "fp32", dlogits=False)


def test_balance_without_tokens():
    x, experts, _ = _router(3, 40, 9, 2, 2)
    lo, counts, got, _ = _balance(x, experts, torch.zeros(3, 40), 2, "softmax", "bf16")
    assert lo == 0.0 and not counts.any() and not got.any()
    loss = torch.full((1,), 4.0, device="cuda")
    counts = torch.full((3, 9), 4, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(16, rs.reshard_balance_loss_workspace((3, 0, 9))), dtype=torch.uint8,
                     device="cuda")
    rs.reshard_balance_loss(None, (3, 0, 9), "bf16", None, 2, 0.01, ws, counts, loss=loss)
    torch.cuda.synchronize()
    assert float(loss) == 0.0 and not bool(counts.any())


def test_balance_gives_equal_bits_every_time():
    x, experts, _ = _router(5, 700, 256, 8, 3)
    first = _balance(x, experts, None, 8, "sigmoid", "fp32")
    for _ in range(3):
        again = _balance(x, experts, None, 8, "sigmoid", "fp32")
        assert first[0] == again[0] and np.array_equal(first[2], again[2])
