"""Timed cases of the operators that run beside a weight refit.

A refit hands a mixture-of-experts model's weights from its trainer to the ranks
that generate with it.  The operators timed here are what both ends compute around
that copy:

  quantize   bfloat16/float16/float32 -> 8-bit floating point (e4m3) with one float32
             scale for each 1x128 (activations) or 128x128 (weights) block;
  matmul     the product of two such matrices, dense or one weight matrix per expert
             over rows sorted by expert;
  sample     one token a row from its logits (temperature, top-k, top-p, min-p) with
             one given uniform number a row, and the token's log-probability;
  balance    the router's load-balance loss, the tokens each expert got, and the
             gradient in the router's logits.

``run`` computes them in elementary torch operations, or with the library's kernels
where ``own`` is true; ``exact`` computes the same definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126   # a block of zeros gets this scale
ONE = 1 << 40             # sampling weights are whole multiples of 2^-40 of the largest

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def cdiv(a, b):
    return -(-a // b)


def up(a, b):
    return cdiv(a, b) * b


# ------------------------------------------------------------------------------ cases
def quantize_case(nmat, rows, cols, dtype, block_rows):
    return {"op": "quantize", "nmat": nmat, "rows": rows, "cols": cols, "dtype": dtype,
            "block_rows": block_rows}


def matmul_case(tokens, n, k, experts, out):
    """experts = 0: one weight matrix; else one for each expert, rows sorted by expert."""
    return {"op": "matmul", "tokens": tokens, "n": n, "k": k, "experts": experts, "out": out}


def sample_case(rows, vocab, dtype, mix):
    """mix: the requests' settings ("greedy", "plain", "nucleus" or "mixed")."""
    return {"op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "mix": mix}


def balance_case(seqs, tokens, experts, topk, dtype, score, padded):
    return {"op": "balance", "seqs": seqs, "tokens": tokens, "experts": experts, "topk": topk,
            "dtype": dtype, "score": score, "padded": padded}


def listed():
    def named(name, case):
        return {"name": name, **case}
    return [
        # one decoded token's hidden state before its product: a call is all latency
        named("quantize_one_token", quantize_case(1, 1, 7168, "bf16", 1)),
        # the trainer's side of an 8-bit refit: one source rank's 16 experts of [2048, 7168]
        named("quantize_experts", quantize_case(16, 2048, 7168, "bf16", 128)),
        # one decoded token through a tensor-parallel rank's eighth of a [21504, 7168] weight
        named("matmul_one_token", matmul_case(1, 2688, 7168, 0, "bf16")),
        # sizes that divide nothing, float32 out: a reduced model
        named("matmul_ragged", matmul_case(777, 2867, 819, 0, "fp32")),
        # a prompt batch through a dense feed-forward up-projection [14336, 4096]
        named("matmul_prompt", matmul_case(8192, 14336, 4096, 0, "bf16")),
        # a decode batch over all 256 experts, each rank holding an eighth of their rows
        named("matmul_experts_decode", matmul_case(1024, 256, 7168, 256, "bf16")),
        # a prompt batch over an expert-parallel rank's 16 whole experts
        named("matmul_experts_prompt", matmul_case(16384, 2048, 7168, 16, "bf16")),
        # one request's next token over a large vocabulary: latency
        named("sample_one", sample_case(1, 131072, "bf16", "nucleus")),
        # odd vocabulary, float32 logits, a few requests of every kind, some tokens masked
        named("sample_odd", sample_case(37, 50021, "fp32", "mixed")),
        # a generation batch of every kind of request
        named("sample_batch", sample_case(256, 131072, "bf16", "mixed")),
        # a short sequence through a small router
        named("balance_small", balance_case(1, 61, 19, 2, "fp32", "softmax", False)),
        # a training micro-batch, sequence-wise loss over 256 experts, 8 of them a token
        named("balance_batch", balance_case(16, 8192, 256, 8, "bf16", "sigmoid", True)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: most elements (quantize, sample, balance) or multiply-adds (matmul) of a drawn case
_MOST = {"quantize": 16 * 2048 * 7168, "matmul": 8192 * 14336 * 4096, "sample": 256 * 131072,
         "balance": 16 * 8192 * 256}


def draw(rng):
    op = rng.choice(("quantize", "matmul", "matmul", "sample", "sample", "balance"))
    while True:
        if op == "quantize":
            block_rows = rng.choice((1, 128))
            nmat = 1 if block_rows == 1 else _log(rng, 1, 16)
            case = quantize_case(nmat, _log(rng, 1, 16384), _log(rng, 17, 14336),
                                 rng.choice(("bf16", "bf16", "fp16", "fp32")), block_rows)
            cost = nmat * case["rows"] * case["cols"]
        elif op == "matmul":
            experts = rng.choice((0, 0, _log(rng, 2, 256)))
            case = matmul_case(_log(rng, 1, 16384), _log(rng, 24, 14336), _log(rng, 40, 8192),
                               experts, rng.choice(("bf16", "bf16", "fp16", "fp32")))
            cost = case["tokens"] * case["n"] * case["k"]
            if max(1, experts) * case["n"] * case["k"] > 256 * 256 * 7168:
                continue
        elif op == "sample":
            case = sample_case(_log(rng, 1, 512), _log(rng, 300, 262144),
                               rng.choice(("bf16", "bf16", "fp16", "fp32")),
                               rng.choice(("greedy", "plain", "nucleus", "mixed", "mixed")))
            cost = case["rows"] * case["vocab"]
        else:
            experts = _log(rng, 4, 512)
            case = balance_case(_log(rng, 1, 32), _log(rng, 1, 16384), experts,
                                rng.randint(1, min(8, experts)),
                                rng.choice(("bf16", "fp16", "fp32")),
                                rng.choice(("softmax", "sigmoid")), rng.random() < 0.5)
            cost = case["seqs"] * case["tokens"] * experts
        if cost <= _MOST[op]:
            return case


# ----------------------------------------------------------------------------- inputs
def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _blocks(x, block_rows):
    """[n, r, c] padded with zeros to whole blocks, as [n, R, block_rows, C, 128]."""
    n, r, c = x.shape
    x = torch.nn.functional.pad(x, (0, up(c, BLOCK) - c, 0, up(r, block_rows) - r))
    return x.view(n, -1, block_rows, x.shape[2] // BLOCK, BLOCK)


def _quantized(x, block_rows):
    """(8-bit values [n, r, pitch], scales [n, R, C]) of float32 x [n, r, c]."""
    n, r, c = x.shape
    b = _blocks(x, block_rows)
    s = (b.abs().amax(dim=(2, 4)) / E4M3_MAX).clamp_min(SCALE_MIN)
    b = (b / s[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = b.view(n, -1, b.shape[3] * BLOCK)[:, :r, :up(c, 16)].contiguous()
    return q, s


def _counts(case, seed):
    """Rows of each expert: uneven, as routers give them, some experts with none."""
    g = _gen(seed + 11, "cpu")
    e = case["experts"]
    popularity = torch.rand(e, generator=g) ** 2 + 1e-3
    chosen = torch.multinomial(popularity, case["tokens"], replacement=True, generator=g)
    return torch.bincount(chosen, minlength=e)


def prepare(case, seed):
    g = _gen(seed)
    state = {"case": case}
    if case["op"] == "quantize":
        n, r, c = case["nmat"], case["rows"], case["cols"]
        weights = case["block_rows"] > 1
        x = _normal((n, r, c), g, 0.02 if weights else 1.0)
        if not weights:   # a few channels of activations are far larger than the rest
            x *= 1 + 20 * (torch.rand((1, 1, c), generator=g, device="cuda") > 0.995)
        state["x"] = x.to(DTYPES[case["dtype"]])
        state["q"] = torch.empty((n, r, c), dtype=torch.float8_e4m3fn, device="cuda")
        state["scale"] = torch.empty((n, cdiv(r, case["block_rows"]), cdiv(c, BLOCK)),
                                     device="cuda")
    elif case["op"] == "matmul":
        t, n, k, e = case["tokens"], case["n"], case["k"], case["experts"]
        x, xs = _quantized(_normal((1, t, k), g), 1)
        state["x"], state["xs"] = x[0], xs[0]
        state["w"], state["ws"] = _quantized(_normal((max(1, e), n, k), g, 0.02), BLOCK)
        state["y"] = torch.empty((t, n), dtype=DTYPES[case["out"]], device="cuda")
        state["offsets"] = None
        if e:
            counts = _counts(case, seed)
            state["most"] = int(counts.max())
            state["offsets"] = torch.cat([torch.zeros(1), counts.cumsum(0)]).to("cuda",
                                                                               torch.int32)
    elif case["op"] == "sample":
        rows, v = case["rows"], case["vocab"]
        # a head's logits: a wide bulk, and a few tokens that the context makes likely
        x = _normal((rows, v), g, 2.0)
        likely = torch.randint(0, v, (rows, 24), generator=g, device="cuda")
        x.scatter_add_(1, likely, 8 + 3 * _normal((rows, 24), g))
        mixed = case["mix"] == "mixed"
        if mixed:         # a grammar forbids some tokens of some rows
            off = torch.rand((rows, v), generator=g, device="cuda") < 0.3
            x[1::4] = x[1::4].masked_fill(off[1::4], -math.inf)
        kind = torch.arange(rows, device="cuda") % 4
        kind = {"greedy": kind * 0, "plain": kind * 0 + 1, "nucleus": kind * 0 + 2,
                "mixed": kind}[case["mix"]]

        def by_kind(*values):
            return torch.tensor(values, device="cuda")[kind]
        # greedy; the whole distribution; nucleus; short list with a floor
        state["logits"] = x.to(DTYPES[case["dtype"]])
        state["temperature"] = by_kind(0.0, 1.0, 0.7, 0.8)
        state["top_k"] = by_kind(0, 0, 0, 50).to(torch.int32)
        state["top_p"] = by_kind(1.0, 1.0, 0.95, 0.9)
        state["min_p"] = by_kind(0.0, 0.0, 0.0, 0.02)
        state["u"] = torch.rand(rows, generator=g, device="cuda")
        state["token"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        state["logprob"] = torch.empty(rows, device="cuda")
    else:
        s, t, e = case["seqs"], case["tokens"], case["experts"]
        x = _normal((s, t, e), g) + _normal((e,), g, 0.5)
        state["logits"] = x.to(DTYPES[case["dtype"]])
        state["experts"] = x.topk(case["topk"], dim=2).indices.to(torch.int32)
        state["mask"] = None
        if case["padded"]:   # sequences of their own lengths; one of several has none left
            lengths = torch.randint(0, t + 1, (s, 1), generator=g, device="cuda")
            lengths[s // 2:s // 2 + 1] *= s == 1
            state["mask"] = (torch.arange(t, device="cuda") < lengths).to(torch.uint8)
        state["loss"] = torch.empty(1, device="cuda")
        state["counts"] = torch.empty((s, e), dtype=torch.int32, device="cuda")
        state["dlogits"] = torch.empty_like(state["logits"])
        # scratch that a program keeps for the calls: ample for any of these sizes
        state["workspace"] = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    return state


COEF = 0.01   # weight of the balance loss


# ------------------------------------------------------------------------- plain forms
def _plain_quantize(state):
    case = state["case"]
    b = _blocks(state["x"].float(), case["block_rows"])
    s = (b.abs().amax(dim=(2, 4)) / E4M3_MAX).clamp_min(SCALE_MIN)
    b = (b / s[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    state["q"].copy_(b.view(case["nmat"], -1, b.shape[3] * BLOCK)[:, :case["rows"],
                                                                 :case["cols"]])
    state["scale"].copy_(s)
    return state["q"], state["scale"]


def _values(q, scale, block_rows, k, dtype):
    """What 8-bit values and their scales stand for."""
    s = scale.to(dtype).repeat_interleave(BLOCK, -1)[..., :k]
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, -2)[..., :q.shape[-2], :]
    return q[..., :k].to(dtype) * s


def _product(state, dtype):
    """The product in `dtype`; of each expert's own rows where there are experts."""
    k = state["case"]["k"]
    x = _values(state["x"], state["xs"], 1, k, dtype)
    w = _values(state["w"], state["ws"], BLOCK, k, dtype)
    if state["offsets"] is None:
        return x @ w[0].T
    first, end = state["offsets"][:-1].long(), state["offsets"][1:].long()
    at = torch.arange(state["most"], device="cuda")
    rows = first[:, None] + at                       # expert e's rows, then padding
    y = torch.bmm(x[rows.clamp_max(len(x) - 1)], w.transpose(1, 2))
    row = torch.arange(len(x), device="cuda")
    expert = torch.searchsorted(end, row, right=True)
    return y[expert, row - first[expert]]


def _plain_matmul(state):
    return state["y"].copy_(_product(state, torch.float32))


def _plain_sample(state):
    x = state["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x)
    temperature = state["temperature"]
    greedy = ~(temperature > 0)
    inverse = 1 / torch.where(greedy, 1.0, temperature)
    top = x.amax(1, keepdim=True)
    z = torch.where(x == top, 0.0, (x - top) * inverse[:, None])
    e = torch.where(x == -math.inf, 0.0, z.exp())
    # whole-number weights: their sums do not depend on the order
    w = (e * ONE).round().long()
    total = w.sum(1)
    # rank by logit, ties to the lowest index
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ranked = w.gather(1, order)
    rank = torch.arange(x.shape[1], device=x.device)
    k = torch.where(state["top_k"] > 0, state["top_k"], x.shape[1])[:, None]
    ranked = torch.where(rank < k, ranked, 0)
    before = ranked.cumsum(1) - ranked
    p = state["top_p"][:, None]
    mass = p.double() * ranked.sum(1, keepdim=True).double()
    keep = (rank < k) & ((p >= 1) | (before.double() < mass) | (rank == 0))
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    kept &= e >= state["min_p"][:, None].clamp_max(1.0)
    w = torch.where(kept, w, 0)
    cum = w.cumsum(1)
    target = state["u"].double() * cum[:, -1].double()
    drawn = (cum.double() <= target[:, None]).sum(1)
    highest = (x == top).int().argmax(1)
    token = torch.where(greedy, highest, drawn)
    token = torch.where(top[:, 0] == -math.inf, -1, token)
    at = z.gather(1, token.clamp_min(0)[:, None])[:, 0]
    logprob = at - torch.log1p(((total - ONE).double() / ONE).float())
    state["token"].copy_(token)
    state["logprob"].copy_(torch.where(token < 0, -math.inf, logprob))
    return state["token"], state["logprob"]


def _balance(state, dtype):
    """(loss, counts, gradient) in `dtype`."""
    case = state["case"]
    e = case["experts"]
    x = state["logits"].to(dtype)
    mask = torch.ones(x.shape[:2], dtype=torch.bool, device="cuda")
    if state["mask"] is not None:
        mask = state["mask"] != 0
    if case["score"] == "softmax":
        a = (x - x.amax(2, keepdim=True)).exp()
    else:
        a = 1 / (1 + (-x).exp())
    total = a.sum(2, keepdim=True)
    p = a / total
    slope = p if case["score"] == "softmax" else p * (1 - a)
    chosen = state["experts"][..., None] == torch.arange(e, device="cuda")
    counts = (chosen & mask[:, :, None, None]).sum((1, 2))
    tokens = mask.sum(1).to(dtype)
    n = tokens.clamp_min(1)[:, None]
    f = counts.to(dtype) * e / (case["topk"] * n)
    share = COEF / (tokens > 0).sum().clamp_min(1).to(dtype)
    dot = torch.where(mask, (f[:, None] * p).sum(2), 0)
    loss = share * (dot / n).sum()
    grad = (share / n)[..., None] * slope * (f[:, None] - dot[..., None])
    return loss.reshape(1), counts, torch.where(mask[..., None], grad, 0)


def _plain_balance(state):
    loss, counts, grad = _balance(state, torch.float32)
    state["loss"].copy_(loss)
    state["counts"].copy_(counts)
    state["dlogits"].copy_(grad)
    return state["loss"], state["counts"], state["dlogits"]


# ----------------------------------------------------------------------- the kernels
def _own_quantize(rs, state):
    case = state["case"]
    rs.reshard_fp8_quantize(state["x"], state["q"], state["scale"],
                            (case["nmat"], case["rows"], case["cols"]), case["dtype"],
                            case["block_rows"])
    return state["q"], state["scale"]


def _own_matmul(rs, state):
    case = state["case"]
    pitch = state["x"].shape[1]
    rs.reshard_fp8_matmul(state["x"], state["xs"], state["w"], state["ws"], state["y"],
                          (case["tokens"], case["n"], case["k"]), case["out"],
                          offsets=state["offsets"], nexperts=max(1, case["experts"]),
                          ldx=pitch, ldw=pitch)
    return state["y"]


def _own_sample(rs, state):
    case = state["case"]
    rs.reshard_sample(state["logits"], (case["rows"], case["vocab"]), case["dtype"], state["u"],
                      state["token"], state["logprob"], temperature=state["temperature"],
                      top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
    return state["token"], state["logprob"]


def _own_balance(rs, state):
    case = state["case"]
    rs.reshard_balance_loss(state["logits"], (case["seqs"], case["tokens"], case["experts"]),
                            case["dtype"], state["experts"], case["topk"], COEF,
                            state["workspace"], state["counts"], loss=state["loss"],
                            dlogits=state["dlogits"], mask=state["mask"], score=case["score"])
    return state["loss"], state["counts"], state["dlogits"]


def run(state):
    op = state["case"]["op"]
    if own:
        import dtensor_reshard_gb300 as rs
        return {"quantize": _own_quantize, "matmul": _own_matmul, "sample": _own_sample,
                "balance": _own_balance}[op](rs, state)
    return {"quantize": _plain_quantize, "matmul": _plain_matmul, "sample": _plain_sample,
            "balance": _plain_balance}[op](state)


# ------------------------------------------------------------------------ definitions
def _exact_quantize(state):
    """Per block: scale = largest magnitude / 448; value = nearest e4m3 to x / scale."""
    case = state["case"]
    x = state["x"].double()
    n, r, c = x.shape
    br = case["block_rows"]
    q = torch.empty_like(x, dtype=torch.float32)
    scale = torch.empty_like(state["scale"], dtype=torch.float64)
    for i in range(scale.shape[2]):
        cols = slice(i * BLOCK, min(c, (i + 1) * BLOCK))
        band = torch.nn.functional.pad(x[:, :, cols], (0, 0, 0, up(r, br) - r))
        band = band.reshape(n, -1, br * band.shape[2])
        s = (band.abs().amax(2) / E4M3_MAX).clamp_min(SCALE_MIN)
        scale[:, :, i] = s
        v = (band / s[..., None]).reshape(n, -1, cols.stop - cols.start)[:, :r]
        # e4m3: steps of 2^(exponent - 3), exponents down to -6; halves to even
        step = torch.exp2(torch.frexp(v)[1].clamp_min(-5).double() - 4)
        q[:, :, cols] = ((v / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX).float()
    return q, scale


def _exact_matmul(state):
    x, w = state["x"].double(), state["w"].double()
    k = state["case"]["k"]
    y = torch.zeros(state["y"].shape, dtype=torch.float64, device="cuda")
    ends = [0, len(x)] if state["offsets"] is None else state["offsets"].tolist()
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        for i in range(0, k, BLOCK):
            cols = slice(i, min(k, i + BLOCK))
            ws = state["ws"][e, :, i // BLOCK].double().repeat_interleave(BLOCK)[:y.shape[1]]
            y[a:b] += (x[a:b, cols] * state["xs"][a:b, i // BLOCK, None].double()) @ (
                w[e, :, cols] * ws[:, None]).T
    return y


def _exact_sample(state):
    token, logprob = [], []
    for r, u in enumerate(state["u"].double().tolist()):
        x = state["logits"][r].double().nan_to_num(nan=-math.inf, posinf=math.inf,
                                                   neginf=-math.inf)
        t = float(state["temperature"][r])
        top = float(x.max())
        if top == -math.inf:
            token.append(-1)
            logprob.append(-math.inf)
            continue
        z = torch.where(x == top, 0.0, (x - top) / (t if t > 0 else 1.0))
        e = z.exp()
        if t > 0:
            order = torch.sort(x, dim=0, descending=True, stable=True).indices
            k = int(state["top_k"][r])
            order = order[:k] if k > 0 else order
            p = float(state["top_p"][r])
            if p < 1:
                cum = e[order].cumsum(0)
                order = order[:max(1, int((cum - e[order] < p * cum[-1]).sum()))]
            order = order[e[order] >= min(1.0, float(state["min_p"][r]))].sort().values
            cum = e[order].cumsum(0)
            token.append(int(order[int((cum <= u * cum[-1]).sum())]))
        else:
            token.append(int((x == top).int().argmax()))
        logprob.append(float(z[token[-1]] - e.sum().log()))
    return (torch.tensor(token, dtype=torch.int32),
            torch.tensor(logprob, dtype=torch.float64))


def _exact_balance(state):
    case = state["case"]
    grad = torch.zeros(state["logits"].shape, dtype=torch.float64, device="cuda")
    counts = torch.zeros(state["counts"].shape, dtype=torch.int32, device="cuda")
    masks = [torch.ones(case["tokens"], dtype=torch.bool, device="cuda") if state["mask"] is None
             else state["mask"][s] != 0 for s in range(case["seqs"])]
    live = max(1, sum(bool(m.any()) for m in masks))
    loss = 0.0
    for s, m in enumerate(masks):
        n = int(m.sum())
        if n == 0:
            continue
        x = state["logits"][s][m].double()
        chosen = state["experts"][s][m].flatten().long()
        counts[s] = torch.bincount(chosen, minlength=case["experts"])
        f = counts[s].double() * case["experts"] / (case["topk"] * n)
        if case["score"] == "softmax":
            p = torch.softmax(x, 1)
            slope = p
        else:
            a = torch.sigmoid(x)
            p = a / a.sum(1, keepdim=True)
            slope = p * torch.sigmoid(-x)
        dot = p @ f
        loss += COEF / live * float(dot.sum()) / n
        grad[s, m] = COEF / (live * n) * slope * (f - dot[:, None])
    return torch.tensor([loss], dtype=torch.float64), counts, grad


def exact(case, seed):
    state = prepare(case, seed)
    return {"quantize": _exact_quantize, "matmul": _exact_matmul, "sample": _exact_sample,
            "balance": _exact_balance}[case["op"]](state)


# ------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "quantize":
        n, r, c = case["nmat"], case["rows"], case["cols"]
        blocks = n * cdiv(r, case["block_rows"]) * cdiv(c, BLOCK)
        return {"bytes": n * r * c * (SIZE[case["dtype"]] + 1) + 4 * blocks,
                "flops": 2 * n * r * c}
    if case["op"] == "matmul":
        t, n, k, e = case["tokens"], case["n"], case["k"], max(1, case["experts"])
        e = min(e, t)   # experts without rows need no weights
        return {"bytes": t * k + e * n * k + 4 * cdiv(k, BLOCK) * (t + e * cdiv(n, BLOCK))
                + t * n * SIZE[case["out"]], "flops": 2 * t * n * k}
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * SIZE[case["dtype"]] + 28 * case["rows"], "flops": 4 * n}
    s, t, e = case["seqs"], case["tokens"], case["experts"]
    return {"bytes": s * t * (2 * e * SIZE[case["dtype"]] + 4 * case["topk"] + case["padded"])
            + 4 * s * e, "flops": 8 * s * t * e}
