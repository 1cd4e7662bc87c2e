"""Timed cases of the operators that train and serve on what a refit has moved.

The ranks that generate answer with tokens, and the trainer learns from them.  Timed here is
what lies between a model's last layer and its loss, and between a router and its experts:

  score      the log-probability of one given token a row, the row's entropy, and the most
             likely tokens with their log-probabilities;
  policy     one step of a policy's loss on the logits: log-probabilities and entropies, and
             then the gradient in the logits from given gradients of both;
  distill    the divergence from a teacher's most likely tokens, and its gradient;
  dispatch   each token's row to the places of its experts, sorted by expert, as it is or in
             8 bits with a scale for each 128 values;
  combine    a token's rows back from its experts, weighted and added up, and for training
             also the gradients in the rows and the weights.

``run`` computes them in elementary torch operations, or with the library's kernels where
``own`` is true; ``exact`` computes the same definitions in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126   # a block of zeros gets this scale

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------ cases
def score_case(rows, vocab, dtype, ntop, masked=False):
    """masked: some rows have most of their tokens forbidden, one row all of them."""
    return {"op": "score", "rows": rows, "vocab": vocab, "dtype": dtype, "ntop": ntop,
            "masked": masked}


def policy_case(rows, vocab, dtype, entropy):
    """entropy: the loss has an entropy term too."""
    return {"op": "policy", "rows": rows, "vocab": vocab, "dtype": dtype, "entropy": entropy}


def distill_case(rows, vocab, dtype, ntop, tail):
    """tail: the teacher's remaining probability counts as one more outcome."""
    return {"op": "distill", "rows": rows, "vocab": vocab, "dtype": dtype, "ntop": ntop,
            "tail": tail}


def dispatch_case(tokens, cols, topk, experts, dtype, quantised, dropped):
    """dropped: a tenth of the choices is dropped, as where experts are full."""
    return {"op": "dispatch", "tokens": tokens, "cols": cols, "topk": topk, "experts": experts,
            "dtype": dtype, "quantised": quantised, "dropped": dropped}


def combine_case(tokens, cols, topk, experts, dtype, weighted, training, dropped):
    """weighted false: plain sums, which are also the gradient of a dispatch."""
    return {"op": "combine", "tokens": tokens, "cols": cols, "topk": topk, "experts": experts,
            "dtype": dtype, "weighted": weighted, "training": training, "dropped": dropped}


def listed():
    def named(name, case):
        return {"name": name, **case}
    return [
        # one request's next token with the alternatives that an answer lists: latency
        named("score_one", score_case(1, 131072, "bf16", 20)),
        # odd vocabulary, float32 logits, rows of a grammar that forbids most tokens
        named("score_odd", score_case(37, 50021, "fp32", 5, masked=True)),
        # a teacher's side of distillation: 64 tokens of every row of a batch
        named("score_teacher", score_case(2048, 131072, "bf16", 64)),
        # a short sequence with an entropy term, odd sizes
        named("policy_odd", policy_case(61, 50021, "fp32", True)),
        # a training micro-batch over a large vocabulary
        named("policy_batch", policy_case(4096, 131072, "bf16", False)),
        # a few rows of a small vocabulary, the rest of the teacher's probability as one outcome
        named("distill_odd", distill_case(53, 32003, "fp16", 50, True)),
        # a training micro-batch learning from 64 tokens of every row
        named("distill_batch", distill_case(2048, 131072, "bf16", 64, False)),
        # a decode batch to the places of its 256 experts, in 8 bits for their products
        named("dispatch_decode", dispatch_case(32, 7168, 8, 256, "bf16", True, False)),
        # a prompt batch of the same model
        named("dispatch_prompt", dispatch_case(8192, 7168, 8, 256, "bf16", True, False)),
        # training with full experts, sizes that divide nothing
        named("dispatch_ragged", dispatch_case(4099, 4098, 6, 60, "bf16", False, True)),
        # the decode batch's way back
        named("combine_decode", combine_case(32, 7168, 8, 256, "bf16", True, False, False)),
        # a training batch's way back with its gradients
        named("combine_train", combine_case(4096, 7168, 8, 256, "bf16", True, True, True)),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: most logits, or values of dispatched rows, of a drawn case
_MOST = {"score": 2048 * 131072, "policy": 4096 * 131072, "distill": 2048 * 131072,
         "dispatch": 8192 * 7168 * 8, "combine": 4096 * 7168 * 8}


def draw(rng):
    op = rng.choice(("score", "score", "policy", "distill", "distill", "dispatch", "combine"))
    while True:
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        if op in ("score", "policy", "distill"):
            rows, vocab = _log(rng, 1, 4096), _log(rng, 300, 262144)
            cost = rows * vocab * SIZE[dtype] // 2
            if op == "score":
                case = score_case(rows, vocab, dtype, rng.choice((0, 1, _log(rng, 2, 128))),
                                  rng.random() < 0.3)
            elif op == "policy":
                case = policy_case(rows, vocab, dtype, rng.random() < 0.5)
            else:
                case = distill_case(rows, vocab, dtype, _log(rng, 1, 128), rng.random() < 0.5)
        else:
            tokens, cols, topk = _log(rng, 1, 16384), _log(rng, 64, 8192), rng.randint(1, 8)
            experts = _log(rng, topk + 1, 384)
            cost = tokens * cols * topk * SIZE[dtype] // 2
            dropped = rng.random() < 0.4
            if op == "dispatch":
                case = dispatch_case(tokens, cols, topk, experts, dtype, rng.random() < 0.5, dropped)
            else:
                case = combine_case(tokens, cols, topk, experts, dtype, rng.random() < 0.7,
                                    rng.random() < 0.5, dropped)
        if cost <= _MOST[op]:
            return case


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(std)


def _logits(rows, vocab, g):
    """A head's logits: a wide bulk, and a few tokens that the context makes likely."""
    x = _normal((rows, vocab), g, 2.0)
    n = min(24, vocab)
    likely = torch.rand((rows, n), generator=g, device="cuda").mul_(vocab).long().clamp_max_(vocab - 1)
    return x.scatter_add_(1, likely, 8 + 3 * _normal((rows, n), g))


def _temperature(rows, g):
    """The temperatures that the tokens were drawn at, 0 for greedy ones."""
    kind = torch.randint(0, 4, (rows,), generator=g, device="cuda")
    return torch.tensor([1.0, 0.7, 1.3, 0.0], device="cuda")[kind]


def _inverse(temperature, dtype):
    return 1 / torch.where(temperature > 0, temperature, 1.0).to(dtype)


def _choices(case, g):
    """[tokens, topk] experts, all different in a row, some more popular than others."""
    t, e = case["tokens"], case["experts"]
    popularity = _normal((e,), g)
    chosen = (popularity + _normal((t, e), g)).topk(case["topk"], dim=1).indices.to(torch.int32)
    if case["dropped"]:
        chosen[torch.rand(chosen.shape, generator=g, device="cuda") < 0.1] = -1
    return chosen


def _places(chosen, experts):
    """(place of each choice among all sorted by expert, -1 for dropped ones; first place of
    each expert, and the end)."""
    flat = torch.where((chosen < 0) | (chosen >= experts), experts, chosen).flatten().long()
    order = torch.argsort(flat, stable=True)
    place = torch.empty_like(order)
    place.scatter_(0, order, torch.arange(len(flat), device="cuda"))
    place = torch.where(flat < experts, place, -1).to(torch.int32).view(chosen.shape)
    ends = (flat[:, None] == torch.arange(experts, device="cuda")).sum(0).cumsum(0)
    return place, torch.nn.functional.pad(ends, (1, 0)).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    state = {"case": case}
    if case["op"] in ("score", "policy", "distill"):
        rows, v, dtype = case["rows"], case["vocab"], DTYPES[case["dtype"]]
        x = _logits(rows, v, g)
        state["temperature"] = _temperature(rows, g)
        if case["op"] == "distill":
            # a teacher that mostly agrees, scored beforehand at the same temperature
            k = min(case["ntop"], v)
            y = _normal((rows, v), g).add_(x).mul_(_inverse(state["temperature"], torch.float32)[:, None])
            top = y.topk(k, dim=1)
            state["top_token"] = top.indices.to(torch.int32)
            state["top_logprob"] = top.values - y.logsumexp(1, keepdim=True)
            # padding: rows without a teacher, and lists shorter than the rest
            short = torch.randint(1, k + 1, (rows, 1), generator=g, device="cuda")
            short[torch.rand((rows, 1), generator=g, device="cuda") < 0.8] = k
            short[torch.rand((rows, 1), generator=g, device="cuda") < 0.05] = 0
            short[0] = k
            state["top_token"][torch.arange(k, device="cuda") >= short] = -1
            state["grad"] = torch.rand(rows, generator=g, device="cuda") + 0.5
            state["loss"] = torch.empty(rows, device="cuda")
        else:
            # most targets are likely ones; some rows are padding and have none
            state["target"] = torch.where(
                torch.rand(rows, generator=g, device="cuda") < 0.7, x.argmax(1),
                torch.randint(0, v, (rows,), generator=g, device="cuda")).to(torch.int32)
            state["target"][torch.rand(rows, generator=g, device="cuda") < 0.1] = -1
            state["target"][0] = v // 3
            state["logprob"] = torch.empty(rows, device="cuda")
            state["entropy"] = torch.empty(rows, device="cuda")
        if case["op"] == "score":
            if case["masked"]:
                off = torch.rand((rows, v), generator=g, device="cuda") < 0.99
                off[0] = False
                off[1:2] = True
                off[2::2] = False
                x = x.masked_fill_(off, -math.inf)
                del off
            state["top_token"] = torch.empty((rows, case["ntop"]), dtype=torch.int32, device="cuda")
            state["top_logprob"] = torch.empty((rows, case["ntop"]), device="cuda")
        elif case["op"] == "policy":
            state["dlogprob"] = _normal((rows,), g)
            state["dentropy"] = _normal((rows,), g, 0.01) if case["entropy"] else None
            state["state"] = torch.empty((rows, 4), device="cuda")
        state["logits"] = x.to(dtype)
        if case["op"] != "score":
            state["dlogits"] = torch.empty_like(state["logits"])
        return state
    t, c, k, dtype = case["tokens"], case["cols"], case["topk"], DTYPES[case["dtype"]]
    chosen = _choices(case, g)
    if case["op"] == "dispatch":
        state["experts"] = chosen
        state["x"] = (_normal((t, c), g) * (1 + 20 * (torch.rand((1, c), generator=g, device="cuda")
                                                     > 0.995))).to(dtype)
        state["slot"] = torch.empty((t, k), dtype=torch.int32, device="cuda")
        state["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device="cuda")
        # rows of no expert are left as they are
        if case["quantised"]:
            state["rows"] = torch.zeros((t * k, c), dtype=torch.uint8,
                                        device="cuda").view(torch.float8_e4m3fn)
            state["scale"] = torch.zeros((t * k, cdiv(c, BLOCK)), device="cuda")
        else:
            state["rows"] = torch.zeros((t * k, c), dtype=dtype, device="cuda")
        return state
    state["slot"] = _places(chosen, case["experts"])[0]
    state["rows"] = _normal((t * k, c), g).to(dtype)
    state["weight"] = None
    if case["weighted"]:
        state["weight"] = torch.softmax(_normal((t, k), g), 1)
    state["out"] = torch.empty((t, c), dtype=dtype, device="cuda")
    if case["training"]:
        state["dout"] = _normal((t, c), g).to(dtype)
        state["drows"] = torch.zeros_like(state["rows"])
        state["dweight"] = torch.empty((t, k), device="cuda") if case["weighted"] else None
    return state


# ------------------------------------------------------------------------- plain forms
def _softmax(state):
    """(z, e^z, its sum) of each row's logits over the temperature, z relative to the largest."""
    x = state["logits"].float()
    top = x.amax(1, keepdim=True)
    z = torch.where(x == top, 0.0, (x - top) * _inverse(state["temperature"], torch.float32)[:, None])
    e = torch.where(x == -math.inf, 0.0, z.exp())
    return z, e, e.sum(1)


def _logprob_and_entropy(state, z, e, total):
    target = state["target"].long()
    counts, empty = target >= 0, total == 0
    normal = total.log()
    logprob = z.gather(1, target.clamp_min(0)[:, None])[:, 0] - normal
    entropy = normal - (e * torch.where(e > 0, z, 0.0)).sum(1) / total
    state["logprob"].copy_(torch.where(counts, torch.where(empty, -math.inf, logprob), 0.0))
    state["entropy"].copy_(torch.where(counts & ~empty, entropy, 0.0))
    return normal


def _plain_score(state):
    z, e, total = _softmax(state)
    normal = _logprob_and_entropy(state, z, e, total)
    k = state["top_token"].shape[1]
    x = state["logits"].float()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    short = k - order.shape[1]
    order = torch.nn.functional.pad(order, (0, short))
    there = (x.gather(1, order) > -math.inf) & (state["target"] >= 0)[:, None]
    there &= torch.arange(k, device="cuda") < k - short
    state["top_token"].copy_(torch.where(there, order, -1))
    state["top_logprob"].copy_(torch.where(there, z.gather(1, order) - normal[:, None], -math.inf))
    return state["logprob"], state["entropy"], state["top_token"], state["top_logprob"]


def _plain_policy(state):
    z, e, total = _softmax(state)
    normal = _logprob_and_entropy(state, z, e, total)
    p = e / total[:, None]
    counts = (state["target"] >= 0)[:, None]
    grad = -state["dlogprob"][:, None] * p
    at = state["target"].clamp_min(0).long()[:, None]
    grad.scatter_add_(1, at, state["dlogprob"][:, None])
    if state["dentropy"] is not None:
        slope = z - normal[:, None] + state["entropy"][:, None]
        grad -= state["dentropy"][:, None] * torch.where(p > 0, p * slope, 0.0)
    grad *= _inverse(state["temperature"], torch.float32)[:, None]
    state["dlogits"].copy_(torch.where(counts, grad, 0.0))
    return state["logprob"], state["entropy"], state["dlogits"]


def _plain_distill(state):
    z, e, total = _softmax(state)
    listed_ = state["top_token"] >= 0
    at = state["top_token"].clamp_min(0).long()
    # the loss is a small difference of large terms: in 64 bits
    y = torch.where(listed_, state["top_logprob"].double(), -math.inf)
    q = y.exp()
    member = torch.zeros_like(e, dtype=torch.int32).scatter_add_(1, at, listed_.int()) > 0
    # (where no other token has a probability, the rest has nowhere to be and counts as none)
    outside = torch.where(member, 0.0, e).sum(1)
    if state["case"]["tail"]:
        rest = torch.where(outside > 0, (1 - q.sum(1)).clamp_min(0), 0.0)
        logq = y
    else:
        rest = torch.zeros_like(q[:, 0])
        logq = y - q.sum(1, keepdim=True).log()
        q = q / q.sum(1, keepdim=True)
    some = listed_.any(1)
    logp = z.gather(1, at).double() - total.double().log()[:, None]
    loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
    share = torch.where(rest > 0, rest * total.double() / outside.double(), 0.0)
    loss += torch.where(rest > 0, rest * share.log(), 0.0)
    scale = (state["grad"] * _inverse(state["temperature"], torch.float32))[:, None]
    p = e / total[:, None]
    grad = torch.where(member, p, p * (1 - share).float()[:, None])
    grad.scatter_add_(1, at, -torch.where(listed_, q, 0.0).float())
    state["loss"].copy_(torch.where(some, loss, 0.0))
    state["dlogits"].copy_(torch.where(some[:, None], grad * scale, 0.0))
    return state["loss"], state["dlogits"]


def _plain_dispatch(state):
    case = state["case"]
    place, offsets = _places(state["experts"], case["experts"])
    state["slot"].copy_(place)
    state["offsets"].copy_(offsets)
    n = place.numel()
    flat = place.flatten().long()
    # the choice of each place; places behind the last expert keep what they hold
    choice = torch.zeros(n + 1, dtype=torch.long, device="cuda")
    choice.scatter_(0, torch.where(flat < 0, n, flat), torch.arange(n, device="cuda"))
    token = choice[:n] // case["topk"]
    used = (torch.arange(n, device="cuda") < offsets[-1])[:, None]
    if not case["quantised"]:
        state["rows"].copy_(torch.where(used, state["x"][token], state["rows"]))
        return state["slot"], state["offsets"], state["rows"]
    t, c = state["x"].shape
    x = torch.nn.functional.pad(state["x"].float(), (0, cdiv(c, BLOCK) * BLOCK - c)).view(t, -1, BLOCK)
    scale = (x.abs().amax(2) / E4M3_MAX).clamp_min(SCALE_MIN)
    q = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = q.view(t, -1)[:, :c].contiguous().view(torch.uint8)
    rows = state["rows"].view(torch.uint8)
    rows.copy_(torch.where(used, q[token], rows))
    state["scale"].copy_(torch.where(used, scale[token], state["scale"]))
    return state["slot"], state["offsets"], state["rows"], state["scale"]


def _plain_combine(state):
    case = state["case"]
    slot = state["slot"].long()
    valid = (slot >= 0)[..., None]
    weight = torch.ones(slot.shape, device="cuda") if state["weight"] is None else state["weight"]
    mine = torch.where(valid, state["rows"][slot.clamp_min(0)].float(), 0.0)   # [t, k, c]
    state["out"].copy_((mine * weight[..., None]).sum(1))
    if not case["training"]:
        return (state["out"],)
    dout = state["dout"].float()[:, None]
    n = slot.numel()
    drows = (dout * weight[..., None]).view(n, -1).to(state["drows"].dtype)
    # back to the places: one more row takes what is dropped
    to = torch.where(slot < 0, n, slot).flatten()
    used = torch.zeros(n + 1, dtype=torch.bool, device="cuda").index_fill_(0, to, True)[:n, None]
    placed = torch.zeros((n + 1, drows.shape[1]), dtype=drows.dtype, device="cuda")
    placed.index_copy_(0, to, drows)
    state["drows"].copy_(torch.where(used, placed[:n], state["drows"]))
    if state["dweight"] is None:
        return state["out"], state["drows"]
    state["dweight"].copy_((mine * dout).sum(2))
    return state["out"], state["drows"], state["dweight"]


# ----------------------------------------------------------------------- the kernels
def _own_score(rs, state):
    case = state["case"]
    rs.reshard_logprob(state["logits"], (case["rows"], case["vocab"]), case["dtype"],
                       target=state["target"], logprob=state["logprob"], entropy=state["entropy"],
                       top_token=state["top_token"], top_logprob=state["top_logprob"],
                       ntop=case["ntop"], temperature=state["temperature"])
    return state["logprob"], state["entropy"], state["top_token"], state["top_logprob"]


def _own_policy(rs, state):
    case = state["case"]
    shape = (case["rows"], case["vocab"])
    rs.reshard_logprob(state["logits"], shape, case["dtype"], target=state["target"],
                       logprob=state["logprob"], entropy=state["entropy"], state=state["state"],
                       temperature=state["temperature"])
    rs.reshard_logprob_grad(state["logits"], shape, case["dtype"], state["state"], state["dlogits"],
                            target=state["target"], dlogprob=state["dlogprob"],
                            dentropy=state["dentropy"], temperature=state["temperature"])
    return state["logprob"], state["entropy"], state["dlogits"]


def _own_distill(rs, state):
    case = state["case"]
    rs.reshard_distill_loss(state["logits"], (case["rows"], case["vocab"]), case["dtype"],
                            state["top_token"], state["top_logprob"], state["top_token"].shape[1],
                            loss=state["loss"], dlogits=state["dlogits"], tail=case["tail"],
                            temperature=state["temperature"], grad=state["grad"])
    return state["loss"], state["dlogits"]


def _own_dispatch(rs, state):
    case = state["case"]
    rs.reshard_expert_sort(state["experts"], (case["tokens"], case["topk"]), case["experts"],
                           state["slot"], state["offsets"])
    shape = (case["tokens"], case["topk"], case["cols"])
    if not case["quantised"]:
        rs.reshard_expert_dispatch(state["x"], shape, case["dtype"], state["slot"], state["rows"])
        return state["slot"], state["offsets"], state["rows"]
    rs.reshard_expert_dispatch(state["x"], shape, case["dtype"], state["slot"], state["rows"],
                               scale=state["scale"])
    return state["slot"], state["offsets"], state["rows"], state["scale"]


def _own_combine(rs, state):
    case = state["case"]
    shape = (case["tokens"], case["topk"], case["cols"])
    rs.reshard_expert_combine(state["rows"], shape, case["dtype"], state["slot"], state["out"],
                              weight=state["weight"])
    if not case["training"]:
        return (state["out"],)
    rs.reshard_expert_combine_grad(state["dout"], shape, case["dtype"], state["slot"],
                                   rows=state["rows"] if case["weighted"] else None,
                                   weight=state["weight"], drows=state["drows"],
                                   dweight=state["dweight"])
    if state["dweight"] is None:
        return state["out"], state["drows"]
    return state["out"], state["drows"], state["dweight"]


def run(state):
    op = state["case"]["op"]
    if own:
        import dtensor_reshard_gb300 as rs
        return {"score": _own_score, "policy": _own_policy, "distill": _own_distill,
                "dispatch": _own_dispatch, "combine": _own_combine}[op](rs, state)
    return {"score": _plain_score, "policy": _plain_policy, "distill": _plain_distill,
            "dispatch": _plain_dispatch, "combine": _plain_combine}[op](state)


# ------------------------------------------------------------------------ definitions
_CHUNK = 1 << 25   # logits that are worked on in 64 bits at a time


def _exact_rows(state):
    """(rows, log-softmax over the temperature) of one chunk of rows after another."""
    x, t = state["logits"], state["temperature"]
    n = max(1, _CHUNK // x.shape[1])
    for a in range(0, len(x), n):
        part = slice(a, min(len(x), a + n))
        inverse = torch.where(t[part] > 0, 1 / t[part].double(), 1.0)
        yield part, torch.log_softmax(x[part].double() * inverse[:, None], 1), inverse


def _exact_values(logp, target):
    """(log-probability of the target, entropy) of rows of log-probabilities."""
    empty = logp[:, 0].isnan()
    p = logp.exp()
    logprob = logp.gather(1, target.clamp_min(0).long()[:, None])[:, 0]
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    logprob = torch.where(empty, -math.inf, logprob)
    entropy = torch.where(empty, 0.0, entropy)
    return torch.where(target < 0, 0.0, logprob), torch.where(target < 0, 0.0, entropy)


def _exact_score(state):
    k, v = state["top_token"].shape[1], state["logits"].shape[1]
    outs = []
    for part, logp, _ in _exact_rows(state):
        target = state["target"][part]
        x = state["logits"][part].double()
        token = torch.full((len(x), k), -1, dtype=torch.int32, device="cuda")
        value = torch.full((len(x), k), -math.inf, dtype=torch.float64, device="cuda")
        # whole numbers in the order of the logits, the lower index first among equal ones
        rank = torch.unique(x, return_inverse=True)[1] * v + (v - 1 - torch.arange(v, device="cuda"))
        best = rank.topk(min(k, v), dim=1).indices if k else rank[:, :0]
        ok = (x.gather(1, best) > -math.inf) & (target >= 0)[:, None]
        token[:, :best.shape[1]] = torch.where(ok, best, -1).to(torch.int32)
        value[:, :best.shape[1]] = torch.where(ok, logp.gather(1, best), -math.inf)
        outs.append((*_exact_values(logp, target), token, value))
    return tuple(torch.cat(o) for o in zip(*outs))


def _exact_policy(state):
    outs = []
    for part, logp, inverse in _exact_rows(state):
        target = state["target"][part]
        logprob, entropy = _exact_values(logp, target)
        p = logp.exp()
        g = state["dlogprob"][part].double() * inverse * (target >= 0)
        grad = p * -g[:, None]
        grad[torch.arange(len(p), device="cuda"), target.clamp_min(0).long()] += g
        if state["dentropy"] is not None:
            h = state["dentropy"][part].double() * inverse * (target >= 0)
            grad -= p * (torch.where(p > 0, logp, 0.0) + entropy[:, None]) * h[:, None]
        outs.append((logprob, entropy, grad))
    return tuple(torch.cat(o) for o in zip(*outs))


def _exact_distill(state):
    loss, grads = [], []
    for part, logp, inverse in _exact_rows(state):
        token, y = state["top_token"][part].long(), state["top_logprob"][part].double()
        g = state["grad"][part].double() * inverse
        # the teacher's and the student's distributions over all tokens
        q = torch.zeros_like(logp)
        inside = torch.zeros_like(logp, dtype=torch.bool)
        for j in range(token.shape[1]):
            r = torch.nonzero(token[:, j] >= 0)[:, 0]
            q[r, token[r, j]] += y[r, j].exp()
            inside[r, token[r, j]] = True
        some = inside.any(1)
        p = logp.exp()
        if not state["case"]["tail"]:
            q = torch.where(some[:, None], q / q.sum(1, keepdim=True), 0.0)
            rest = torch.zeros_like(q[:, 0])
        else:
            rest = (1 - q.sum(1)).clamp_min(0) * some
        outside = torch.where(inside, 0.0, p).sum(1)
        rest = torch.where(outside > 0, rest, 0.0)
        kl = torch.where(q > 0, q * (q.log() - logp), 0.0).sum(1)
        kl += torch.where(rest > 0, rest * (rest / outside).log(), 0.0)
        other = p * torch.where(rest > 0, 1 - rest / outside, 1.0)[:, None]
        grad = torch.where(inside, p - q, other) * (g * some)[:, None]
        loss.append(torch.where(some, kl, 0.0))
        grads.append(grad)
    return torch.cat(loss), torch.cat(grads)


def _exact_dispatch(state):
    case = state["case"]
    experts, k = state["experts"].flatten().tolist(), case["topk"]
    by_expert = [[] for _ in range(case["experts"])]
    for i, e in enumerate(experts):
        if 0 <= e < case["experts"]:
            by_expert[e].append(i)
    slot = torch.full((len(experts),), -1, dtype=torch.int32)
    offsets, order = [0], []
    for mine in by_expert:
        order += mine
        offsets.append(len(order))
    slot[torch.tensor(order, dtype=torch.long)] = torch.arange(len(order), dtype=torch.int32)
    offsets = torch.tensor(offsets, dtype=torch.int32)
    slot = slot.view(-1, k)
    token = (torch.tensor(order, dtype=torch.long) // k).cuda()
    x = state["x"].double()
    if not case["quantised"]:
        rows = torch.zeros(state["rows"].shape, dtype=torch.float64, device="cuda")
        rows[:len(order)] = x[token]
        return slot, offsets, rows
    rows = torch.zeros(state["rows"].shape, dtype=torch.float32, device="cuda")
    scale = torch.zeros(state["scale"].shape, dtype=torch.float64, device="cuda")
    for i in range(scale.shape[1]):
        block = x[:, i * BLOCK:(i + 1) * BLOCK]
        s = (block.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
        v = block / s[:, None]
        # e4m3: steps of 2^(exponent - 3), exponents down to -6; halves to even
        step = torch.exp2(torch.frexp(v)[1].clamp_min(-5).double() - 4)
        v = ((v / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX).float()
        rows[:len(order), i * BLOCK:(i + 1) * BLOCK] = v[token]
        scale[:len(order), i] = s[token]
    return slot, offsets, rows, scale


def _exact_combine(state):
    case, slot = state["case"], state["slot"]
    out = torch.zeros(state["out"].shape, dtype=torch.float64, device="cuda")
    training = case["training"]
    if training:
        drows = torch.zeros(state["drows"].shape, dtype=torch.float64, device="cuda")
        dweight = torch.zeros(slot.shape, dtype=torch.float64, device="cuda")
        dout = state["dout"].double()
    for j in range(case["topk"]):
        t = torch.nonzero(slot[:, j] >= 0)[:, 0]
        at = slot[t, j].long()
        w = 1.0 if state["weight"] is None else state["weight"][t, j, None].double()
        row = state["rows"][at].double()
        out[t] += w * row
        if training:
            drows[at] = w * dout[t]
            dweight[t, j] = (dout[t] * row).sum(1)
    if not training:
        return (out,)
    return (out, drows) if state["dweight"] is None else (out, drows, dweight)


def exact(case, seed):
    state = prepare(case, seed)
    return {"score": _exact_score, "policy": _exact_policy, "distill": _exact_distill,
            "dispatch": _exact_dispatch, "combine": _exact_combine}[case["op"]](state)


# ------------------------------------------------------------------------------- work
def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] in ("score", "policy", "distill"):
        rows, n = case["rows"], case["rows"] * case["vocab"]
        if case["op"] == "score":
            return {"bytes": n * size + rows * (16 + 8 * case["ntop"]), "flops": 6 * n}
        if case["op"] == "policy":
            return {"bytes": 2 * n * size + rows * 24, "flops": (14 if case["entropy"] else 11) * n}
        return {"bytes": 2 * n * size + rows * (12 + 8 * case["ntop"]), "flops": 9 * n}
    t, c, k = case["tokens"], case["cols"], case["topk"]
    kept = t * k * (9 if case["dropped"] else 10) // 10
    if case["op"] == "dispatch":
        row = c + 4 * cdiv(c, BLOCK) if case["quantised"] else c * size
        return {"bytes": t * c * size + kept * row + 8 * t * k + 4 * case["experts"],
                "flops": 2 * t * c if case["quantised"] else 0}
    once = kept * c * size + t * c * size + t * k * (8 if case["weighted"] else 4)
    if not case["training"]:
        return {"bytes": once, "flops": 2 * kept * c}
    return {"bytes": once + (t * c + kept * c) * size + (4 * t * k if case["weighted"] else 0),
            "flops": (5 if case["weighted"] else 1) * kept * c}
