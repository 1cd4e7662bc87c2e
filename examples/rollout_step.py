"""One refit and one generation step of a small mixture-of-experts layer, on one GPU.

The trainer holds the experts' weights sharded over experts; the ranks that generate hold
them sharded over the features, in 8 bits.  The refit quantises on the trainer's side and
reshards bytes and scales; then a step routes tokens, multiplies them with the refitted
experts, and draws each token's successor.  Run it with ``python examples/rollout_step.py``.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dtensor_reshard_gb300 as rs  # noqa: E402

EXPERTS, FFN, HIDDEN = 8, 512, 384     # one weight [FFN, HIDDEN] an expert
EP, TP = 4, 2                          # trainer: experts over 4 ranks; generator: FFN over 2
VOCAB, TOKENS, TOPK = 1000, 96, 2


def refit(weights):
    """weights[r] [EXPERTS / EP, FFN, HIDDEN] bf16 of trainer rank r -> for each generating
    rank (8-bit weights [EXPERTS, FFN / TP, HIDDEN], scales [EXPERTS, FFN / TP / 128, HIDDEN / 128])."""
    values, scales = [], []
    for w in weights:
        q = torch.empty(w.shape, dtype=torch.uint8, device="cuda")
        s = torch.empty((w.shape[0], FFN // 128, HIDDEN // 128), device="cuda")
        rs.reshard_fp8_quantize(w, q, s, tuple(w.shape), "bf16", block_rows=128)
        values.append(q)
        scales.append(s)
    out = []
    for srcs, shape, dtype in ((values, (EXPERTS, FFN, HIDDEN), "u8"),
                               (scales, (EXPERTS, FFN // 128, HIDDEN // 128), "fp32")):
        plan = rs.reshard_plan_create(shape, dtype, (EP,), ("S0",), (TP,), ("S1",))
        dsts = [torch.empty(rs.reshard_plan_local_shape(plan, 1, r)[0], dtype=srcs[0].dtype,
                            device="cuda") for r in range(TP)]
        rs.reshard_execute(plan, srcs, dsts)
        out.append(dsts)
    return list(zip(*out))


def route(router_logits):
    """(choices [TOKENS, TOPK], loss, gradient, tokens of each expert) of the router."""
    choices = router_logits.topk(TOPK, dim=1).indices.to(torch.int32)
    shape = (1, TOKENS, EXPERTS)
    workspace = torch.empty(rs.reshard_balance_loss_workspace(shape), dtype=torch.uint8, device="cuda")
    counts = torch.empty(EXPERTS, dtype=torch.int32, device="cuda")
    loss, grad = torch.empty(1, device="cuda"), torch.empty_like(router_logits)
    rs.reshard_balance_loss(router_logits, shape, "fp32", choices, TOPK, 0.01, workspace, counts,
                            loss=loss, dlogits=grad)
    return choices, loss, grad, counts


def experts(x, choices, counts, ranks):
    """Each choice's product [TOKENS, TOPK, FFN], computed by expert on every rank's features."""
    order = choices.flatten().argsort(stable=True)           # rows sorted by expert
    rows = x[order // TOPK].contiguous()
    q = torch.empty(rows.shape, dtype=torch.uint8, device="cuda")
    s = torch.empty((len(rows), HIDDEN // 128), device="cuda")
    rs.reshard_fp8_quantize(rows, q, s, tuple(rows.shape), "bf16")
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    parts = []
    for w, ws in ranks:
        y = torch.empty((len(rows), FFN // TP), dtype=torch.bfloat16, device="cuda")
        rs.reshard_fp8_matmul(q, s, w, ws, y, (len(rows), FFN // TP, HIDDEN), "bf16",
                              offsets=offsets, nexperts=EXPERTS)
        parts.append(y)
    y = torch.empty((len(rows), FFN), dtype=torch.bfloat16, device="cuda")
    y[order] = torch.cat(parts, dim=1)
    return y.view(TOKENS, TOPK, FFN)


def sample(logits, u):
    token = torch.empty(TOKENS, dtype=torch.int32, device="cuda")
    logprob = torch.empty(TOKENS, device="cuda")
    temperature = torch.full((TOKENS,), 0.8, device="cuda")
    top_p = torch.full((TOKENS,), 0.95, device="cuda")
    rs.reshard_sample(logits, (TOKENS, VOCAB), "bf16", u, token, logprob, temperature=temperature,
                      top_p=top_p)
    return token, logprob


def main(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std
    weights = [normal(EXPERTS // EP, FFN, HIDDEN, std=0.05).bfloat16() for _ in range(EP)]
    x = normal(TOKENS, HIDDEN).bfloat16()
    router_logits = normal(TOKENS, EXPERTS)
    head = normal(FFN, VOCAB, std=0.05).bfloat16()
    ranks = refit(weights)
    choices, loss, grad, counts = route(router_logits)
    y = experts(x, choices, counts, ranks)
    gate = torch.softmax(router_logits.gather(1, choices.long()), dim=1).bfloat16()
    logits = (y * gate[..., None]).sum(1) @ head
    token, logprob = sample(logits, torch.rand(TOKENS, generator=g, device="cuda"))
    return {"weights": torch.cat(weights), "x": x, "router_logits": router_logits,
            "choices": choices, "loss": loss, "grad": grad, "counts": counts, "y": y,
            "logits": logits, "token": token, "logprob": logprob}


if __name__ == "__main__":
    out = main()
    print("tokens of each expert", out["counts"].tolist(), "balance loss", float(out["loss"]))
    print("drawn", out["token"][:8].tolist(), "log-probabilities", out["logprob"][:8].tolist())
