"""One training step of a small mixture-of-experts layer on what a rollout drew, on one GPU.

The teacher is the layer as the generating ranks hold it, in 8 bits: it routes the tokens, multiplies
them with its experts, draws each one's successor, and lists its most likely tokens.  The student
learns from both: it comes nearer to the teacher's list, and a policy term raises or lowers the drawn
tokens' log-probabilities by their advantages.  The gradients go back through the experts to the
layer's input, its weights and its gates.  Run it with ``python examples/distill_step.py``.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dtensor_reshard_gb300 as rs  # noqa: E402

EXPERTS, FFN, HIDDEN = 8, 256, 384     # one weight [FFN, HIDDEN] an expert
VOCAB, TOKENS, TOPK, LISTED = 1003, 90, 2, 16


def order(choices):
    """(places of the choices, first place of each expert) of the router's choices [TOKENS, TOPK]."""
    slot = torch.empty_like(choices)
    offsets = torch.empty(EXPERTS + 1, dtype=torch.int32, device="cuda")
    rs.reshard_expert_sort(choices, (TOKENS, TOPK), EXPERTS, slot, offsets)
    return slot, offsets


def teacher_logits(x, weights, head, slot, offsets, gate):
    """Logits of the layer in 8 bits: rows to their experts' places, products, and back."""
    q, s = (torch.empty(EXPERTS, FFN, HIDDEN, dtype=torch.uint8, device="cuda"),
            torch.empty(EXPERTS, FFN // 128, HIDDEN // 128, device="cuda"))
    rs.reshard_fp8_quantize(weights, q, s, (EXPERTS, FFN, HIDDEN), "fp32", block_rows=128)
    n = TOKENS * TOPK
    rows, scale = (torch.empty(n, HIDDEN, dtype=torch.uint8, device="cuda"),
                   torch.empty(n, HIDDEN // 128, device="cuda"))
    rs.reshard_expert_dispatch(x, (TOKENS, TOPK, HIDDEN), "fp32", slot, rows, scale=scale)
    y = torch.empty(n, FFN, device="cuda")
    rs.reshard_fp8_matmul(rows, scale, q, s, y, (n, FFN, HIDDEN), "fp32", offsets=offsets, nexperts=EXPERTS)
    out = torch.empty(TOKENS, FFN, device="cuda")
    rs.reshard_expert_combine(y, (TOKENS, TOPK, FFN), "fp32", slot, out, weight=gate)
    return out @ head


def rollout(logits, u, temperature):
    """Each row's drawn token, and the teacher's LISTED most likely ones with log-probabilities."""
    shape = (TOKENS, VOCAB)
    drawn = torch.empty(TOKENS, dtype=torch.int32, device="cuda")
    rs.reshard_sample(logits, shape, "fp32", u, drawn, temperature=temperature)
    token = torch.empty(TOKENS, LISTED, dtype=torch.int32, device="cuda")
    logprob = torch.empty(TOKENS, LISTED, device="cuda")
    rs.reshard_logprob(logits, shape, "fp32", top_token=token, top_logprob=logprob, ntop=LISTED,
                       temperature=temperature)
    return drawn, token, logprob


def per_expert(offsets):
    ends = offsets.tolist()
    return [slice(a, b) for a, b in zip(ends, ends[1:])]


def student_step(x, weights, head, slot, offsets, gate, temperature, drawn, token, logprob, advantage, bonus):
    """Losses of the step and the gradients of their sum: the divergence from the teacher, minus
    advantage times the drawn token's log-probability, minus bonus times the entropy, summed over rows."""
    hidden, ffn, shape = (TOKENS, TOPK, HIDDEN), (TOKENS, TOPK, FFN), (TOKENS, VOCAB)
    # forward
    rows = torch.empty(TOKENS * TOPK, HIDDEN, device="cuda")
    rs.reshard_expert_dispatch(x, hidden, "fp32", slot, rows)
    y = torch.empty(TOKENS * TOPK, FFN, device="cuda")
    for e, part in enumerate(per_expert(offsets)):
        y[part] = rows[part] @ weights[e].T
    out = torch.empty(TOKENS, FFN, device="cuda")
    rs.reshard_expert_combine(y, ffn, "fp32", slot, out, weight=gate)
    logits = out @ head
    # losses and their gradients in the logits
    divergence, dlogits = torch.empty(TOKENS, device="cuda"), torch.empty_like(logits)
    rs.reshard_distill_loss(logits, shape, "fp32", token, logprob, LISTED, loss=divergence, dlogits=dlogits,
                            tail=True, temperature=temperature)
    score, entropy = torch.empty(TOKENS, device="cuda"), torch.empty(TOKENS, device="cuda")
    state = torch.empty(TOKENS, 4, device="cuda")
    rs.reshard_logprob(logits, shape, "fp32", target=drawn, logprob=score, entropy=entropy, state=state,
                       temperature=temperature)
    rs.reshard_logprob_grad(logits, shape, "fp32", state, logits, target=drawn, dlogprob=-advantage,
                            dentropy=torch.full_like(entropy, -bonus), temperature=temperature)
    dlogits += logits                      # (the logits' place holds the policy's gradient now)
    # and back through the layer
    dhead, dout = out.T @ dlogits, dlogits @ head.T
    dy, dgate = torch.empty_like(y), torch.empty_like(gate)
    rs.reshard_expert_combine_grad(dout, ffn, "fp32", slot, rows=y, weight=gate, drows=dy, dweight=dgate)
    dweights, drows = torch.empty_like(weights), torch.empty_like(rows)
    for e, part in enumerate(per_expert(offsets)):
        dweights[e] = dy[part].T @ rows[part]
        drows[part] = dy[part] @ weights[e]
    dx = torch.empty_like(x)
    rs.reshard_expert_combine(drows, hidden, "fp32", slot, dx)
    return {"divergence": divergence, "score": score, "entropy": entropy, "dx": dx, "dweights": dweights,
            "dgate": dgate, "dhead": dhead}


def main(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std
    x, weights, head = normal(TOKENS, HIDDEN), normal(EXPERTS, FFN, HIDDEN, std=0.05), normal(FFN, VOCAB, std=0.1)
    router = normal(TOKENS, EXPERTS)
    choices = router.topk(TOPK, dim=1).indices.to(torch.int32)
    gate = torch.softmax(router.gather(1, choices.long()), dim=1)
    temperature = torch.full((TOKENS,), 0.8, device="cuda")
    slot, offsets = order(choices)
    teacher = teacher_logits(x, weights + normal(*weights.shape, std=0.02), head, slot, offsets, gate)
    drawn, token, logprob = rollout(teacher, torch.rand(TOKENS, generator=g, device="cuda"), temperature)
    advantage, bonus = normal(TOKENS), 0.01
    out = student_step(x, weights, head, slot, offsets, gate, temperature, drawn, token, logprob, advantage, bonus)
    out.update(x=x, weights=weights, head=head, choices=choices, gate=gate, temperature=temperature, drawn=drawn,
               token=token, logprob=logprob, advantage=advantage, bonus=bonus, teacher=teacher)
    return out


if __name__ == "__main__":
    out = main()
    print("divergence from the teacher", float(out["divergence"].mean()), "entropy", float(out["entropy"].mean()))
    print("gradients' norms", {k: round(float(out[k].norm()), 4) for k in ("dx", "dweights", "dgate", "dhead")})
