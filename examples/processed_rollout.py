"""A rollout under a sampler's rules, and the trainer's step on it.

An engine decodes a batch of requests from a small random head: every step's
logits go through `process_logits` (penalties for repeated tokens, biases,
temperature, a grammar for every other request) and the next tokens are drawn
from them.  The trainer then scores the packed sequences under the same rules
(`processed_logprob`), compares the two sides (`mismatch_stats`), takes the
TIS-weighted PPO surrogate's gradient through the rules
(`processed_logprob_backward`) and adds a distillation term from a teacher's top
logits (`distill_topk_step`).  For comparison it also scores the tokens without
the rules: that mismatch is what a trainer sees that forgets them.

    python examples/processed_rollout.py          # on a GB300
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import rollout_logprob_mismatch_gb300 as tim  # noqa: E402


def draw_rules(B, V, gen, dev):
    """Per-request rules: parameters, three biased ids each, two grammars."""
    uniform = lambda lo, hi: torch.rand(B, generator=gen, device=dev) * (hi - lo) + lo   # noqa: E731
    return {
        "temperature": uniform(0.7, 1.1), "repetition": uniform(1.0, 1.3), "presence": uniform(0.0, 0.6),
        "frequency": uniform(0.0, 0.3),
        "bias_ids": (torch.arange(3, device=dev) * (V // 3) + torch.arange(B, device=dev).view(-1, 1)).int(),
        "bias_values": torch.randn(B, 3, generator=gen, device=dev),
        # bit v of a grammar: all ids but the multiples of 7, or the even ids only
        "allowed": torch.stack([_bits(torch.arange(V, device=dev) % 7 != 0), _bits(torch.arange(V, device=dev) % 2 == 0)]),
        "grammar": torch.where(torch.arange(B, device=dev) % 2 == 0, -1, torch.arange(B, device=dev) // 2 % 2).int(),
    }


def _bits(keep):
    V = keep.numel()
    w = torch.zeros((V + 31) // 32 * 32, dtype=torch.int64, device=keep.device)
    w[:V] = keep.long()
    w = (w.view(-1, 32) << torch.arange(32, device=keep.device)).sum(1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).int()


def rows_of(rules, rows, history, spans):
    """The LogitsRules of logits rows that belong to requests `rows`."""
    n = rows.numel()
    return tim.LogitsRules(
        temperature=rules["temperature"][rows], repetition=rules["repetition"][rows],
        presence=rules["presence"][rows], frequency=rules["frequency"][rows], history=history, history_spans=spans,
        bias_offsets=(torch.arange(n + 1, device=rows.device) * 3).int(),
        bias_ids=rules["bias_ids"][rows].reshape(-1), bias_values=rules["bias_values"][rows].reshape(-1),
        allowed=rules["allowed"], allowed_rows=rules["grammar"][rows])


def main(B=8, prompt=12, steps=40, V=1024, D=256, K=16, seed=0):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    E = torch.randn(V, D, generator=gen, device=dev)                  # a token's hidden state
    W = torch.randn(V, D, generator=gen, device=dev) * 0.12           # the head
    rules = draw_rules(B, V, gen, dev)
    every = torch.arange(B, device=dev)

    # the engine: one token per request and step
    T = prompt + steps
    tokens = torch.zeros(B, T, dtype=torch.int32, device=dev)
    tokens[:, :prompt] = torch.randint(0, V, (B, prompt), generator=gen, device=dev).int()
    rollout = torch.zeros(B, T, device=dev)
    begin = every * T
    for t in range(prompt, T):
        spans = torch.stack([begin, begin + prompt, begin + t], 1).int()
        logits = E[tokens[:, t - 1].long()] @ W.t()
        tim.process_logits(logits, rows_of(rules, every, tokens.view(-1), spans), out=logits)   # in place
        logp = torch.log_softmax(logits, 1)
        drawn = torch.multinomial(logp.exp(), 1, generator=gen)
        tokens[:, t] = drawn.view(-1).int()
        rollout[:, t] = logp.gather(1, drawn).view(-1)

    # the trainer: position t of a sequence predicts token t + 1
    inputs, targets = tokens[:, :-1].reshape(-1).contiguous(), tokens[:, 1:].reshape(-1).contiguous()
    l_rollout = rollout[:, 1:].reshape(-1).contiguous()
    S = T - 1
    N = B * S
    offsets = (torch.arange(B + 1, device=dev) * S).int()
    mask = (torch.arange(S, device=dev) >= prompt - 1).repeat(B).to(torch.uint8)
    request = torch.arange(N, device=dev) // S
    spans = tim.packed_spans(offsets, torch.full((B,), prompt, dtype=torch.int32, device=dev), N)
    h = E[inputs.long()]
    z = h @ W.t()
    under = rows_of(rules, request, inputs, spans)
    l_old, _ = tim.processed_logprob(z, under, targets)
    stats = tim.mismatch_stats(l_old, l_rollout, mask, offsets)
    without, _ = tim.processed_logprob(z, None, targets)
    forgot = tim.mismatch_stats(without, l_rollout, mask, offsets)

    # one update: a slightly moved head, the surrogate's gradient through the rules
    # and a distillation term towards a teacher that knows the old head's top logits
    W2 = W + torch.randn(V, D, generator=gen, device=dev) * 0.002
    z2 = h @ W2.t()
    l_theta, lse = tim.processed_logprob(z2, under, targets)
    advantages = torch.randn(B, generator=gen, device=dev).repeat_interleave(S)
    ppo = tim.tis_ppo(l_theta, l_old, l_rollout, advantages, mask, offsets)
    weight = mask.float() / mask.sum()
    dz = tim.processed_logprob_backward(z2, under, targets, ppo["token_grad"] * weight, lse)
    top = torch.topk(z, K, dim=1)
    kd = tim.distill_topk_step(z2, top.indices.int().contiguous(), top.values.contiguous(), weight,
                               teacher_lse=torch.logsumexp(z, 1))
    dW = (dz + kd["dlogits"]).t() @ h
    tim.check()
    i = tim.BATCH_FIELDS.index("mean_abs_delta")
    return {
        "tokens": int(mask.sum()), "mean_abs_delta": stats["batch"][i].item(),
        "mean_abs_delta_without_the_rules": forgot["batch"][i].item(),
        "ppo_loss": ppo["batch"][tim.PPO_FIELDS.index("mean_loss")].item(),
        "distill_loss": float((kd["loss"] * weight).sum()), "grad_norm": float(dW.norm()), "dW": dW, "sampled": tokens,
        "kd": kd, "z2": z2, "weight": weight,
    }


if __name__ == "__main__":
    for k, v in main().items():
        if not isinstance(v, (torch.Tensor, dict)):
            print("%-34s %s" % (k, v))
