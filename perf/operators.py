"""The operators on a head's logits, as cases that can be timed and compared.

Three operators that take the logits [N, V] of a vocabulary head:

  process        the sampler's side: sparse biases, penalties for repeated
                 tokens, temperature and a grammar mask, written as logits;
  logprob        the trainer's side: the log-probability of the chosen token
                 under those processed logits, which are not written, and its
                 gradient with respect to the raw logits;
  distill        distillation from a teacher's top logits: the loss, its
                 gradient, and both in one call.

With the module's ``own`` false, `run` computes them from elementary torch
operations in fp32; with ``own`` true it calls this library.  `exact` is the
definition in fp64, row block by row block.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


# ----------------------------------------------------------------------------- cases
def _process(name, N, V, dtype, out, hist_median, hist_max, bias, masked, sharp):
    """hist_median / hist_max: tokens of a row's history (lognormal, clipped);
    bias: biased ids of a row that has any (every other row); masked: fraction
    of rows under a grammar; sharp: ids a grammar allows (0: half of them)."""
    return {"name": name, "op": "process", "N": N, "V": V, "dtype": dtype, "out": out, "hist_median": hist_median,
            "hist_max": hist_max, "bias": bias, "masked": masked, "sharp": sharp}


def _logprob(name, N, V, dtype, backward, seq_len, prompt, ragged, bias, masked):
    """Rows are the positions of packed sequences of about seq_len tokens
    (ragged: lognormal lengths), the first `prompt` of each the prompt."""
    return {"name": name, "op": "logprob_backward" if backward else "logprob", "N": N, "V": V, "dtype": dtype,
            "seq_len": seq_len, "prompt": prompt, "ragged": ragged, "bias": bias, "masked": masked}


def _distill(name, what, N, V, dtype, K, tail, holes):
    """what: forward, backward or step; tail: the teacher's mass outside its K
    ids is one more outcome; holes: rows list fewer than K ids."""
    return {"name": name, "op": "distill_" + what, "N": N, "V": V, "dtype": dtype, "K": K, "tail": tail,
            "holes": holes}


def listed():
    return [
        # one request in a decoding engine: latency is what counts
        _process("process_one_row", 1, 151936, "f32", "f32", 700, 700, 16, 0.0, 0),
        # a decoding batch whose sampler works in fp32: half of the requests under a grammar
        _process("process_batch", 64, 128256, "bf16", "f32", 1024, 4096, 32, 0.5, 0),
        # a large decoding batch with long contexts
        _process("process_large", 512, 151936, "bf16", "bf16", 1024, 8192, 8, 0.25, 0),
        # a vocabulary of odd size (rows start at odd offsets), every request under a tight grammar
        _process("process_odd", 77, 50261, "f16", "f16", 300, 2000, 5, 1.0, 12),
        # the smallest head of the benchmark, one sequence
        _logprob("logprob_tiny", 64, 1024, "f32", False, 64, 16, False, 4, 0.0),
        # a trainer's batch of 16 sequences of 512, prompts of 128, all rules but the mask
        _logprob("logprob_packed", 8192, 151936, "bf16", False, 512, 128, False, 0, 0.0),
        # the gradient on packed sequences of different lengths, some under a grammar
        _logprob("logprob_backward_packed", 4096, 128256, "bf16", True, 1024, 128, True, 8, 0.25),
        # the same on fp32 logits of an odd vocabulary
        _logprob("logprob_backward_odd", 333, 32003, "f32", True, 100, 20, True, 3, 0.5),
        # the loss alone (a validation pass), odd sizes
        _distill("distill_forward_odd", "forward", 500, 50261, "f16", 20, False, True),
        # a training step's loss and gradient in one call
        _distill("distill_step", "step", 4096, 151936, "bf16", 64, False, False),
        # the same with the tail outcome, fp32 logits, rows with fewer ids
        _distill("distill_step_tail", "step", 1024, 129280, "f32", 128, True, True),
        # the gradient for a handful of rows with many ids each
        _distill("distill_backward_few", "backward", 7, 151936, "bf16", 256, True, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    V = _log_int(rng, 1000, 152000)
    if rng.random() < 0.6:
        V = (V + 63) // 64 * 64
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    op = rng.choice(["process", "logprob", "logprob_backward", "distill_forward", "distill_step", "distill_backward"])
    top = 512 if op == "process" else 4096
    N = min(_log_int(rng, 1, top), max(1, 300000000 // V))
    if op == "process":
        med = _log_int(rng, 4, 2000)
        return _process("", N, V, dtype, rng.choice([dtype, "f32"]), med, min(8192, 4 * med), rng.choice([0, 1, 8, 40]),
                        rng.choice([0.0, 0.3, 1.0]), rng.choice([0, 0, 3, 200]))
    if op.startswith("logprob"):
        length = _log_int(rng, 8, 1500)
        return _logprob("", N, V, dtype, op == "logprob_backward", length, rng.randrange(0, length // 2 + 1),
                        rng.random() < 0.7, rng.choice([0, 1, 6]), rng.choice([0.0, 0.3, 1.0]))
    return _distill("", op[len("distill_"):], N, V, dtype, min(_log_int(rng, 1, 300), V // 2), rng.random() < 0.5,
                    rng.random() < 0.5)


# ----------------------------------------------------------------------------- inputs
def _lengths(g, n, median, most):
    return np.clip(np.exp(g.normal(math.log(median), 0.5, n)), 1, most).astype(np.int64)


def _tokens(gen, n, V, dev):
    # repeats as in text: a few ids often, most of them hardly ever
    return (torch.rand(n, generator=gen, device=dev) ** 4 * V).to(torch.int32).clamp_(max=V - 1)


def _bits_of(ids, words, dev):
    """Bitmask rows (int32 [R, words]) with the bits ids [R, k] set."""
    m = torch.zeros((ids.shape[0], words * 32), dtype=torch.bool, device=dev)
    m.scatter_(1, ids.long(), True)
    w = m.view(ids.shape[0], words, 32).long() << torch.arange(32, device=dev)
    w = w.sum(2)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def _rules(case, g, gen, dev, targets=None, spans=None, history=None):
    """The processing rules of a case's rows: what a sampler keeps per request
    (and a trainer per position)."""
    N, V = case["N"], case["V"]
    r = {}
    if spans is None:
        lens = _lengths(g, N, case["hist_median"], case["hist_max"])
        if N > 4:
            lens[g.integers(N)] = 0           # a request that has nothing behind it
        begin = np.concatenate([[0], np.cumsum(lens)[:-1]])
        spans = np.stack([begin, begin + (lens * g.uniform(0.1, 0.9, N)).astype(np.int64), begin + lens], 1)
        history = _tokens(gen, max(1, int(lens.sum())), V, dev)
    r["history"] = history
    r["history_spans"] = torch.from_numpy(spans.astype(np.int32)).to(dev)
    rows = lambda x: torch.from_numpy(x.astype(np.float32)).to(dev)   # noqa: E731
    r["repetition"] = rows(g.choice([1.0, 1.05, 1.2], N))
    r["presence"] = rows(g.choice([0.0, 0.5, 1.0], N))
    r["frequency"] = rows(g.choice([0.0, 0.1, 0.3], N))
    r["temperature"] = rows(g.uniform(0.6, 1.2, N))
    if case["bias"]:
        k = min(case["bias"], V)
        counts = np.where(np.arange(N) % 2 == 0, k, 0)
        r["bias_offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(dev)
        ids = np.concatenate([np.sort(g.integers(0, V // k, k) + np.arange(k) * (V // k)) if c else [] for c in counts])
        r["bias_ids"] = torch.from_numpy(ids.astype(np.int32)).to(dev)
        r["bias_values"] = torch.from_numpy(g.uniform(-4, 4, ids.size).astype(np.float32)).to(dev)
    if case["masked"] > 0:
        on = g.random(N) < case["masked"]
        on[0] = True
        R, words = int(on.sum()), (V + 31) // 32
        sharp = case.get("sharp", 0)
        if sharp:
            ids = torch.randint(0, V, (R, sharp), generator=gen, device=dev)
            m = _bits_of(ids, words, dev)
            if R > 8:
                m[R // 2] = 0                 # a grammar that has come to its end: nothing is left
        else:
            m = torch.randint(-2 ** 31, 2 ** 31, (R, words), generator=gen, device=dev, dtype=torch.int64).to(torch.int32)
        if targets is not None:               # the token was drawn under this grammar
            a = targets[torch.from_numpy(np.nonzero(on)[0]).to(dev)].long().view(-1, 1)
            m = m | _bits_of(a, words, dev)
        r["allowed"] = m
        r["allowed_rows"] = torch.from_numpy(np.where(on, np.cumsum(on) - 1, -1).astype(np.int32)).to(dev)
    return r, spans


def _logits(case, gen, dev, ids=None, lift=None):
    N, V = case["N"], case["V"]
    out = torch.empty((N, V), dtype=DTYPES[case["dtype"]], device=dev)
    step = max(1, 200000000 // V)
    for i in range(0, N, step):
        z = torch.randn((min(step, N - i), V), generator=gen, device=dev) * 2
        if ids is not None:
            z.scatter_add_(1, ids[i:i + step].long(), lift[i:i + step])
        out[i:i + step] = z
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = np.random.default_rng([seed, case["N"], case["V"]])
    gen = torch.Generator(device=dev).manual_seed(int(g.integers(2 ** 62)))
    N, V, op = case["N"], case["V"], case["op"]
    state = {"case": case}
    if op == "process":
        state["rules"], spans = _rules(case, g, gen, dev)
        state["pairs"] = int((spans[:, 2] - spans[:, 0]).sum())
        state["logits"] = _logits(case, gen, dev)
        state["out"] = torch.empty((N, V), dtype=DTYPES[case["out"]], device=dev)
        return state
    if op.startswith("logprob"):
        left, lens = N, []
        while left > 0:
            n = int(_lengths(g, 1, case["seq_len"], 4 * case["seq_len"])[0]) if case["ragged"] else case["seq_len"]
            lens.append(min(n, left))
            left -= lens[-1]
        lens = np.array(lens)
        start = np.repeat(np.concatenate([[0], np.cumsum(lens)[:-1]]), lens)
        stop = np.repeat(np.cumsum(lens), lens)
        pos = np.arange(N)
        # row t has read the tokens up to its own and predicts the next one
        spans = np.stack([start, np.minimum(np.minimum(start + case["prompt"], stop), pos + 1), pos + 1], 1)
        tokens = _tokens(gen, N + 1, V, dev)
        targets = tokens[1:].contiguous()
        state["targets"] = targets
        state["rules"], _ = _rules(case, g, gen, dev, targets, spans, tokens[:N].contiguous())
        state["pairs"] = int((spans[:, 2] - spans[:, 0]).sum())
        lift = torch.rand((N, 1), generator=gen, device=dev) * 12
        state["logits"] = _logits(case, gen, dev, targets.view(-1, 1), lift)
        if op == "logprob_backward":
            state["grad"] = torch.randn(N, generator=gen, device=dev)
            if N > 4:
                state["grad"][:: 5] = 0       # prompt tokens and rejected ones
            state["lse"] = _exact_logprob(state)["lse"].float()
            state["out"] = torch.empty_like(state["logits"])
        return state
    K = case["K"]
    step = torch.from_numpy(g.integers(1, max(2, V // K), (N, 1))).to(dev)
    ids = (torch.from_numpy(g.integers(0, V, (N, 1))).to(dev) + step * torch.arange(K, device=dev)) % V
    base = torch.rand((N, 1), generator=gen, device=dev) * 6 + 6
    shape = base - 1.5 * torch.log(torch.arange(1, K + 1, device=dev, dtype=torch.float32))
    state["logits"] = _logits(case, gen, dev, ids, (shape - 2).clamp(min=0))
    state["teacher_logits"] = (shape + torch.randn((N, K), generator=gen, device=dev) * 0.3).contiguous()
    ids = ids.to(torch.int32)
    if case["holes"]:
        keep = torch.from_numpy(g.integers(0, K + 1, (N, 1))).to(dev)
        ids = torch.where(torch.arange(K, device=dev) < keep, ids, -1).to(torch.int32)
    state["teacher_ids"] = ids.contiguous()
    if case["tail"]:
        t = state["teacher_logits"].double().masked_fill(ids < 0, -math.inf)
        mass = torch.from_numpy(g.uniform(0.001, 0.3, N)).to(dev)
        lse = torch.logsumexp(t, 1) - torch.log1p(-mass)
        state["teacher_lse"] = torch.where(torch.isfinite(lse), lse, 0.0).float()
    if case["op"] != "distill_forward":
        state["grad"] = torch.rand(N, generator=gen, device=dev)
        if N > 4:
            state["grad"][:: 7] = 0           # tokens outside the loss mask
        state["out"] = torch.empty_like(state["logits"])
    if case["op"] == "distill_backward":
        e = _exact_distill(state)
        state["lse"] = e["lse"].float()
        if case["tail"]:
            state["lse_tail"] = e["lse_tail"].float()
    return state


# ----------------------------------------------------------------------------- plain forms (fp32)
def _plain_parts(state):
    """(y, dy/dz) of every logit: the processed logits and their slope, fp32."""
    r, z = state["rules"], state["logits"].float()
    N, V = z.shape
    dev = z.device
    y = z
    if "bias_ids" in r:
        n = r["bias_offsets"][1:] - r["bias_offsets"][:-1]
        row = torch.repeat_interleave(torch.arange(N, device=dev), n.long(), output_size=r["bias_ids"].numel())
        y = y.index_put((row, r["bias_ids"].long()), r["bias_values"], accumulate=True)
    spans = r["history_spans"].long()
    n = spans[:, 2] - spans[:, 0]
    total = state["pairs"]
    row = torch.repeat_interleave(torch.arange(N, device=dev), n, output_size=total)
    first = torch.cumsum(n, 0) - n
    j = torch.arange(total, device=dev) - first[row] + spans[row, 0]
    flat = row * V + r["history"][j].long()
    seen = torch.zeros(N * V, dtype=torch.bool, device=dev)
    seen[flat] = True
    seen = seen.view(N, V)
    made = torch.zeros(N * V, dtype=torch.float32, device=dev)
    made.scatter_add_(0, flat, (j >= spans[row, 1]).float())
    made = made.view(N, V)
    rep = r["repetition"].view(N, 1)
    slope = torch.where(seen, torch.where(y > 0, 1 / rep, rep), torch.ones_like(y))
    y = torch.where(seen, torch.where(y > 0, y / rep, y * rep), y)
    y = y - r["frequency"].view(N, 1) * made - r["presence"].view(N, 1) * (made > 0)
    tau = r["temperature"].view(N, 1)
    y, slope = y / tau, slope / tau
    if "allowed" in r:
        col = torch.arange(V, device=dev)
        k = r["allowed_rows"].long()
        ok = ((r["allowed"][k.clamp(min=0)][:, col >> 5] >> (col & 31).int()) & 1).bool()
        ok = ok | (k < 0).view(N, 1)
        y = torch.where(ok, y, torch.full_like(y, -math.inf))
    return y, torch.where(y == -math.inf, torch.zeros_like(slope), slope)


def _plain_lse(y):
    m = y.max(1, keepdim=True).values
    m0 = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    return m0.view(-1), torch.log(torch.exp(y - m0).sum(1))


def _plain_process(state):
    return _plain_parts(state)[0].to(state["out"].dtype)


def _plain_logprob(state):
    y, _ = _plain_parts(state)
    m, ls = _plain_lse(y)
    a = y.gather(1, state["targets"].long().view(-1, 1)).view(-1)
    logp = torch.where(a == -math.inf, a, (a - m) - ls)
    return {"logp": logp, "lse": m + ls}


def _plain_logprob_backward(state):
    y, slope = _plain_parts(state)
    d = -torch.exp(y - state["lse"].view(-1, 1))
    d.scatter_add_(1, state["targets"].long().view(-1, 1), torch.ones_like(d[:, :1]))
    return (d * slope * state["grad"].view(-1, 1)).to(state["logits"].dtype)


def _plain_teacher(state):
    ids = state["teacher_ids"].long()
    on = ids >= 0
    t = torch.where(on, state["teacher_logits"], torch.full_like(state["teacher_logits"], -math.inf))
    if "teacher_lse" in state:
        logq = t - state["teacher_lse"].view(-1, 1)
    else:
        m, ls = _plain_lse(t)
        logq = t - m.view(-1, 1) - ls.view(-1, 1)
    q = torch.where(on, torch.exp(logq), torch.zeros_like(t))
    return ids.clamp(min=0), on, torch.where(on, logq, torch.zeros_like(t)), q


def _plain_distill_forward(state):
    z = state["logits"].float()
    ids, on, logq, q = _plain_teacher(state)
    m, ls = _plain_lse(z)
    logp = z.gather(1, ids) - m.view(-1, 1) - ls.view(-1, 1)
    loss = torch.where(on, q * (logq - logp), torch.zeros_like(q)).sum(1)
    out = {"loss": loss, "lse": m + ls}
    if "teacher_lse" in state:
        rest = z.scatter_add(1, ids, torch.where(on, torch.full_like(q, -math.inf), torch.zeros_like(q)))
        mt, lt = _plain_lse(rest)
        qt = (1 - q.sum(1)).clamp(min=0)
        more = qt * (torch.log(qt) - ((mt - m) + lt - ls))
        out["loss"] = loss + torch.where(qt > 0, more, torch.zeros_like(qt))
        out["lse_tail"] = mt + lt
    return out


def _plain_distill_backward(state, fwd):
    z = state["logits"].float()
    ids, on, _, q = _plain_teacher(state)
    p = torch.exp(z - fwd["lse"].view(-1, 1))
    if "teacher_lse" in state:
        qt = (1 - q.sum(1)).clamp(min=0)
        w = (1 - qt / torch.exp(fwd["lse_tail"] - fwd["lse"])).view(-1, 1)
        at = torch.zeros_like(z).scatter_add_(1, ids, on.float())
        d = p * torch.where(at > 0, torch.ones_like(p), w.expand_as(p))
    else:
        d = p * on.any(1, keepdim=True)
    d = d.scatter_add(1, ids, -q)
    return (d * state["grad"].view(-1, 1)).to(state["logits"].dtype)


# ----------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "process":
            return _plain_process(state)
        if op == "logprob":
            return _plain_logprob(state)
        if op == "logprob_backward":
            return _plain_logprob_backward(state)
        if op == "distill_backward":
            return _plain_distill_backward(state, state)
        out = _plain_distill_forward(state)
        if op == "distill_step":
            out["dlogits"] = _plain_distill_backward(state, out)
        return out
    import rollout_logprob_mismatch_gb300 as tim

    if op in ("process", "logprob", "logprob_backward"):
        rules = tim.LogitsRules(**state["rules"])
        if op == "process":
            return tim.process_logits(state["logits"], rules, out=state["out"])
        if op == "logprob":
            logp, lse = tim.processed_logprob(state["logits"], rules, state["targets"])
            return {"logp": logp, "lse": lse}
        return tim.processed_logprob_backward(state["logits"], rules, state["targets"], state["grad"], state["lse"],
                                              dlogits=state["out"])
    t = (state["logits"], state["teacher_ids"], state["teacher_logits"])
    tail = state.get("teacher_lse")
    if op == "distill_backward":
        return tim.distill_topk_backward(*t, state["grad"], state["lse"], state.get("lse_tail"), teacher_lse=tail,
                                         dlogits=state["out"])
    if op == "distill_forward":
        out = tim.distill_topk(*t, teacher_lse=tail)
    else:
        out = tim.distill_topk_step(*t, state["grad"], teacher_lse=tail, dlogits=state["out"])
    return {k: v for k, v in out.items() if v is not None}


# ----------------------------------------------------------------------------- work
def work(case):
    N, V, op = case["N"], case["V"], case["op"]
    es = SIZES[case["dtype"]]
    nv = N * V
    if op in ("process", "logprob", "logprob_backward"):
        b = nv * es + N * (12 + 16)                              # logits, spans, four parameters
        b += 4 * (N * case["hist_median"] if op == "process" else N)
        b += 4 * case["bias"] * N + (N * case["masked"]) * ((V + 31) // 32) * 4
        if op == "process":
            return {"bytes": int(b + nv * SIZES[case["out"]]), "flops": 2 * nv}
        if op == "logprob":
            return {"bytes": int(b + 12 * N), "flops": 4 * nv}
        return {"bytes": int(b + 12 * N + nv * es), "flops": 5 * nv}
    b = nv * es + N * case["K"] * 8 + 4 * N * (2 if case["tail"] else 1)
    if op == "distill_forward":
        return {"bytes": b + 8 * N, "flops": 4 * nv}
    return {"bytes": b + nv * es + 12 * N, "flops": (8 if op == "distill_step" else 4) * nv}


# ----------------------------------------------------------------------------- the definition in fp64
def _blocks(N, V):
    step = max(1, 60000000 // V)
    return [(i, min(N, i + step)) for i in range(0, N, step)]


def _exact_processed(state, i0, i1):
    """fp64 (y, slope) of rows i0..i1: counts by sorting each row's (row, id) keys."""
    r = state["rules"]
    z = state["logits"][i0:i1].double()
    n, V = z.shape
    dev = z.device
    spans = r["history_spans"][i0:i1].long()
    at = torch.arange(int((spans[:, 2] - spans[:, 0]).max()), device=dev)
    j = spans[:, :1] + at
    live = j < spans[:, 2:]
    key = torch.arange(n, device=dev).view(-1, 1) * V + r["history"][j.clamp(max=r["history"].numel() - 1)].long()
    u = torch.unique(key[live])
    rep_of = r["repetition"][i0:i1].double()
    if "bias_ids" in r:
        lo, hi = int(r["bias_offsets"][i0]), int(r["bias_offsets"][i1])
        row = torch.bucketize(torch.arange(lo, hi, device=dev), r["bias_offsets"][i0:i1 + 1].long(), right=True) - 1
        z.view(-1)[row * V + r["bias_ids"][lo:hi].long()] += r["bias_values"][lo:hi].double()
    slope = torch.ones_like(z)
    x = z.view(-1)[u]
    f = torch.where(x > 0, 1 / rep_of[u // V], rep_of[u // V])
    z.view(-1)[u] = x * f
    slope.view(-1)[u] = f
    w, c = torch.unique(key[live & (j >= spans[:, 1:2])], return_counts=True)
    z.view(-1)[w] -= r["frequency"][i0:i1].double()[w // V] * c + r["presence"][i0:i1].double()[w // V]
    tau = r["temperature"][i0:i1].double().view(-1, 1)
    z /= tau
    slope /= tau
    if "allowed" in r:
        for k, m in enumerate(r["allowed_rows"][i0:i1].tolist()):
            if m >= 0:
                bits = (r["allowed"][m].view(-1, 1) >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
                off = bits.reshape(-1)[:V] == 0
                z[k, off] = -math.inf
                slope[k, off] = 0
    return z, slope


def _exact_logprob(state):
    N, V = state["logits"].shape
    logp = torch.empty(N, dtype=torch.float64, device=state["logits"].device)
    lse = torch.empty_like(logp)
    for i0, i1 in _blocks(N, V):
        y, _ = _exact_processed(state, i0, i1)
        lse[i0:i1] = torch.logsumexp(y, 1)
        a = y.gather(1, state["targets"][i0:i1].long().view(-1, 1)).view(-1)
        logp[i0:i1] = torch.where(a == -math.inf, a, a - lse[i0:i1])
    return {"logp": logp, "lse": lse}


def _exact_teacher(state, i0, i1):
    ids = state["teacher_ids"][i0:i1].long()
    t = state["teacher_logits"][i0:i1].double().masked_fill(ids < 0, -math.inf)
    if "teacher_lse" in state:
        q = torch.exp(t - state["teacher_lse"][i0:i1].double().view(-1, 1))
    else:
        q = torch.softmax(t, 1).nan_to_num(nan=0.0)
    return ids, q


def _exact_distill(state, gradient=False):
    z_all = state["logits"]
    N, V = z_all.shape
    tail = "teacher_lse" in state
    out = {k: torch.empty(N, dtype=torch.float64, device=z_all.device)
           for k in ("loss", "lse") + (("lse_tail",) if tail else ())}
    if gradient:
        out["dlogits"] = torch.empty((N, V), dtype=torch.float64, device=z_all.device)
    given = state.get("lse")
    for i0, i1 in _blocks(N, V):
        z = z_all[i0:i1].double()
        ids, q = _exact_teacher(state, i0, i1)
        row = torch.arange(i1 - i0, device=z.device).view(-1, 1).expand_as(ids)[ids >= 0]
        col, qs = ids[ids >= 0], q[ids >= 0]
        lse = torch.logsumexp(z, 1)
        logp = z[row, col] - lse[row]
        terms = torch.where(qs > 0, qs * (torch.log(qs) - logp), 0.0)
        loss = torch.zeros_like(lse).index_add_(0, row, terms)
        if tail:
            rest = z.clone()
            rest[row, col] = -math.inf
            lt = torch.logsumexp(rest, 1)
            qt = (1 - q.sum(1)).clamp(min=0)
            loss = loss + torch.where(qt > 0, qt * (torch.log(qt) - (lt - lse)), 0.0)
            out["lse_tail"][i0:i1] = lt
        out["loss"][i0:i1], out["lse"][i0:i1] = loss, lse
        if gradient:
            if given is not None:             # the gradient takes the forward's own figures
                lse = given[i0:i1].double()
                lt = state["lse_tail"][i0:i1].double() if tail else None
            p = torch.exp(z - lse.view(-1, 1))
            d = p * (1 - qt / torch.exp(lt - lse)).view(-1, 1) if tail else p * (q.sum(1, keepdim=True) > 0)
            d[row, col] = p[row, col] - qs
            out["dlogits"][i0:i1] = d * state["grad"][i0:i1].double().view(-1, 1)
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "logprob":
        return _exact_logprob(state)
    if op.startswith("distill"):
        out = _exact_distill(state, gradient=op != "distill_forward")
        return out["dlogits"] if op == "distill_backward" else out
    N, V = state["logits"].shape
    res = torch.empty((N, V), dtype=torch.float64, device=state["logits"].device)
    for i0, i1 in _blocks(N, V):
        y, slope = _exact_processed(state, i0, i1)
        if op == "process":
            res[i0:i1] = y
            continue
        d = -torch.exp(y - state["lse"][i0:i1].double().view(-1, 1))
        d.scatter_add_(1, state["targets"][i0:i1].long().view(-1, 1), torch.ones_like(d[:, :1]))
        res[i0:i1] = torch.where(slope == 0, 0.0, d * slope * state["grad"][i0:i1].double().view(-1, 1))
    return res
