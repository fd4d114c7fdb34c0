"""Operators beside a vocabulary head's table, as cases that can be timed and compared.

  adapters            low-rank adapters of many requests beside the shared head: the
                      rows of one batch of logits belong to different adapters;
  adapters_backward   their gradient (hidden states, A and B) from the logits' gradient;
  embedding           rows of the table for a batch of tokens, scaled;
  embedding_backward  the table's gradient from the rows' gradients.

With the module's ``own`` false, `run` computes them from elementary torch
operations in fp32; with ``own`` true it calls this library.  `exact` is the
definition in fp64.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZES = {"f32": 4, "bf16": 2, "f16": 2}


# ----------------------------------------------------------------------------- cases
def _adapters(name, N, V, D, R, n, dtype, backward, runs):
    """N rows of logits of type dtype, n loaded adapters of rank R; runs: rows come in
    sequences (a trainer's packed batch), else each row is a request of its own.
    About one row (or sequence) in eight is under no adapter."""
    return {"name": name, "op": "adapters_backward" if backward else "adapters", "N": N, "V": V, "D": D, "R": R, "n": n,
            "dtype": dtype, "runs": runs}


def _embedding(name, N, V, D, dtype, out, backward, pads):
    """dtype: of the table (of the rows' gradient when backward), out: of the rows;
    pads: fraction of padding tokens (id -1)."""
    return {"name": name, "op": "embedding_backward" if backward else "embedding", "N": N, "V": V, "D": D,
            "dtype": dtype, "out": out, "pads": pads}


def listed():
    return [
        # one request in a decoding engine that has eight adapters loaded: latency is what counts
        _adapters("adapters_one_row", 1, 151936, 4096, 16, 8, "f32", False, False),
        # a decoding batch, two requests an adapter on average
        _adapters("adapters_decode", 64, 128256, 4096, 16, 32, "bf16", False, False),
        # a large decoding batch under many adapters of rank 32
        _adapters("adapters_decode_large", 256, 151936, 4096, 32, 64, "bf16", False, False),
        # a trainer's packed batch of the benchmark's head, four tenants
        _adapters("adapters_packed", 8192, 151936, 4096, 16, 4, "bf16", False, True),
        # odd sizes: rows start at odd offsets, the smallest rank, fp32 logits
        _adapters("adapters_odd", 333, 32003, 1000, 8, 5, "f32", False, True),
        # a training step's gradient on packed sequences, eight tenants
        _adapters("adapters_backward_packed", 4096, 128256, 4096, 16, 8, "bf16", True, True),
        # the same on fp32 logits, rank 32, a wide model
        _adapters("adapters_backward_f32", 1024, 129280, 7168, 32, 3, "f32", True, True),
        # odd sizes, fp16 logits with a loss scale, a rank between powers of two, rows in any order
        _adapters("adapters_backward_odd", 500, 50261, 1000, 24, 7, "f16", True, False),
        # one request's next token
        _embedding("embedding_one_row", 1, 151936, 4096, "bf16", "bf16", False, 0.0),
        # a training batch of packed sequences
        _embedding("embedding_packed", 32768, 128256, 4096, "bf16", "bf16", False, 0.0),
        # the table's gradient of that batch
        _embedding("embedding_backward_packed", 32768, 128256, 4096, "bf16", "bf16", True, 0.0),
        # odd sizes, fp32, padded sequences
        _embedding("embedding_backward_odd", 1777, 32003, 1001, "f32", "f32", True, 0.3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    V = _log_int(rng, 1000, 152000)
    if rng.random() < 0.6:
        V = (V + 63) // 64 * 64
    D = 8 * _log_int(rng, 16, 900)
    dtype = rng.choice(["bf16", "bf16", "f32", "f16"])
    op = rng.choice(["adapters", "adapters", "adapters_backward", "adapters_backward", "embedding", "embedding_backward"])
    if op.startswith("adapters"):
        backward = op == "adapters_backward"
        runs = rng.random() < 0.6
        N = min(_log_int(rng, 1, 8192 if runs else 300), max(1, (500000000 if backward else 1000000000) // V))
        R = rng.choice([8, 16, 16, 24, 32, 32, 40, 64, 128])
        n = min(_log_int(rng, 1, 64), max(1, 600000000 // (V * R)))
        return _adapters("", N, V, D, R, n, dtype, backward, runs)
    N = _log_int(rng, 1, 32768)
    if rng.random() < 0.3:
        D += rng.randrange(1, 8)
    V = min(V, 530000000 // D)
    return _embedding("", N, V, D, dtype, rng.choice([dtype, "bf16", "f32"]), op == "embedding_backward",
                      rng.choice([0.0, 0.0, 0.3]))


def work(case):
    N, V, D, op = case["N"], case["V"], case["D"], case["op"]
    if op.startswith("adapters"):
        R, es = case["R"], SIZES[case["dtype"]]
        used = min(case["n"], N)
        weights = used * R * (V + D)
        if op == "adapters":
            return {"bytes": 2 * N * V * es + 2 * N * D + 2 * weights, "flops": 2 * N * R * (V + D)}
        return {"bytes": N * V * es + 2 * N * D + 2 * weights + 4 * N * D + 4 * case["n"] * R * (V + D),
                "flops": 4 * N * R * V + 6 * N * R * D}
    es, eo = SIZES[case["dtype"]], SIZES[case["out"]]
    live = int(N * (1 - case["pads"]))
    if op == "embedding":
        return {"bytes": 4 * N + min(live, V) * D * es + N * D * eo, "flops": live * D}
    return {"bytes": 4 * N + live * D * es + 4 * V * D, "flops": live * D}


# ----------------------------------------------------------------------------- inputs
def _tokens(gen, n, V, dev):
    # repeats as in text: a few ids often, most of them hardly ever
    return (torch.rand(n, generator=gen, device=dev) ** 4 * V).to(torch.int32).clamp_(max=V - 1)


def _blocks(N, V, most=100000000):
    step = max(1, most // V)
    return [(i, min(N, i + step)) for i in range(0, N, step)]


def _logits(case, gen, dev):
    N, V = case["N"], case["V"]
    out = torch.empty((N, V), dtype=DTYPES[case["dtype"]], device=dev)
    for i0, i1 in _blocks(N, V):
        out[i0:i1] = torch.randn((i1 - i0, V), generator=gen, device=dev) * 2
    return out


def _dlogits(case, gen, dev):
    """g (onehot - softmax) of random logits; every fifth row outside the loss."""
    N, V = case["N"], case["V"]
    scale = 256.0 if case["dtype"] == "f16" else 1.0
    out = torch.empty((N, V), dtype=DTYPES[case["dtype"]], device=dev)
    for i0, i1 in _blocks(N, V):
        d = -torch.softmax(torch.randn((i1 - i0, V), generator=gen, device=dev) * 3, 1)
        t = _tokens(gen, i1 - i0, V, dev).long().view(-1, 1)
        d.scatter_add_(1, t, torch.ones_like(d[:, :1]))
        g = torch.randn((i1 - i0, 1), generator=gen, device=dev) * scale
        g[(-i0) % 5::5] = 0
        out[i0:i1] = d * g
    return out


def _rows(case, g):
    """The adapter of each row, -1 = none."""
    N, n = case["N"], case["n"]
    if not case["runs"]:
        rows = np.where(g.random(N) < 0.125, -1, g.integers(0, n, N))
    else:
        parts, left = [], N
        while left > 0:
            k = min(left, int(np.clip(np.exp(g.normal(math.log(512), 0.5)), 1, 4096)))
            parts.append(np.full(k, -1 if g.random() < 0.125 else g.integers(0, n)))
            left -= k
        rows = np.concatenate(parts)
    if (rows < 0).all():
        rows[:] = n - 1
    return rows.astype(np.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = np.random.default_rng([seed, case["N"], case["V"], case["D"]])
    gen = torch.Generator(device=dev).manual_seed(int(g.integers(2 ** 62)))
    N, V, D, op = case["N"], case["V"], case["D"], case["op"]
    state = {"case": case}
    if op.startswith("adapters"):
        R, n = case["R"], case["n"]
        rows = _rows(case, g)
        state["rows"] = torch.from_numpy(rows).to(dev)
        # what a scheduler knows of its batch on the host: the rows of each adapter (the plain form goes by it)
        state["groups"] = [(a, torch.from_numpy(np.nonzero(rows == a)[0]).to(dev)) for a in np.unique(rows).tolist()]
        state["h"] = torch.randn((N, D), generator=gen, device=dev).to(torch.bfloat16)
        state["A"] = ((torch.rand((n, R, D), generator=gen, device=dev) * 2 - 1) / math.sqrt(D)).to(torch.bfloat16)
        state["B"] = torch.empty((n, V, R), dtype=torch.bfloat16, device=dev)
        for a in range(n):
            state["B"][a] = torch.randn((V, R), generator=gen, device=dev) * 0.1
        state["scale"] = torch.from_numpy(g.choice([0.5, 1.0, 2.0], n).astype(np.float32)).to(dev)
        if op == "adapters":
            state["logits"] = _logits(case, gen, dev)
            state["out"] = torch.empty_like(state["logits"])
        else:
            state["dlogits"] = _dlogits(case, gen, dev)
        if own:
            import rollout_logprob_mismatch_gb300 as tim
            state["adapters"] = tim.Adapters(state["A"], state["B"], state["scale"])
        return state
    tokens = _tokens(gen, N, V, dev)
    if case["pads"] > 0:
        off = torch.rand(N, generator=gen, device=dev) < case["pads"]
        tokens = torch.where(off, -1, tokens).to(torch.int32)
    state["tokens"] = tokens
    state["scale"] = math.sqrt(D)
    shape = (V, D) if op == "embedding" else (N, D)
    x = torch.empty(shape, dtype=DTYPES[case["dtype"]], device=dev)
    for i0, i1 in _blocks(*shape):
        x[i0:i1] = torch.randn((i1 - i0, D), generator=gen, device=dev) * (0.02 if op == "embedding" else 0.001)
    state["table" if op == "embedding" else "grad"] = x
    return state


# ----------------------------------------------------------------------------- plain forms (fp32)
def _plain_adapters(state):
    z, out = state["logits"], state["out"]
    for a, i in state["groups"]:
        if a < 0:
            out[i] = z[i]
            continue
        t = state["scale"][a] * (state["h"][i].float() @ state["A"][a].float().t())
        out[i] = (z[i].float() + t @ state["B"][a].float().t()).to(out.dtype)
    return out


def _plain_adapters_backward(state):
    dy, h, A, B = state["dlogits"], state["h"], state["A"], state["B"]
    dh = torch.zeros(h.shape, dtype=torch.float32, device=h.device)
    dA = torch.zeros(A.shape, dtype=torch.float32, device=h.device)
    dB = torch.zeros(B.shape, dtype=torch.float32, device=h.device)
    for a, i in state["groups"]:
        if a < 0:
            continue
        d, x, s = dy[i].float(), h[i].float(), state["scale"][a]
        t = s * (x @ A[a].float().t())
        du = s * (d @ B[a].float())
        dB[a] = d.t() @ t
        dA[a] = du.t() @ x
        dh[i] = du @ A[a].float()
    return {"dh": dh, "dA": dA, "dB": dB}


def _plain_embedding(state):
    t, W = state["tokens"].long(), state["table"]
    x = W[t.clamp(min=0)].float() * state["scale"]
    return torch.where((t >= 0).view(-1, 1), x, 0.0).to(DTYPES[state["case"]["out"]])


def _plain_embedding_backward(state):
    t, g = state["tokens"].long(), state["grad"].float() * state["scale"]
    # one row more takes the padding tokens' gradients
    V = state["case"]["V"]
    dW = torch.zeros((V + 1, g.shape[1]), dtype=torch.float32, device=g.device)
    return dW.index_add_(0, torch.where(t >= 0, t, V), g)[:V]


# ----------------------------------------------------------------------------- the calls
def run(state):
    op = state["case"]["op"]
    if not own:
        return globals()["_plain_" + op](state)
    import rollout_logprob_mismatch_gb300 as tim
    if op == "adapters":
        return tim.adapter_logits(state["logits"], state["h"], state["adapters"], state["rows"], out=state["out"])
    if op == "adapters_backward":
        dh, dA, dB = tim.adapter_logits_backward(state["dlogits"], state["h"], state["adapters"], state["rows"])
        return {"dh": dh, "dA": dA, "dB": dB}
    if op == "embedding":
        return tim.embedding(state["tokens"], state["table"], scale=state["scale"],
                             out_dtype=DTYPES[state["case"]["out"]])
    return tim.embedding_backward(state["tokens"], state["grad"], state["case"]["V"], scale=state["scale"])


# ----------------------------------------------------------------------------- definitions (fp64)
def _exact_adapters(state):
    z = state["logits"]
    N, V = z.shape
    res = torch.empty((N, V), dtype=torch.float64, device=z.device)
    for i0, i1 in _blocks(N, V):
        res[i0:i1] = z[i0:i1].double()
    for a in range(state["A"].shape[0]):
        mine = torch.nonzero(state["rows"] == a).view(-1)
        u = torch.einsum("nd,rd->nr", state["h"][mine].double(), state["A"][a].double())
        Bt = state["B"][a].double().t() * state["scale"][a].double()
        for i0, i1 in _blocks(mine.numel(), V):
            res[mine[i0:i1]] += u[i0:i1] @ Bt
    return res


def _exact_adapters_backward(state):
    dy, h, A, B = state["dlogits"], state["h"].double(), state["A"].double(), state["B"]
    V = dy.shape[1]
    out = {"dh": torch.zeros_like(h), "dA": torch.zeros_like(A),
           "dB": torch.zeros(B.shape, dtype=torch.float64, device=h.device)}
    for a in range(A.shape[0]):
        mine = torch.nonzero(state["rows"] == a).view(-1)
        s, Ba = state["scale"][a].double(), B[a].double()
        for i0, i1 in _blocks(mine.numel(), V):
            i = mine[i0:i1]
            d = dy[i].double()
            out["dB"][a] += d.t() @ (h[i] @ A[a].t()) * s
            du = (d @ Ba) * s
            out["dA"][a] += du.t() @ h[i]
            out["dh"][i] = du @ A[a]
    return out


def _exact_embedding(state):
    t, W = state["tokens"], state["table"]
    res = torch.zeros((t.shape[0], W.shape[1]), dtype=torch.float64, device=W.device)
    on = torch.nonzero((t >= 0) & (t < W.shape[0])).view(-1)
    # the scale is an argument of the call in 32 bits
    res[on] = W[t[on].long()].double() * float(np.float32(state["scale"]))
    return res


def _exact_embedding_backward(state):
    t, g = state["tokens"], state["grad"]
    res = torch.zeros((state["case"]["V"], g.shape[1]), dtype=torch.float64, device=g.device)
    on = torch.nonzero(t >= 0).view(-1)
    for i0, i1 in _blocks(on.numel(), g.shape[1]):
        i = on[i0:i1]
        res.index_add_(0, t[i].long(), g[i].double() * float(np.float32(state["scale"])))
    return res


def exact(case, seed):
    return globals()["_exact_" + case["op"]](prepare(case, seed))
