"""The operators on a head's logits in plain fp64 numpy, row by row from their
formulas, and the error bounds the GPU tests allow.

Bounds (u = 2^-24 is fp32's unit roundoff; none was fitted to a result):
  * a processed logit takes at most seven fp32 roundings, each of a value below
    A = (|z| + |bias|) max(repetition, 1) + frequency c + presence, then one
    division: 8 u A / temperature, plus one rounding to the output's type;
  * lse and logp: the base-2 exponents t = y log2(e) carry 4 u |t|, a term of the
    sum 2^-22 from the exponential and the sum below 64 roundings, the result
    three more: u (8 Y + 96), Y the row's largest finite |y|;
  * a probability e^(y - lse): relative u (8 (Y + |lse|) + 96), so a gradient
    |g slope| (p u (8 (Y + |lse|) + 96) + 4 u), plus one rounding;
  * a distillation loss: sum_k q_k (the bound of log p_k + that of log q_k), with
    the bound of q itself, relative u (8 T + 32), times |log q_k - log p_k|.
"""
import numpy as np

U = 2.0 ** -24
# half a unit in the last place: relative (24, 8 and 11 significant bits) and of the smallest subnormal
HALF_ULP = {"f32": (2.0 ** -24, 2.0 ** -150), "bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def rounding(x, dtype):
    rel, sub = HALF_ULP[dtype]
    x = np.where(np.isfinite(x), np.abs(x), 0.0)
    return rel * x + sub


def processed(z, r, i):
    """(y, slope, A / temperature) of row i: z fp64 [V], r a dict of numpy arrays
    named like LogitsRules' fields (absent = no rule)."""
    V = z.size
    x = z.astype(np.float64).copy()
    bias = np.zeros(V)
    if "bias_ids" in r:
        for j in range(r["bias_offsets"][i], r["bias_offsets"][i + 1]):
            bias[r["bias_ids"][j]] += float(r["bias_values"][j])
    x = x + bias
    slope = np.ones(V)
    scale = np.abs(z) + np.abs(bias)
    rho = float(r["repetition"][i]) if "repetition" in r else 1.0
    if "history" in r:
        b, g, e = (int(k) for k in r["history_spans"][i])
        ids = r["history"][b:e]
        ids = ids[(ids >= 0) & (ids < V)]
        seen = np.zeros(V, bool)
        seen[ids] = True
        made = r["history"][g:e]
        c = np.bincount(made[(made >= 0) & (made < V)], minlength=V).astype(np.float64)
        with np.errstate(invalid="ignore"):
            up = x > 0
        slope = np.where(seen, np.where(up, 1.0 / rho, rho), 1.0)
        x = np.where(seen, np.where(up, x / rho, x * rho), x)
        af = float(r["frequency"][i]) if "frequency" in r else 0.0
        ap = float(r["presence"][i]) if "presence" in r else 0.0
        x = np.where(c > 0, x - af * c - ap, x)
        scale = scale * max(rho, 1.0) + np.abs(af) * c + np.abs(ap) * (c > 0)
    tau = float(r["temperature"][i]) if "temperature" in r else 1.0
    y, slope, scale = x / tau, slope / tau, scale / tau
    if "allowed" in r:
        m = int(r["allowed_rows"][i]) if "allowed_rows" in r else i
        if m >= 0:
            w = r["allowed"][m].view(np.uint32)
            v = np.arange(V)
            off = (w[v >> 5] >> (v & 31).astype(np.uint32)) & 1 == 0
            y = np.where(off, -np.inf, y)
    slope = np.where(y == -np.inf, 0.0, slope)
    return y, slope, scale


def lse64(y):
    m = np.max(y) if y.size else -np.inf
    if m == -np.inf:
        return -np.inf
    return float(m + np.log(np.sum(np.exp(y - m))))


def top(y):
    f = np.abs(y[np.isfinite(y)])
    return float(f.max()) if f.size else 0.0


def process_ref(z, r, dtype):
    """(y, tolerance) [N, V]."""
    out = np.empty(z.shape)
    tol = np.empty(z.shape)
    for i in range(z.shape[0]):
        out[i], _, a = processed(z[i], r, i)
        tol[i] = 8 * U * np.where(np.isfinite(a), a, 0.0) + rounding(out[i], dtype)
    return out, tol


def logprob_ref(z, r, targets):
    """(logp, lse, tolerance) [N]."""
    N, V = z.shape
    logp, lse, tol = np.empty(N), np.empty(N), np.empty(N)
    for i in range(N):
        y, _, a = processed(z[i], r, i)
        lse[i] = lse64(y)
        t = int(targets[i])
        if not 0 <= t < V:
            logp[i] = np.nan
        else:
            logp[i] = -np.inf if y[t] == -np.inf else y[t] - lse[i]
        tol[i] = U * (8 * max(top(y), top(a)) + 96)
    return logp, lse, tol


def backward_ref(z, r, targets, g, lse, dtype):
    """(gradient, tolerance) [N, V] from the given (fp32) lse."""
    N, V = z.shape
    out, tol = np.zeros((N, V)), np.zeros((N, V))
    for i in range(N):
        y, slope, a = processed(z[i], r, i)
        L = float(lse[i])
        p = np.zeros(V) if L == -np.inf else np.exp(y - L)
        one = np.zeros(V)
        if 0 <= int(targets[i]) < V:
            one[int(targets[i])] = 1.0
        gi = float(g[i])
        if gi == 0.0:
            continue
        out[i] = np.where(slope == 0, 0.0, gi * slope * (one - p))
        tol[i] = abs(gi) * slope * (p * U * (8 * (max(top(y), top(a)) + (abs(L) if np.isfinite(L) else 0)) + 96) + 4 * U)
        tol[i] += rounding(out[i], dtype)
    return out, tol


def teacher64(ids, t, tlse, tau, V):
    on = (ids >= 0) & (ids < V)
    tt = np.where(on, t.astype(np.float64) / tau, -np.inf)
    if tlse is not None:
        logq = tt - float(tlse)
    else:
        logq = tt - lse64(tt) if np.max(tt) > -np.inf else np.full(tt.shape, -np.inf)
    return on, logq, np.exp(logq)


def distill_ref(z, ids, t, tlse, tau, g=None, dtype="f32", given=None):
    """dict of loss, lse, lse_tail, dlogits and their tolerances (suffix _tol).
    given: fp32 (lse, lse_tail) to take the gradient from."""
    N, V = z.shape
    tail = tlse is not None
    o = {k: np.zeros(N) for k in ("loss", "lse", "lse_tail", "loss_tol", "lse_tol")}
    o["dlogits"], o["dlogits_tol"] = np.zeros((N, V)), np.zeros((N, V))
    for i in range(N):
        y = z[i].astype(np.float64) / tau
        lse = lse64(y)
        on, logq, q = teacher64(ids[i], t[i], tlse[i] if tail else None, tau, V)
        T = top(logq) + (abs(float(tlse[i])) if tail else 0.0)
        lt = U * (8 * top(y) + 96)
        lq = U * (8 * T + 32)
        loss = tol = 0.0
        for k in range(ids.shape[1]):
            if on[k] and q[k] > 0:
                d = logq[k] - (y[ids[i, k]] - lse)
                loss += q[k] * d
                tol += q[k] * (lt + lq + lq * abs(d)) if np.isfinite(d) else 0.0
        listed = np.zeros(V, bool)
        listed[ids[i][on]] = True
        rest = np.where(listed, -np.inf, y)
        lr = lse64(rest)
        qo = 0.0
        if tail:
            qo = max(0.0, 1.0 - float(np.sum(q)))
            qerr = float(np.sum(q)) * lq + 8 * U
            if qo > 0:
                d = np.log(qo) - (lr - lse)
                loss += qo * d
                if np.isfinite(d):
                    tol += qo * 2 * lt + qerr * (abs(d) + 1)
        o["loss"][i], o["loss_tol"][i] = loss, tol + 8 * U * abs(loss) if np.isfinite(loss) else 0.0
        o["lse"][i], o["lse_tail"][i], o["lse_tol"][i] = lse, lr, lt
        if g is None or float(g[i]) == 0.0:
            continue
        if given is not None:
            lse = float(given[0][i])
            lr = float(given[1][i]) if tail else lr
        gi = float(g[i]) / tau
        p = np.zeros(V) if lse == -np.inf else np.exp(y - lse)
        qv = np.zeros(V)
        for k in range(ids.shape[1]):
            if on[k]:
                qv[ids[i, k]] += q[k]
        w, wtol = (1.0 if np.sum(q) > 0 else 0.0), 0.0
        if tail:
            po = np.exp(lr - lse) if lr > -np.inf else 0.0
            w = 0.0 if po == 0 else 1.0 - qo / po
            wtol = 0.0 if po == 0 else (qerr + qo * 3 * lt) / po + 4 * U * (1 + qo / po)
        elif not np.any(on):
            w = 0.0
        rel = U * (8 * (top(y) + (abs(lse) if np.isfinite(lse) else 0)) + 96)
        o["dlogits"][i] = gi * np.where(listed, p - qv, p * w)
        o["dlogits_tol"][i] = abs(gi) * np.where(listed, p * rel + qv * lq + 2 * U * (p + qv), p * (abs(w) * rel + wtol))
        o["dlogits_tol"][i] += rounding(o["dlogits"][i], dtype) + 2.0 ** -126
    return o
