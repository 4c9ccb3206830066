"""Plain forms of the 8-bit integer products and of the router's training operators, on the CPU, with the error bounds
that the tests use.  Written from the definitions in include/r9k.h alone.

Bounds.  One rounding to a type t is off by at most half a step, eps(t) / 2 of the value: u = 2^-24 in fp32, 2^-8 in
bf16 (and half of bf16's smallest subnormal, 2^-134, next to zero).  The integer sums are exact, so a product's output is
known to the bit: int -> fp32, times as, times ws, -> bf16."""
import numpy as np
import torch

F64 = torch.float64
U = 2.0 ** -24


def quant(x):
    """r9k_quant_i8's rule, step by step in fp32 (numpy): codes int8 [..., K], scales fp32 [...]."""
    f = x.float().numpy().astype(np.float32)
    bad = ~np.isfinite(f).all(-1)
    one = np.float32
    b = np.maximum(np.abs(np.where(bad[..., None], one(0), f)).max(-1), one(1e-10)).astype(np.float32)
    q = np.rint(f * (one(127) / b)[..., None], where=~bad[..., None], out=np.zeros_like(f))
    s = np.where(bad, one("nan"), b / one(127)).astype(np.float32)
    return torch.from_numpy(q.astype(np.int8)), torch.from_numpy(s)


def product32(aq, as_, wq, ws):
    """The product's fp32 value, to the bit: [M,K] codes and [M] scales with [N,K] and [N]."""
    acc = (aq.to(F64) @ wq.to(F64).T)          # whole numbers below 2^31: exact
    return acc.float() * as_[:, None] * ws[None, :]


def product(aq, as_, wq, ws):
    """(value, bound on its fp32 value's error) in 64 bits: three roundings."""
    want = (aq.to(F64) @ wq.to(F64).T) * as_.to(F64)[:, None] * ws.to(F64)[None, :]
    return want, 3.0001 * U * want.abs() + 2.0 ** -148


def bf16_bound(want, before):
    """Bound for an output rounded once to bf16 whose fp32 value is within `before` of `want`."""
    return before + 2.0 ** -8 * (want.abs() + before) + 2.0 ** -134


def probs(logits):
    """Softmax in 64 bits (0 for a logit of -inf, also where all are), and a bound on the error of its fp32 value: the
    difference d to the maximum is off by u d and so, with one more, is exp, of the value; exp, the division and the product by
    8 u together; the sum of E terms by at most E u of itself and by its terms' own errors (depth-weighted, at most the
    largest d that matters, 88: exp is below fp32's smallest normal value, 2^-126, from there on and may count as 0)."""
    x = logits.to(F64)
    mx = x.amax(1, keepdim=True)
    e = torch.where(x == -float("inf"), torch.zeros_like(x), torch.exp(x - mx))
    s = e.sum(1, keepdim=True)
    one = torch.where(s == 0, torch.ones_like(s), s)
    d = torch.where(torch.isfinite(x), mx - x, torch.zeros_like(x)).clamp_max(88.0)
    p = e / one
    mean = (p * d).sum(1, keepdim=True)
    return p, p * (2 * (d + mean) + x.shape[1] + 8) * U + 2.0 ** -126


def balance(logits, ids, mask=None):
    """(loss, counts [E+1], psum [E]) and bounds for loss and psum."""
    T, E = logits.shape
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    k = ids.shape[1]
    counts = torch.zeros(E + 1, dtype=torch.int64)
    for t in torch.nonzero(keep).flatten().tolist():
        for e in ids[t].tolist():
            if 0 <= e < E:
                counts[e] += 1
    n = int(keep.sum())
    counts[E] = n
    p, err = probs(logits[keep])
    psum, perr = p.sum(0), err.sum(0)
    perr = perr + (n + 1) * U * (psum + perr)   # a sum of n positive terms, in any order
    if not n:
        return (torch.zeros((), dtype=F64), counts.int(), psum), (torch.zeros((), dtype=F64), perr)
    f = counts[:E].to(F64) * E / (k * n * n)
    loss = (f * psum).sum()
    return (loss, counts.int(), psum), ((f * perr).sum() + (E + 8) * U * loss, perr)


def balance_grad(gloss, logits, counts, k, mask=None):
    """(gradient, bound on its fp32 value's error) in 64 bits."""
    T, E = logits.shape
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    n = int(counts[E])
    if n == 0:
        return torch.zeros((T, E), dtype=F64), torch.zeros((T, E), dtype=F64)
    p, err = probs(torch.where(keep[:, None], logits.float(), torch.zeros(())))
    f = counts[:E].to(F64) * E / (k * n)
    mean, merr = (p @ f)[:, None], (err @ f)[:, None]
    g = p * (f - mean)
    # f: three roundings; the mean E more; the difference, two products and the scale's division
    bad = err * (f + mean) + p * merr + p * (f + mean) * (E + 12) * U
    scale, live = abs(float(gloss)) / n, keep.to(F64)[:, None]
    return float(gloss) / n * g * live, (bad * scale * (1 + 4 * U) + 2.0 ** -148) * live


def route_grad(gw, ids, w, E):
    """(gradient [T,E], bound on its fp32 value's error) in 64 bits."""
    T, k = gw.shape
    g, v = gw.to(F64), w.to(F64)
    dot, size = (g * v).sum(1, keepdim=True), (g * v).abs().sum(1, keepdim=True)
    d = v * (g - dot)
    e = v.abs() * ((k + 1) * U * size + 3 * U * (g.abs() + dot.abs()))
    out, err = torch.zeros((T, E), dtype=F64), torch.zeros((T, E), dtype=F64)
    for t in range(T):
        for j in range(k):
            i = int(ids[t, j])
            if 0 <= i < E:
                out[t, i] += d[t, j]
                err[t, i] += e[t, j] + k * U * d[t, j].abs()   # up to k terms in one place
    return out, err
