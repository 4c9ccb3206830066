"""The workloads of the 8-bit integer products and of the router's training operators: cases, inputs, plain forms.

Four families, for models whose experts and dense layers hold int8 weights, and for training their router:

  gemm       C = A W^T in 8-bit integers, a scale per token and per output channel; from bf16 activations,
             which the call quantises a row at a time ("qa"), or from codes and scales ("codes");
  experts    rows quantised, then the experts' products on the rows sorted by expert: gate_up with
             silu(gate) * up read through the sort's index, and down on the sorted rows;
  balance    the load balance loss of a routed batch, with the slots of each expert counted;
  router     the gradient of the router's logits: of the chosen experts' weights, and of the balance loss.

A row's int8 rule: s = max(amax, 1e-10) / 127, code = rint(x * (127 / max(amax, 1e-10))), each step in fp32.
The loss: E * sum_e (counts[e] / (topk * n)) * (psum[e] / n), over the n tokens that the mask keeps, with
counts[e] their slots of expert e and psum[e] the sum of their softmax probabilities of e.

`own` false: elementary torch operations in 32 bits, rounded once at the end.  `own` true: the calls of
block_scaled_fp8_r9k_amd.
"""
from __future__ import annotations

import math

import torch

own = False


def _r9k():
    import block_scaled_fp8_r9k_amd as r9k
    return r9k


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # the smallest call: one token, a small projection; launch latency counts
        dict(name="gemm_m1_k512_n1024", op="gemm", M=1, K=512, N=1024, form="qa"),
        # one token through a wide up projection
        dict(name="gemm_m1_k4096_n14336", op="gemm", M=1, K=4096, N=14336, form="qa"),
        # a full decode batch through the long-K down projection, codes from the layer before
        dict(name="gemm_m16_k14336_n4096_codes", op="gemm", M=16, K=14336, N=4096, form="codes"),
        # a speculative or chunked batch, ragged against every tile
        dict(name="gemm_m100_k4096_n4096", op="gemm", M=100, K=4096, N=4096, form="qa"),
        # prefill through the widest projection, the codes shared with other projections of the same rows
        dict(name="gemm_m4096_k4096_n12288_codes", op="gemm", M=4096, K=4096, N=12288, form="codes"),
        # a decode step's gate_up products: 16 tokens, top-8 of 128 experts
        dict(name="experts_gate_up_t16", op="experts", T=16, H=2048, I=768, E=128, topk=8, part="gate_up"),
        # a prefill batch's down products
        dict(name="experts_down_t2048", op="experts", T=2048, H=2048, I=768, E=128, topk=8, part="down"),
        # a short training batch's balance loss, padded sequences masked out; an odd token count
        dict(name="balance_t1023_e128_mask", op="balance", T=1023, E=128, topk=8, dtype="fp32", mask=True,
             limited=False),
        # a large training batch's balance loss, experts limited to groups, logits kept in bf16
        dict(name="balance_t65536_e256_bf16", op="balance", T=65536, E=256, topk=8, dtype="bf16", mask=False,
             limited=True),
        # fine-tuning with a frozen balance: the gradient of the routing weights alone
        dict(name="router_t512_e8", op="router", T=512, E=8, topk=2, dtype="fp32", mask=False, limited=False,
             balance=False),
        # a training batch's whole gradient of the logits, padded sequences masked out
        dict(name="router_t8191_e128_balance_mask", op="router", T=8191, E=128, topk=8, dtype="fp32", mask=True,
             limited=False, balance=True),
        # a large training batch's whole gradient
        dict(name="router_t65536_e256_balance", op="router", T=65536, E=256, topk=8, dtype="fp32", mask=False,
             limited=True, balance=True),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    """A further case of the ranges: single tokens to prefill, narrow to wide, few to many experts."""
    top = max(work(c)["flops"] for c in listed())
    top_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["gemm", "gemm", "gemm", "experts", "experts", "balance", "router"])
        if op == "gemm":
            c = dict(op=op, M=_log_int(rng, 1, 4096), K=_log_int(rng, 128, 14336, 128),
                     N=_log_int(rng, 64, 14336, 16), form=rng.choice(["qa", "codes"]))
        elif op == "experts":
            E = _log_int(rng, 4, 256)
            c = dict(op=op, T=_log_int(rng, 1, 4096), H=_log_int(rng, 256, 4096, 128),
                     I=_log_int(rng, 128, 2048, 128), E=E, topk=rng.randint(1, min(E, 10)),
                     part=rng.choice(["gate_up", "down"]))
        else:
            E = _log_int(rng, 2, 512)
            c = dict(op=op, T=_log_int(rng, 1, 65536), E=E, topk=rng.randint(1, min(E, 10)),
                     dtype=rng.choice(["fp32", "fp32", "bf16"]), mask=rng.random() < 0.5, limited=rng.random() < 0.3)
            if op == "router":
                c["balance"] = rng.random() < 0.7 or c["dtype"] == "bf16"
        w = work(c)
        if w["flops"] <= top and w["bytes"] <= top_bytes:
            return c


def work(case):
    op = case["op"]
    if op == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        a = 2 * M * K if case["form"] == "qa" else M * K + 4 * M
        return {"bytes": N * K + 4 * N + a + 2 * M * N, "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["topk"]
    R = T * k
    if op == "experts":
        H, I = case["H"], case["I"]
        touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that uniform routing reaches, on average
        if case["part"] == "gate_up":
            return {"bytes": int(touched * 2 * I * (H + 4) + 2 * T * H + 4 * R + 2 * R * I), "flops": 2 * R * H * 2 * I}
        return {"bytes": int(touched * H * (I + 4) + 2 * R * I + 2 * R * H), "flops": 2 * R * I * H}
    b = 2 if case["dtype"] == "bf16" else 4
    mask = T if case["mask"] else 0
    if op == "balance":
        return {"bytes": T * E * b + 4 * R + mask + 8 * E, "flops": 5 * T * E}
    route = 12 * R
    if not case["balance"]:
        return {"bytes": T * E * b + route, "flops": 3 * R}
    return {"bytes": 2 * T * E * b + route + mask + 4 * E, "flops": 8 * T * E}


# ----------------------------------------------------------------- inputs ----

def _rows(gen, n, width):
    """Activations: normal values, one channel in a hundred twenty times as large."""
    x = torch.randn((n, width), generator=gen, device="cuda")
    x[:, torch.randperm(width, generator=gen, device="cuda")[: width // 100]] *= 20.0
    return x.to(torch.bfloat16)


def _weight(gen, N, K):
    """int8 weights of normal values, a scale for each of the N channels."""
    w = 0.02 * torch.randn((N, K), generator=gen, device="cuda")
    s = w.abs().amax(1) / 127.0
    return torch.round(w / s[:, None]).clamp(-127, 127).to(torch.int8), s


def _routing(gen, case):
    """Router logits, the topk experts of each token and their softmax weights over the chosen."""
    T, E, k = case["T"], case["E"], case["topk"]
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if case.get("limited") and E >= 4 * k:  # half of each token's experts are closed to it
        closed = torch.rand((T, E), generator=gen, device="cuda").argsort(1) < E // 2
        logits = logits.masked_fill(closed, float("-inf"))
    if case.get("dtype") == "bf16":
        logits = logits.to(torch.bfloat16)
    top, ids = logits.float().topk(k, dim=1)
    return logits, ids.to(torch.int32).contiguous(), torch.softmax(top, 1).contiguous()


def _sort(ids, E):
    """Stable sort of the slots by expert: src (slot of each sorted row) and offsets."""
    key, src = torch.sort(ids.reshape(-1), stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=ids.device, dtype=key.dtype))
    return src.int(), offsets.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        st["a"] = _rows(gen, M, K)
        st["w"] = _weight(gen, N, K)
        if case["form"] == "codes":
            st["aq"], st["as"] = _quant(st["a"])
        if own:
            r9k = _r9k()
            st["packed"] = r9k.pack_weight_i8(st["w"][0])
            st["c"] = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
            need = r9k.gemm_i8_workspace(M, K, N)
            st["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        return st
    T, E, k = case["T"], case["E"], case["topk"]
    logits, ids, tw = _routing(gen, case)
    if op == "experts":
        H, I, R = case["H"], case["I"], T * k
        gate_up = case["part"] == "gate_up"
        N, K = (2 * I, H) if gate_up else (H, I)
        parts = [_weight(gen, N, K) for _ in range(E)]
        w = tuple(torch.stack(p) for p in zip(*parts))
        src, offsets = _sort(ids, E)
        rows = T if gate_up else R
        st.update(w=w, src=src, offsets=offsets, bounds=offsets.tolist(), x=_rows(gen, rows, K))
        if own:
            st["packed"] = _r9k().pack_weight_i8(w[0])
            st["q"] = torch.empty((rows, K), dtype=torch.int8, device="cuda")
            st["s"] = torch.empty(rows, dtype=torch.float32, device="cuda")
            st["out"] = torch.empty((R, I if gate_up else H), dtype=torch.bfloat16, device="cuda")
        return st
    st.update(logits=logits, ids=ids, tw=tw)
    # sequences padded to one length: a fifth of the tokens are padding
    st["mask"] = torch.rand(T, generator=gen, device="cuda") >= 0.2 if case["mask"] else None
    if op == "balance":
        if own:
            need = _r9k().moe_balance_loss_workspace(T, E, k)
            st["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        return st
    st["gw"] = torch.randn((T, k), generator=gen, device="cuda")
    if case["balance"]:
        keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"]
        st["counts"] = _counts(ids, keep, E)  # what the forward pass returned
        # the loss's weight in the whole, times the tokens so that both parts are of one size
        st["gloss"] = 0.01 * T * (0.5 + torch.rand((), generator=gen, device="cuda"))
    return st


# ------------------------------------------------------------- plain forms ----

def _quant(x):
    """int8 codes and scales of the rows."""
    f = x.float()
    amax = f.abs().amax(1).clamp_min(1e-10)
    return torch.round(f * (127.0 / amax)[:, None]).to(torch.int8), amax / 127.0


def _counts(ids, keep, E):
    """Slots of each expert among the kept tokens, and last the kept tokens."""
    flat = torch.where(keep[:, None], ids, E).reshape(-1).long()
    counts = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    counts[E] = keep.sum()
    return counts


def _probs(logits):
    x = logits.float()
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        q, s = _quant(st["a"]) if case["form"] == "qa" else (st["aq"], st["as"])
        wq, ws = st["w"]
        return ((q.float() @ wq.float().t()) * s[:, None] * ws[None, :]).to(torch.bfloat16)
    if op == "experts":
        src, off, I = st["src"], st["bounds"], case["I"]
        gate_up = case["part"] == "gate_up"
        q, s = _quant(st["x"])
        out = torch.empty((src.numel(), I if gate_up else case["H"]), dtype=torch.bfloat16, device=q.device)
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            r = src[lo:hi].long() // case["topk"] if gate_up else slice(lo, hi)
            p = (q[r].float() @ st["w"][0][e].float().t()) * s[r][:, None] * st["w"][1][e][None, :]
            if gate_up:
                p = p[:, :I] / (1.0 + torch.exp(-p[:, :I])) * p[:, I:]
            out[lo:hi] = p.to(torch.bfloat16)
        return out
    T, E, k = case["T"], case["E"], case["topk"]
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"]
    if op == "balance":
        counts = _counts(st["ids"], keep, E)
        psum = (_probs(st["logits"]) * keep[:, None]).sum(0)
        n = counts[E].float().clamp_min(1.0)
        loss = (counts[:E].float() * psum).sum() * (E / k) / (n * n)
        return loss, counts, psum
    d = st["tw"] * (st["gw"] - (st["tw"] * st["gw"]).sum(1, keepdim=True))
    g = torch.zeros((T, E), device="cuda").scatter_add_(1, st["ids"].long(), d)
    if case["balance"]:
        p = _probs(st["logits"])
        c = st["counts"][:E].float()
        n = st["counts"][E].float().clamp_min(1.0)
        b = p * (c[None, :] - (p * c[None, :]).sum(1, keepdim=True))
        g = g + b * keep[:, None] * (st["gloss"] * (E / k) / (n * n))
    return g.to(st["logits"].dtype)


def _calls(st):
    """The framework's operators, as a program that holds its weights, outputs and workspaces calls them."""
    r9k = _r9k()
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        ws = st["w"][1]
        if case["form"] == "qa":
            return r9k.gemm_i8_qa(st["a"], st["packed"], ws, c=st["c"], workspace=st["workspace"])
        return r9k.gemm_i8(st["aq"], st["as"], st["packed"], ws, c=st["c"], workspace=st["workspace"])
    if op == "experts":
        q, s = r9k.quant_i8(st["x"], q=st["q"], s=st["s"])
        if case["part"] == "gate_up":
            return r9k.moe_gemm_i8(q, s, st["offsets"], st["packed"], st["w"][1], src=st["src"], topk=case["topk"],
                                   act="silu_mul", c=st["out"])
        return r9k.moe_gemm_i8(q, s, st["offsets"], st["packed"], st["w"][1], c=st["out"])
    if op == "balance":
        return r9k.moe_balance_loss(st["logits"], st["ids"], mask=st["mask"], workspace=st["workspace"])
    if not case["balance"]:
        return r9k.moe_route_backward(st["gw"], st["ids"], st["tw"], case["E"])
    return r9k.moe_balance_loss_backward(st["gloss"], st["logits"], st["counts"], case["topk"], mask=st["mask"],
                                         route=(st["gw"], st["ids"], st["tw"]))


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    """The same outputs from the definitions, in 64 bits (the codes and scales of a row are fp32 by definition)."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def codes(x):
        top = torch.maximum(x.max(1).values, -x.min(1).values).to(torch.float32)
        top = torch.maximum(top, torch.full_like(top, 1e-10))
        inv = (127.0 / top.to(f64)).to(torch.float32)
        scaled = (x.to(f64) * inv.to(f64)[:, None]).to(torch.float32)
        return torch.round(scaled.to(f64)), (top.to(f64) / 127.0).to(torch.float32).to(f64)

    if op == "gemm":
        q, s = codes(st["a"]) if case["form"] == "qa" else (st["aq"].to(f64), st["as"].to(f64))
        wq, ws = st["w"]
        return torch.matmul(q, wq.to(f64).T) * torch.outer(s, ws.to(f64))
    T, E, k = case["T"], case["E"], case["topk"]
    if op == "experts":
        q, s = codes(st["x"])
        rows = []
        for e in range(E):
            r = torch.arange(st["bounds"][e], st["bounds"][e + 1], device="cuda")
            if case["part"] == "gate_up":
                r = torch.div(st["src"][r].long(), k, rounding_mode="floor")
            p = torch.matmul(q[r], st["w"][0][e].to(f64).T) * torch.outer(s[r], st["w"][1][e].to(f64))
            if case["part"] == "gate_up":
                gate, up = p.chunk(2, dim=1)
                p = gate * torch.sigmoid(gate) * up
            rows.append(p)
        return torch.cat(rows)
    kept = [True] * T if st["mask"] is None else st["mask"].tolist()
    p = torch.softmax(st["logits"].to(f64), 1)
    if op == "balance":
        counts = [0] * E + [sum(kept)]
        for row, live in zip(st["ids"].tolist(), kept):
            for e in row if live else ():
                counts[e] += 1
        psum = p[torch.tensor(kept, device="cuda")].sum(0)
        counts = torch.tensor(counts, dtype=torch.int32, device="cuda")
        n = max(sum(kept), 1)
        loss = E * torch.dot(counts[:E].to(f64) / (k * n), psum / n)
        return loss, counts, psum
    w, gw = st["tw"].to(f64), st["gw"].to(f64)
    g = torch.zeros((T, E), dtype=f64, device="cuda")
    inner = torch.linalg.vecdot(w, gw)
    t = torch.arange(T, device="cuda")
    for j in range(k):  # a token's experts are distinct
        g[t, st["ids"][:, j].long()] += w[:, j] * (gw[:, j] - inner)
    if case["balance"]:
        c = st["counts"].to(f64)
        n = c[E].clamp_min(1)
        f = E * c[:E] / (k * n)  # the loss is the mean over kept tokens of sum_e f[e] * p[e]
        mean = torch.matmul(p, f)
        live = torch.tensor(kept, device="cuda").to(f64)
        g += st["gloss"].to(f64) / n * live[:, None] * p * (f[None, :] - mean[:, None])
    return g
