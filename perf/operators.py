"""The workloads of the 4-bit and expert-sorting operators: cases, inputs, plain forms.

Three families, as they follow each other in a model whose experts hold 4-bit weights:

  gemm       C = A W^T with 4-bit weights and a scale per group along K: int4 codes with bf16 scales and
             optional zero points, or mxfp4 (e2m1 codes with a power-of-two scale per 32);
  permute    token rows sorted by expert (stable), and the way back with the routing weights, each with
             its gradient;
  experts    the experts' products on sorted rows: gate_up with silu(gate) * up read through the sort's
             index, and down on the sorted rows.

`own` false: elementary torch operations in 32 bits, rounded once at the end.  `own` true: the calls of
block_scaled_fp8_r9k_amd.
"""
from __future__ import annotations

import math

import torch

own = False

# The values of the sixteen e2m1 codes: sign, two exponent bits, one mantissa bit.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _r9k():
    import block_scaled_fp8_r9k_amd as r9k
    return r9k


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # the smallest call: one token, a small projection; launch latency counts
        dict(name="gemm_m1_k512_n1024", op="gemm", M=1, K=512, N=1024, fmt="int4", group=128, zeros=False),
        # one token through a wide up projection, zero points as most 4-bit checkpoints have them
        dict(name="gemm_m1_k4096_n14336_zeros", op="gemm", M=1, K=4096, N=14336, fmt="int4", group=128, zeros=True),
        # a full decode batch through the long-K down projection on mxfp4 weights
        dict(name="gemm_m16_k14336_n4096_mxfp4", op="gemm", M=16, K=14336, N=4096, fmt="mxfp4", group=32, zeros=False),
        # a speculative or chunked batch, ragged against every tile, the finest groups
        dict(name="gemm_m100_k4096_n4096_g32_zeros", op="gemm", M=100, K=4096, N=4096, fmt="int4", group=32, zeros=True),
        # prefill through the widest projection
        dict(name="gemm_m4096_k4096_n12288_zeros", op="gemm", M=4096, K=4096, N=12288, fmt="int4", group=128, zeros=True),
        # a decode step's sort: 16 tokens, top-8 of 128 experts
        dict(name="permute_t16_h2048", op="permute", T=16, H=2048, E=128, topk=8, dtype="bf16", drop=False),
        # a training batch's sort, some slots sent to experts of another shard
        dict(name="permute_t8192_h2048_drop", op="permute", T=8192, H=2048, E=128, topk=8, dtype="bf16", drop=True),
        # a decode step's way back, weights applied
        dict(name="unpermute_t16_h2048", op="unpermute", T=16, H=2048, E=128, topk=8, dtype="bf16", drop=False),
        # a training batch's gradient of the sort, rows kept in fp32, fewer and wider experts
        dict(name="permute_grad_t4097_h4096_fp32", op="permute_grad", T=4097, H=4096, E=16, topk=2, dtype="fp32",
             drop=False),
        # a training batch's gradient of the way back, for the rows and for the routing weights; an odd token count
        dict(name="unpermute_grad_t8191_h2048", op="unpermute_grad", T=8191, H=2048, E=128, topk=8, dtype="bf16",
             drop=False),
        # a decode step's gate_up products: the sorted rows read through the index, silu * up
        dict(name="experts_gate_up_t16", op="experts", T=16, H=2048, I=768, E=128, topk=8, part="gate_up", fmt="int4",
             group=128, zeros=True),
        # a prefill batch's down products
        dict(name="experts_down_t2048_mxfp4", op="experts", T=2048, H=2048, I=768, E=128, topk=8, part="down",
             fmt="mxfp4", group=32, zeros=False),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def _draw_weight(rng):
    fmt = rng.choice(["int4", "int4", "mxfp4"])
    group = rng.choice([32, 64, 128]) if fmt == "int4" else 32
    return dict(fmt=fmt, group=group, zeros=fmt == "int4" and rng.random() < 0.5)


def draw(rng):
    """A further case of the ranges: single tokens to prefill, narrow to wide, few to many experts."""
    top = max(work(c)["flops"] for c in listed())
    top_bytes = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["gemm", "gemm", "gemm", "permute", "permute_grad", "unpermute", "unpermute_grad", "experts",
                         "experts"])
        if op == "gemm":
            c = dict(op=op, M=_log_int(rng, 1, 4096), K=_log_int(rng, 128, 14336, 128),
                     N=_log_int(rng, 64, 14336, 16), **_draw_weight(rng))
        elif op == "experts":
            E = _log_int(rng, 4, 256)
            c = dict(op=op, T=_log_int(rng, 1, 4096), H=_log_int(rng, 256, 4096, 128),
                     I=_log_int(rng, 128, 2048, 128), E=E, topk=rng.randint(1, min(E, 10)),
                     part=rng.choice(["gate_up", "down"]), **_draw_weight(rng))
        else:
            E = _log_int(rng, 2, 512)
            c = dict(op=op, T=_log_int(rng, 1, 16384), H=_log_int(rng, 64, 8192, 8), E=E,
                     topk=rng.randint(1, min(E, 10)), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                     drop=rng.random() < 0.3)
        w = work(c)
        if w["flops"] <= top and w["bytes"] <= top_bytes:
            return c


def _elem(case):
    return 4 if case.get("dtype") == "fp32" else 2


def _weight_bytes(case, rows, K):
    per_group = 1 if case["fmt"] == "mxfp4" else 2.5 if case["zeros"] else 2  # a zero point holds 4 bits
    return rows * K / 2 + rows * (K / case["group"]) * per_group


def work(case):
    op = case["op"]
    if op == "gemm":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": int(_weight_bytes(case, N, K) + 2 * M * K + 2 * M * N), "flops": 2 * M * N * K}
    T, H, E, k = case["T"], case["H"], case["E"], case["topk"]
    R = T * k
    if op == "experts":
        I = case["I"]
        touched = E * (1.0 - (1.0 - k / E) ** T)  # experts that uniform routing reaches, on average
        if case["part"] == "gate_up":
            return {"bytes": int(touched * _weight_bytes(case, 2 * I, H) + 2 * T * H + 4 * R + 2 * R * I),
                    "flops": 2 * R * H * 2 * I}
        return {"bytes": int(touched * _weight_bytes(case, H, I) + 2 * R * I + 2 * R * H), "flops": 2 * R * I * H}
    kept = int(R * (0.75 if case["drop"] else 1.0))
    b = _elem(case)
    if op == "permute":
        return {"bytes": (T + kept) * H * b + 12 * R + 4 * E, "flops": 0}
    if op == "permute_grad":
        return {"bytes": (T + kept) * H * b + 4 * R, "flops": kept * H}
    if op == "unpermute":
        return {"bytes": (T + kept) * H * b + 8 * R, "flops": 2 * kept * H}
    return {"bytes": (T + 2 * kept) * H * b + 12 * R, "flops": 3 * kept * H}


# ----------------------------------------------------------------- inputs ----

def _rows(gen, n, width, dtype=torch.bfloat16):
    """Activations: normal values, one channel in a hundred twenty times as large."""
    x = torch.randn((n, width), generator=gen, device="cuda")
    x[:, torch.randperm(width, generator=gen, device="cuda")[: width // 100]] *= 20.0
    return x.to(dtype)


def _weight(gen, case, N, K):
    """4-bit weights of normal values: codes [N, K/2] (element 2i in the low half of byte i), scales, zeros."""
    g = case["group"]
    w = (0.02 * torch.randn((N, K), generator=gen, device="cuda")).view(N, K // g, g)
    z = None
    if case["fmt"] == "mxfp4":
        e = torch.floor(torch.log2(w.abs().amax(2).clamp_min(1e-30))) - 2.0
        s = (e + 127.0).clamp(0, 254).to(torch.uint8)
        v = w / torch.exp2(e)[..., None]
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        q = torch.bucketize(v.abs(), edges) + 8 * (v < 0)
    elif case["zeros"]:
        lo, hi = w.amin(2), w.amax(2)
        s = ((hi - lo) / 15.0).to(torch.bfloat16)
        z = torch.round(-lo / s.float()).clamp(0, 15)
        q = (torch.round(w / s.float()[..., None]) + z[..., None]).clamp(0, 15)
        z = z.to(torch.uint8)
    else:
        s = (w.abs().amax(2) / 7.5).to(torch.bfloat16)
        q = (torch.round(w / s.float()[..., None]) + 8.0).clamp(0, 15)
    q = q.to(torch.uint8).view(N, K // 2, 2)
    return q[..., 0] | (q[..., 1] << 4), s, z


def _routing(gen, case):
    """The topk experts of each token by random logits, and their softmax weights."""
    T, E, k = case["T"], case["E"], case["topk"]
    logits, ids = torch.randn((T, E), generator=gen, device="cuda").topk(k, dim=1)
    ids = ids.to(torch.int32)
    if case.get("drop"):  # a quarter of the slots belong to experts elsewhere
        ids = torch.where(torch.rand((T, k), generator=gen, device="cuda") < 0.25, -1, ids)
    return ids.contiguous(), torch.softmax(logits, 1).contiguous()


def _sort(ids, E):
    """Stable sort of the slots by expert: src (slot of each sorted row), pos (row of each slot), offsets."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    kept = key[order] < E
    row = torch.arange(T * k, device=ids.device)
    pos = torch.empty_like(order)
    pos[order] = torch.where(kept, row, -1)
    src = torch.where(kept, order, -1)
    offsets = (key[None, :] < torch.arange(E + 1, device=ids.device)[:, None]).sum(1)
    return src.int(), pos.int().view(T, k), offsets.int()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "gemm":
        st["a"] = _rows(gen, case["M"], case["K"])
        st["w"] = _weight(gen, case, case["N"], case["K"])
        if own:
            r9k = _r9k()
            st["packed"] = r9k.pack_weight_w4(*st["w"])
            st["c"] = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device="cuda")
            need = r9k.gemm_w4_workspace(case["M"], case["K"], case["N"])
            st["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        return st
    T, H, E, k = case["T"], case["H"], case["E"], case["topk"]
    R = T * k
    ids, tw = _routing(gen, case)
    src, pos, offsets = _sort(ids, E)
    if op == "experts":
        N, K = (2 * case["I"], H) if case["part"] == "gate_up" else (H, case["I"])
        parts = [_weight(gen, case, N, K) for _ in range(E)]
        w = tuple(None if p[0] is None else torch.stack(p) for p in zip(*parts))
        st.update(w=w, src=src, offsets=offsets, bounds=offsets.tolist(),
                  x=_rows(gen, T if case["part"] == "gate_up" else R, K))
        if own:
            r9k = _r9k()
            st["packed"] = r9k.pack_weight_w4(*w)
            st["out"] = torch.empty((R, case["I"] if case["part"] == "gate_up" else H), dtype=torch.bfloat16,
                                    device="cuda")
        return st
    dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    st.update(ids=ids, tw=tw, src=src, pos=pos)
    # rows behind the last kept one are nobody's: a program that pads its sorted rows zeroes them once
    if op == "permute":
        st.update(x=_rows(gen, T, H, dtype), xs=torch.zeros((R, H), dtype=dtype, device="cuda"))
        if own:
            need = _r9k().moe_permute_workspace(T, E, k)
            st["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    elif op == "permute_grad":
        st["g"] = _rows(gen, R, H, dtype)
    elif op == "unpermute":
        st["y"] = _rows(gen, R, H, dtype)
    else:
        st.update(g=_rows(gen, T, H, dtype), y=_rows(gen, R, H, dtype),
                  gy=torch.zeros((R, H), dtype=dtype, device="cuda"))
    return st


# ------------------------------------------------------------- plain forms ----

def _dequant(w, fmt, dtype=torch.float32):
    codes, s, z = w
    N = codes.shape[0]
    q = torch.stack((codes & 15, codes >> 4), 2).view(N, -1)
    if fmt == "mxfp4":
        v = torch.tensor(E2M1, dtype=dtype, device=codes.device)[q.long()]
        sc = torch.exp2(s.to(dtype) - 127.0)
    else:
        v, sc = q.to(dtype), s.to(dtype)
    v = v.view(N, s.shape[1], -1)
    if fmt != "mxfp4":
        v = v - (8.0 if z is None else z.to(dtype)[..., None])
    return (v * sc[..., None]).view(N, -1)


def _kept(pos):
    """Rows to read (0 for dropped slots) and which slots are kept."""
    return pos.long().clamp_min(0), (pos >= 0)


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        return (st["a"].float() @ _dequant(st["w"], case["fmt"]).t()).to(torch.bfloat16)
    if op == "experts":
        src, off, x = st["src"], st["bounds"], st["x"]
        I = case["I"]
        gate_up = case["part"] == "gate_up"
        out = torch.empty((src.numel(), I if gate_up else case["H"]), dtype=torch.bfloat16, device=x.device)
        for e in range(case["E"]):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            a = x[src[lo:hi].long() // case["topk"]] if gate_up else x[lo:hi]
            w = _dequant([None if t is None else t[e] for t in st["w"]], case["fmt"])
            p = a.float() @ w.t()
            if gate_up:
                p = p[:, :I] / (1.0 + torch.exp(-p[:, :I])) * p[:, I:]
            out[lo:hi] = p.to(torch.bfloat16)
        return out
    if op == "permute":
        src, pos, offsets = _sort(st["ids"], case["E"])
        kept = src >= 0
        xs = torch.where(kept[:, None], st["x"][src.long().clamp_min(0) // case["topk"]], st["xs"])
        return xs, src, pos, offsets
    row, kept = _kept(st["pos"])
    if op == "permute_grad":
        g = st["g"].float()[row] * kept[..., None]
        return g.sum(1).to(st["g"].dtype)
    if op == "unpermute":
        y = st["y"].float()[row] * (st["tw"] * kept)[..., None]
        return y.sum(1).to(st["y"].dtype)
    g, y = st["g"].float(), st["y"].float()
    gw = (g[:, None, :] * y[row]).sum(2) * kept
    src = st["src"]
    tok = src.long().clamp_min(0)
    gy = g[tok // case["topk"]] * (st["tw"].reshape(-1)[tok] * (src >= 0))[:, None]
    return gy.to(st["g"].dtype), gw


def _calls(st):
    """The framework's operators, as a program that holds its weights, outputs and workspaces calls them."""
    r9k = _r9k()
    case = st["case"]
    op = case["op"]
    if op == "gemm":
        wp, sp, zp = st["packed"]
        return r9k.gemm_w4(st["a"], wp, sp, zp, c=st["c"], workspace=st["workspace"])
    if op == "experts":
        wp, sp, zp = st["packed"]
        if case["part"] == "gate_up":
            return r9k.moe_gemm_w4(st["x"], st["offsets"], wp, sp, zp, src=st["src"], topk=case["topk"],
                                   act="silu_mul", c=st["out"])
        return r9k.moe_gemm_w4(st["x"], st["offsets"], wp, sp, zp, c=st["out"])
    if op == "permute":
        return r9k.moe_permute(st["x"], st["ids"], case["E"], xs=st["xs"], workspace=st["workspace"])
    if op == "permute_grad":
        return r9k.moe_permute_backward(st["g"], st["pos"])
    if op == "unpermute":
        return r9k.moe_unpermute(st["y"], st["pos"], st["tw"])
    return r9k.moe_unpermute_backward(st["g"], st["y"], st["pos"], st["tw"], gy=st["gy"])


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------- exact ----

def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64

    def weights(codes, s, z):
        half = codes.to(torch.int64)
        q = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=f64, device=codes.device)
        if case["fmt"] == "mxfp4":
            mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=f64, device=codes.device) / 2
            for i, h in enumerate((half % 16, half // 16)):
                q[:, i::2] = mag[h % 8] * (1 - 2 * (h // 8))
            sc = torch.pow(torch.tensor(2.0, dtype=f64, device=codes.device), s.to(f64) - 127)
        else:
            q[:, 0::2], q[:, 1::2] = (half % 16).to(f64), (half // 16).to(f64)
            q -= 8 if z is None else z.to(f64).repeat_interleave(case["group"], 1)
            sc = s.to(f64)
        return q * sc.repeat_interleave(case["group"], 1)

    if op == "gemm":
        return torch.matmul(st["a"].to(f64), weights(*st["w"]).T)
    E, k = case["E"], case["topk"]
    if op == "experts":
        codes, s, z = st["w"]
        rows = []
        for e in range(E):
            lo, hi = st["bounds"][e], st["bounds"][e + 1]
            r = torch.arange(lo, hi, device="cuda")
            if case["part"] == "gate_up":
                r = torch.div(st["src"][lo:hi].long(), k, rounding_mode="floor")
            p = torch.matmul(st["x"][r].to(f64), weights(codes[e], s[e], None if z is None else z[e]).T)
            if case["part"] == "gate_up":
                gate, up = p.chunk(2, dim=1)
                p = gate * torch.sigmoid(gate) * up
            rows.append(p)
        return torch.cat(rows)
    ids = (st["ids"] if op == "permute" else None)
    if op == "permute":
        T = case["T"]
        flat = ids.reshape(-1).tolist()
        by = [[] for _ in range(E)]
        for slot, e in enumerate(flat):
            if 0 <= e < E:
                by[e].append(slot)
        order = [slot for lst in by for slot in lst]
        offsets = [0]
        for lst in by:
            offsets.append(offsets[-1] + len(lst))
        pos = [-1] * (T * k)
        for r, slot in enumerate(order):
            pos[slot] = r
        xs = torch.zeros((T * k, case["H"]), dtype=f64, device="cuda")
        xs[: len(order)] = st["x"].to(f64)[torch.tensor(order, dtype=torch.long, device="cuda") // k]
        i32 = dict(dtype=torch.int32, device="cuda")
        return (xs, torch.tensor(order + [-1] * (T * k - len(order)), **i32), torch.tensor(pos, **i32).view(T, k),
                torch.tensor(offsets, **i32))
    pos = st["pos"].long()
    if op in ("permute_grad", "unpermute"):
        rows = st["g" if op == "permute_grad" else "y"].to(f64)
        rows = torch.cat((rows, rows.new_zeros((1, rows.shape[1]))))  # row -1: a dropped slot's
        out = rows.new_zeros((case["T"], case["H"]))
        for j in range(k):
            out += rows[pos[:, j]] * (1.0 if op == "permute_grad" else st["tw"][:, j:j + 1].to(f64))
        return out
    g, y = st["g"].to(f64), st["y"].to(f64)
    gy = torch.zeros_like(y)
    gw = torch.zeros((case["T"], k), dtype=f64, device="cuda")
    for j in range(k):
        t = torch.nonzero(pos[:, j] >= 0).flatten()
        gy[pos[t, j]] = g[t] * st["tw"][t, j:j + 1].to(f64)
        gw[t, j] = torch.linalg.vecdot(g[t], y[pos[t, j]])
    return gy, gw
