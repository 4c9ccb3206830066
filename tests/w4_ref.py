"""Plain 64-bit forms of the 4-bit weight products and of the rows sorted by expert, on the CPU, with the
error bounds that the tests use.  Written from the definitions in include/r9k.h alone.

Bounds.  One rounding to a type t is off by at most half a step, eps(t) / 2 of the value.  An fp32 sum of n
terms in any order is off by at most n * u of the sum of the terms' magnitudes, u = 2^-23 for each addition (a
whole step, not half of one: the matrix instruction's adder may truncate).  In a product with a 4-bit weight
every a * q is exact in fp32; a term passes at most K additions in all, and 4 more roundings when its group is
scaled and added; so |sum - exact| <= (K + 4) * 2^-23 * M, M the sum of the magnitudes of all terms, which for int4 are
s * |a| * q and s * |a| * z (the zero point is subtracted as a sum of its own), for mxfp4 |a * value|."""
import numpy as np
import torch

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
F64 = torch.float64


def codes_of(wq: torch.Tensor) -> torch.Tensor:
    """[..., K/2] bytes -> [..., K] codes, the low half of a byte first."""
    b = wq.cpu().to(torch.int64)
    return torch.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1)


def dequant(wq, s, z, group):
    """(values, magnitudes) [..., N, K] in 64 bits: the weight, and s * (q + z) (the terms' size in a product)."""
    q = codes_of(wq)
    rep = lambda t: t.cpu().to(F64).repeat_interleave(group, -1)
    if s.dtype == torch.uint8:
        v = torch.from_numpy(E2M1)[q & 7] * torch.where(q >= 8, -1.0, 1.0) * torch.exp2(rep(s) - 127.0)
        return v, v.abs()
    zz = torch.full(s.shape, 8.0, dtype=F64).repeat_interleave(group, -1) if z is None else rep(z)
    return (q - zz) * rep(s), (q + zz) * rep(s).abs()


def product(a, wq, s, z, group):
    """(c, bound on an fp32 sum's error) of a [M,K] with the weight [N,K], 64 bits."""
    v, mag = dequant(wq, s, z, group)
    x = a.cpu().to(F64)
    return x @ v.T, (x.shape[1] + 4) * 2.0 ** -23 * (x.abs() @ mag.T)


def bf16_bound(want, before):
    """Bound for an output rounded once to bf16 whose fp32 value is within `before` of `want`."""
    return before + 2.0 ** -8 * (want.abs() + before)


def silu_mul(gate, up, dg, du):
    """silu(gate) * up and a bound on its fp32 value's error, for factors known to dg and du: |silu'| <= 1.1, and
    expf, the sum, the division and the product lose at most 8 * 2^-24 of the value together."""
    h = gate * torch.sigmoid(gate)
    p = h * up
    return p, 1.1 * dg * (up.abs() + du) + h.abs() * du + 8 * 2.0 ** -24 * (p.abs() + 1.1 * dg * up.abs() + h.abs() * du)


def quant(w, group, mxfp4=False, zeros=False):
    """r9k_quant_weight_w4's rule on bf16 w [N,K], in fp32 -> codes [N,K], scales, zeros (numpy)."""
    f = w.float().numpy().astype(np.float32)
    g = f.reshape(f.shape[0], -1, group)
    one = np.float32
    if mxfp4:
        amax = np.abs(g).max(2)
        e = np.clip((amax.view(np.uint32) >> 23).astype(np.int64) - 2, 1, 254)
        v = np.abs(g.astype(np.float64)) * np.exp2(127.0 - e)[..., None]
        lo, hi = np.zeros_like(v, np.int64), None
        # nearest value, ties to the even code, by comparing distances
        d = np.abs(v[..., None] - E2M1)
        best = d.min(-1)
        cand = d == best[..., None]
        first = cand.argmax(-1)
        last = 7 - cand[..., ::-1].argmax(-1)
        m = np.where(first == last, first, np.where(first % 2 == 0, first, last))
        q = m + 8 * np.signbit(g)
        return q.reshape(f.shape), e.astype(np.uint8), None

    def bf16(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
    lo, hi = np.minimum(g.min(2), one(0)), np.maximum(g.max(2), one(0))
    if zeros:
        s = bf16(np.maximum(hi - lo, one(1e-10)) / one(15))
        z = np.clip(np.rint(-lo / s.float().numpy()), 0, 15)
    else:
        s = bf16(np.maximum(np.maximum(-lo, hi), one(1e-10)) / one(7))
        z = np.full(lo.shape, 8, np.float32)
    q = np.clip(np.rint(g / s.float().numpy()[..., None]) + z[..., None], 0, 15).astype(np.int64)
    return q.reshape(f.shape), s, z.astype(np.uint8) if zeros else None


def sort(ids, E):
    """Stable sort of the slots: (src, pos, offsets) as r9k_moe_permute defines them (numpy, one slot at a time)."""
    T, k = ids.shape
    rows = [[] for _ in range(E)]
    for p, e in enumerate(ids.reshape(-1).tolist()):
        if 0 <= e < E:
            rows[e].append(p)
    src = np.full(T * k, -1, np.int32)
    pos = np.full(T * k, -1, np.int32)
    off = np.zeros(E + 1, np.int32)
    r = 0
    for e in range(E):
        for p in rows[e]:
            src[r], pos[p] = p, r
            r += 1
        off[e + 1] = r
    return src, pos.reshape(T, k), off


def unpermute(y, pos, w):
    """(out, sum of |terms|) in 64 bits; y [R,H], pos [T,k], w [T,k] or None."""
    y = y.cpu().to(F64)
    T, k = pos.shape
    out, mag = torch.zeros(T, y.shape[1], dtype=F64), torch.zeros(T, y.shape[1], dtype=F64)
    for j in range(k):
        p = torch.as_tensor(pos[:, j]).long()
        ok = (p >= 0).to(F64)[:, None]
        g = torch.ones(T, 1, dtype=F64) if w is None else w.cpu().to(F64)[:, j:j + 1]
        term = y[p.clamp_min(0)] * g * ok if y.shape[0] else torch.zeros_like(out)
        out += term
        mag += term.abs()
    return out, mag
