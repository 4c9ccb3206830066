"""4-bit weights: the quantiser, the packed layout and the products, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import inputs
from tests import w4_ref as ref
from tests.gpu_util import dev, say

pytestmark = pytest.mark.gpu
# (format, group, zeros)
FORMATS = [("int4", 32, False), ("int4", 32, True), ("int4", 64, False), ("int4", 64, True), ("int4", 128, False),
           ("int4", 128, True), ("mxfp4", 32, False)]


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


def _fmt(r9k, fmt):
    return r9k.W4_INT if fmt == "int4" else r9k.W4_MXFP4


def weight(lead, K, fmt, group, zeros, seed, wild=False):
    """Random codes, scales and zeros (all code values; `wild`: scales over many powers of two)."""
    g = np.random.default_rng(seed)
    wq = torch.from_numpy(g.integers(0, 256, (*lead, K // 2), dtype=np.uint8))
    if fmt == "mxfp4":
        s = torch.from_numpy(g.integers(90, 165, (*lead, K // group)) if wild else g.integers(118, 124, (*lead, K // group)))
        return wq, s.to(torch.uint8), None
    s = g.standard_normal((*lead, K // group)) * 0.01
    if wild:
        s = s * np.exp2(g.integers(-30, 30, s.shape))
    z = torch.from_numpy(g.integers(0, 16, s.shape, dtype=np.uint8)) if zeros else None
    return wq, torch.from_numpy(s).to(torch.bfloat16), z


def packed(r9k, w):
    return r9k.pack_weight_w4(*(None if t is None else t.cuda() for t in w))


def acts(M, K, seed):
    return torch.from_numpy(inputs.activations(seed, M, K).view(np.int16)).view(torch.bfloat16)


# ------------------------------------------------------------ load time ----

@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("N,K", [(16, 128), (48, 384), (256, 1024)])
def test_quantiser(r9k, fmt, group, zeros, N, K):
    say("quant_weight_w4", fmt, group, zeros, N, K)
    w = torch.from_numpy(inputs.weights(N + group, N, K).view(np.int16)).view(torch.bfloat16).clone()
    w[0] = 0                                           # a row of zeros
    w[1, :group] = torch.linspace(-6, 6, group).to(torch.bfloat16)
    w[2, :group] = torch.arange(group).to(torch.bfloat16) / 4 - 4   # ties in both formats
    w[3] = w[3].abs()                                  # one sign: the range still holds 0
    w[4] = -w[4].abs()
    w[5] = 1e-38
    w[6] = 3e38
    w[7, ::2] = 1e-30
    q, s, z = r9k.quant_weight_w4(w.cuda(), group, _fmt(r9k, fmt), zeros)
    rq, rs, rz = ref.quant(w, group, fmt == "mxfp4", zeros)
    assert np.array_equal(ref.codes_of(q).numpy(), rq)
    if fmt == "mxfp4":
        assert np.array_equal(s.cpu().numpy(), rs)
    else:
        assert torch.equal(s.cpu().view(torch.int16), rs.view(torch.int16))
    assert (z is None and rz is None) or np.array_equal(z.cpu().numpy(), rz)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_packed_copy_holds_the_same_values(r9k, fmt, group, zeros):
    """Products with unit rows give the weight's columns: every code, scale and zero is where the kernel reads it.
    One term of a sum is not zero, so the fp32 value is exact to one rounding of q * s - z * s."""
    N, K = 80, 256
    w = weight((N,), K, fmt, group, zeros, 3, wild=True)
    a = torch.eye(K, dtype=torch.bfloat16)
    got = r9k.gemm_w4(a.cuda(), *packed(r9k, w)).cpu().to(ref.F64)
    want, mag = ref.dequant(*w, group)
    assert torch.all((got - want.T).abs() <= ref.bf16_bound(want.T, 4 * 2.0 ** -23 * mag.T))
    if fmt == "mxfp4":
        assert torch.equal(got, want.T)


def test_mxfp4_scales_at_the_ends(r9k):
    """Scale bytes 1 (2^-126) and 254 (2^127): the smallest weights and products are bf16 subnormals."""
    N, K = 16, 128
    wq = torch.full((N, K // 2), 0x21, dtype=torch.uint8)        # 0.5, 1
    for byte in (1, 2, 100, 253, 254):
        s = torch.full((N, 4), byte, dtype=torch.uint8)
        a = torch.zeros((2, K), dtype=torch.bfloat16)
        a[0, 0], a[1, 1] = 2.0, 0.5
        got = r9k.gemm_w4(a.cuda(), *packed(r9k, (wq, s, None))).cpu()
        want = torch.tensor([1.0, 0.5], dtype=ref.F64) * 2.0 ** (byte - 127)
        assert torch.equal(got.to(ref.F64), want[:, None].expand(2, N).contiguous()), byte


# ------------------------------------------------------------- products ----

def check(r9k, a, w, group, packed_w, what):
    got = r9k.gemm_w4(a.cuda(), *packed_w)
    want, before = ref.product(a, *w, group)
    err, bound = (got.cpu().to(ref.F64) - want).abs(), ref.bf16_bound(want, before)
    assert torch.all(err <= bound), f"{what}: {float((err / bound).max()):.3f} of the bound"
    # the bound above holds for any order of the sum; a typical sum is far closer, and a wrong term far off:
    # root mean square within one bf16 rounding (half a step, 2^-8, is its largest; its mean square is below a third)
    rms = lambda t: float(t.square().mean().sqrt())
    assert rms(err) <= 2.0 ** -8 * rms(want) + 1e-30, f"{what}: rms {rms(err) / rms(want):.2e}"
    return got


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,K,N", [(1, 128, 16), (1, 512, 1024), (2, 1280, 48), (5, 256, 272), (16, 896, 128),
                                   (17, 2048, 64), (33, 384, 80), (65, 640, 528), (130, 1024, 144), (257, 256, 400),
                                   (300, 4224, 96), (700, 512, 1040)])
def test_product(r9k, fmt, group, zeros, M, K, N):
    say("gemm_w4", fmt, group, zeros, M, K, N)
    w = weight((N,), K, fmt, group, zeros, M + K + N)
    p = packed(r9k, w)
    a = acts(M, K, M + N)
    c = check(r9k, a, w, group, p, f"{fmt} g{group} {M}x{K}x{N}")
    assert torch.equal(r9k.gemm_w4(a.cuda(), *p), c)             # the same bits again


@pytest.mark.parametrize("M,K,N,fmt,group,zeros", [(1, 14336, 4096, "int4", 128, True), (16, 4096, 14336, "mxfp4", 32, False),
                                                   (3, 16384, 1024, "int4", 64, False), (100, 4096, 4096, "int4", 32, True),
                                                   (1, 4096, 32000, "int4", 128, False), (64, 14336, 2048, "mxfp4", 32, False),
                                                   (1500, 2048, 2064, "int4", 128, True)])
def test_product_of_a_model(r9k, M, K, N, fmt, group, zeros):
    say("gemm_w4", fmt, group, zeros, M, K, N)
    w = weight((N,), K, fmt, group, zeros, K)
    check(r9k, acts(M, K, N), w, group, packed(r9k, w), f"{fmt} g{group} {M}x{K}x{N}")


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_every_row_count_agrees(r9k, fmt, group, zeros):
    """A row's result within its bound at every row count around the tiles' edges, and rows do not reach each other."""
    K, N = 512, 160
    w = weight((N,), K, fmt, group, zeros, 9)
    p = packed(r9k, w)
    a = acts(300, K, 4)
    want, before = ref.product(a, *w, group)
    bound = ref.bf16_bound(want, before)
    for M in (1, 2, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300):
        say("rows", M)
        c = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
        r9k.gemm_w4(a[:M].contiguous().cuda(), *p, c=c[:M])
        assert torch.all((c[:M].cpu().to(ref.F64) - want[:M]).abs() <= bound[:M]), M
        assert torch.all(c[M:] == 7.0), M                         # nothing behind the last row


def test_wide_scales_and_values(r9k):
    for fmt, group, zeros in FORMATS:
        w = weight((64,), 1024, fmt, group, zeros, 21, wild=True)
        a = acts(9, 1024, 2).float() * torch.exp2(torch.arange(9.0)[:, None] * 8 - 32)
        a[4] = 0
        a = a.to(torch.bfloat16)
        want, before = ref.product(a, *w, group)
        got = r9k.gemm_w4(a.cuda(), *packed(r9k, w)).cpu()
        assert torch.all((got.to(ref.F64) - want).abs() <= ref.bf16_bound(want, before)), fmt
        assert torch.all(got[4] == 0)


def test_streams_workspaces_and_graphs(r9k):
    """A side stream with its own allocations, a caller's workspace with anything in it, and two captured graphs
    replayed in turn with other work between them."""
    shapes = [(1, 4096, 1024), (48, 2048, 512), (200, 2048, 1024)]
    calls = []
    for i, (M, K, N) in enumerate(shapes):
        w = weight((N,), K, "int4", 128, True, i)
        p, a = packed(r9k, w), acts(M, K, i).cuda()
        c = r9k.gemm_w4(a, *p)
        need = r9k.gemm_w4_workspace(M, K, N)
        ws = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(r9k.gemm_w4(a, *p, workspace=ws), c)
        calls.append((a, p, c))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [r9k.gemm_w4(a, *p, stream=side) for a, p, _ in calls]
    side.synchronize()
    assert all(torch.equal(o, c) for o, (_, _, c) in zip(outs, calls))
    graphs = []
    for a, p, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = r9k.gemm_w4(a, *p)
        graphs.append((g, o))
    for _ in range(4):
        for (g, o), (a, p, c) in zip(graphs, calls):
            o.zero_()
            g.replay()
            assert torch.equal(r9k.gemm_w4(a, *p), c)
        torch.cuda.synchronize()
        assert all(torch.equal(o, c) for (_, o), (_, _, c) in zip(graphs, calls))


def test_refusals(r9k):
    w = weight((32,), 256, "int4", 64, True, 1)
    wp, sp, zp = packed(r9k, w)
    a = acts(2, 256, 1).cuda()
    with pytest.raises(ValueError):
        r9k.gemm_w4(a[:, :128].contiguous(), wp, sp, zp)             # another K
    with pytest.raises(ValueError):
        r9k.gemm_w4(a, wp, sp[:, :3].contiguous(), zp)               # groups that do not divide K
    with pytest.raises(ValueError):
        r9k.gemm_w4(a, wp, sp, zp[:, :2].contiguous())
    with pytest.raises(ValueError):
        r9k.gemm_w4(a, wp[:16], sp, zp)
    with pytest.raises(ValueError):
        r9k.gemm_w4(a.t().contiguous().t(), wp, sp, zp)              # a strided view
    with pytest.raises(ValueError):
        r9k.gemm_w4(a, wp, sp, zp, c=torch.empty((2, 48), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        r9k.gemm_w4(a.half(), wp, sp, zp)
    with pytest.raises(TypeError):
        r9k.gemm_w4(a, wp, sp.float(), zp)
    with pytest.raises(r9k.R9kError) as e:
        r9k.gemm_w4(a, wp, torch.zeros((32, 4), dtype=torch.uint8, device="cuda"), None)   # mxfp4 in groups of 64
    assert e.value.code == -7
    with pytest.raises(r9k.R9kError) as e:
        r9k.gemm_w4(a, wp, torch.zeros((32, 8), dtype=torch.uint8, device="cuda"),
                    torch.zeros((32, 8), dtype=torch.uint8, device="cuda"))                # mxfp4 with zeros
    assert e.value.code == -7
    with pytest.raises(ValueError):
        r9k.pack_weight_w4(w[0][:24].contiguous().cuda(), w[1][:24].contiguous().cuda())   # 24 rows
    with pytest.raises(ValueError):
        r9k.quant_weight_w4(torch.zeros((16, 128), dtype=torch.bfloat16, device="cuda"), group=96)
    with pytest.raises(r9k.R9kError) as e:
        r9k.quant_weight_w4(torch.zeros((16, 128), dtype=torch.bfloat16, device="cuda"), group=16)
    assert e.value.code == -7
    assert r9k.gemm_w4(torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), wp, sp, zp).shape == (0, 32)


# ------------------------------------------------------ experts' products ----

def _routing(T, k, E, kind, seed):
    g = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), E // 2, np.int32)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if kind != "skew" else \
        np.minimum(g.geometric(0.4, (T, k)) - 1, E - 1).astype(np.int32)
    if kind == "drop":
        ids[g.random((T, k)) < 0.4] = -1
    return ids


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M", [7, 33, 150])
def test_a_row_without_a_finite_value_stays_alone(r9k, fmt, group, zeros, M):
    """An infinity or NaN among a row's activations: no finite value in that row of the product, and the other rows are
    to the bit what they are without it, dense and as experts' rows."""
    say("gemm_w4 non-finite", fmt, group, zeros, M)
    K, N, E = 512, 96, 2
    w = weight((E, N), K, fmt, group, zeros, 31)
    p, x = packed(r9k, w), acts(M, K, 4)
    y = x.clone()
    bad = [0, 3, 5, M - 1]
    for r, k, v in zip(bad, (0, 200, K - 1, 77), (float("inf"), float("nan"), -float("inf"), float("inf"))):
        y[r, k] = v
    good = torch.ones(M, dtype=torch.bool)
    good[bad] = False
    off = torch.tensor([0, 4, M], dtype=torch.int32).cuda()
    one = tuple(None if t is None else t[0].contiguous() for t in p)
    for f in (lambda t: r9k.gemm_w4(t.cuda(), *one), lambda t: r9k.moe_gemm_w4(t.cuda(), off, *p),
              lambda t: r9k.moe_gemm_w4(t.cuda(), off, *p, act="silu_mul")):
        fine, got = f(x).cpu(), f(y).cpu()
        assert torch.all(torch.isfinite(fine)) and torch.equal(got[good], fine[good])
        assert not torch.any(torch.isfinite(got[bad]))


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("T,k,E,K,N,kind", [(1, 1, 1, 128, 32, "rand"), (1, 8, 16, 256, 96, "rand"), (5, 2, 7, 384, 64, "drop"),
                                            (16, 4, 32, 256, 224, "rand"), (40, 2, 3, 256, 160, "rand"),
                                            (90, 3, 6, 128, 64, "skew"), (150, 2, 4, 256, 96, "one"),
                                            (400, 2, 70, 128, 32, "skew"), (700, 2, 3, 256, 288, "drop")])
def test_experts(r9k, fmt, group, zeros, T, k, E, K, N, kind):
    say("moe_gemm_w4", fmt, group, zeros, T, k, E, K, N, kind)
    ids = _routing(T, k, E, kind, T)
    src, pos, off = ref.sort(ids, E)
    n = int(off[E])
    w = weight((E, N), K, fmt, group, zeros, T + N)
    p = packed(r9k, w)
    x = acts(T, K, T)
    s = torch.from_numpy(src[:n]).long()
    rows = x[s // k]
    want, before = torch.zeros((n, N), dtype=ref.F64), torch.zeros((n, N), dtype=ref.F64)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            want[lo:hi], before[lo:hi] = ref.product(rows[lo:hi], w[0][e], w[1][e], None if w[2] is None else w[2][e], group)
    offd, srcd = torch.from_numpy(off).cuda(), torch.from_numpy(src).cuda()

    c = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    r9k.moe_gemm_w4(x.cuda(), offd, *p, src=srcd, topk=k, c=c)
    assert torch.all((c[:n].cpu().to(ref.F64) - want).abs() <= ref.bf16_bound(want, before))
    assert torch.all(c[n:] == 7.0)                                # rows behind the last kept one
    xs = torch.zeros((T * k, K), dtype=torch.bfloat16)
    xs[:n] = rows
    c2 = torch.full_like(c, 7.0)
    r9k.moe_gemm_w4(xs.cuda(), offd, *p, c=c2)                    # the sorted copy: the same sums
    assert torch.equal(c2, c)

    h = torch.full((T * k, N // 2), 7.0, dtype=torch.bfloat16, device="cuda")
    r9k.moe_gemm_w4(x.cuda(), offd, *p, src=srcd, topk=k, act="silu_mul", c=h)
    I = N // 2
    wh, bh = ref.silu_mul(want[:, :I], want[:, I:], before[:, :I], before[:, I:])
    assert torch.all((h[:n].cpu().to(ref.F64) - wh).abs() <= ref.bf16_bound(wh, bh))
    assert torch.all(h[n:] == 7.0)


def test_bad_offsets_and_indexes_stay_inside(r9k):
    """Device data the host cannot check: offsets beyond the rows are held to them, an index beyond the tokens reads row
    0; the rows of the other experts are right."""
    T, E, K, N = 6, 3, 128, 32
    w = weight((E, N), K, "int4", 128, False, 1)
    p, x = packed(r9k, w), acts(T, K, 2)
    off = torch.tensor([-4, 2, 4, 99], dtype=torch.int32).cuda()
    src = torch.tensor([0, 1, 2, 2 ** 31 - 1, -9, 5], dtype=torch.int32).cuda()
    c = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    r9k.moe_gemm_w4(x.cuda(), off, *p, src=src, c=c[:T])
    rows = x[torch.tensor([0, 1, 2, 0, 0, 5])]
    for e, (lo, hi) in enumerate(((0, 2), (2, 4), (4, 6))):
        want, before = ref.product(rows[lo:hi], w[0][e], w[1][e], None, 128)
        assert torch.all((c[lo:hi].cpu().to(ref.F64) - want).abs() <= ref.bf16_bound(want, before)), e
    assert torch.all(c[T:] == 7.0)


def test_experts_refusals(r9k):
    w = weight((4, 48), 128, "int4", 128, False, 1)
    p = packed(r9k, w)
    x, off = acts(8, 128, 1).cuda(), torch.zeros(5, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        r9k.moe_gemm_w4(x, off[:4].contiguous(), *p)
    with pytest.raises(ValueError):
        r9k.moe_gemm_w4(x, off, *p, act="gelu")
    with pytest.raises(TypeError):
        r9k.moe_gemm_w4(x, off.long(), *p)
    with pytest.raises(r9k.R9kError) as e:
        r9k.moe_gemm_w4(x, off, *p, act="silu_mul")               # 48 columns: the halves are not whole tiles
    assert e.value.code == -2
    with pytest.raises(r9k.R9kError) as e:
        r9k.moe_gemm_w4(x, off, *p, src=torch.zeros(8, dtype=torch.int32, device="cuda"), topk=0)
    assert e.value.code == -2
    assert r9k.moe_gemm_w4(x[:0], off, *p).shape == (0, 48)


# ------------------------------------------------ the operators together ----

@pytest.mark.parametrize("T,H,E,I,k,fmt,group,zeros", [(1, 256, 8, 128, 2, "int4", 128, True), (16, 512, 32, 256, 8, "mxfp4", 32, False),
                                                       (33, 256, 5, 384, 3, "int4", 32, False), (300, 256, 16, 128, 4, "int4", 64, True)])
def test_moe_layer(r9k, T, H, E, I, k, fmt, group, zeros):
    """Routing, the sort, gate_up read through its index, down, and the way back, as a layer runs them; eager, and as
    one captured graph replayed with eager work between."""
    say("moe layer", T, H, E, I, k, fmt)
    w13 = weight((E, 2 * I), H, fmt, group, zeros, 1)
    w2 = weight((E, H), I, fmt, group, zeros, 2)
    p13, p2 = packed(r9k, w13), packed(r9k, w2)
    x = acts(T, H, 3)
    logits = torch.from_numpy(inputs.router_logits(5, T, E)).cuda()
    xd = x.cuda()

    def layer():
        ids, tw = r9k.moe_route(logits, k)
        _, src, pos, off = r9k.moe_permute(None, ids, E)
        h = r9k.moe_gemm_w4(xd, off, *p13, src=src, topk=k, act="silu_mul")
        y = r9k.moe_gemm_w4(h, off, *p2)
        return ids, tw, h, y, r9k.moe_unpermute(y, pos, tw)

    ids, tw, h, y, out = layer()
    src, pos, off = ref.sort(ids.cpu().numpy(), E)
    one = lambda w, e: [None if t is None else t[e] for t in w]
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        rows = x[torch.from_numpy(src[lo:hi]).long() // k]
        p, b = ref.product(rows, *one(w13, e), group)
        wh, bh = ref.silu_mul(p[:, :I], p[:, I:], b[:, :I], b[:, I:])
        assert torch.all((h[lo:hi].cpu().to(ref.F64) - wh).abs() <= ref.bf16_bound(wh, bh)), e
        p, b = ref.product(h[lo:hi].cpu(), *one(w2, e), group)       # from the kernel's own h
        assert torch.all((y[lo:hi].cpu().to(ref.F64) - p).abs() <= ref.bf16_bound(p, b)), e
    want, mag = ref.unpermute(y, pos, tw)
    before = (k + 1) * 2.0 ** -23 * mag
    assert torch.all((out.cpu().to(ref.F64) - want).abs() <= ref.bf16_bound(want, before))
    # the copied rows give the same products
    xs, src2, _, off2 = r9k.moe_permute(xd, ids, E)
    assert torch.equal(r9k.moe_gemm_w4(xs, off2, *p13, act="silu_mul"), h)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = layer()
    for _ in range(3):
        got[-1].zero_()
        g.replay()
        again = layer()[-1]
        torch.cuda.synchronize()
        assert torch.equal(got[-1], out) and torch.equal(again, out)


# ------------------------------------------------------------ far and wide ----

@pytest.mark.parametrize("seed", range(24))
def test_drawn_products(r9k, seed):
    """Shapes drawn over the whole range, the sizes' logarithms uniform; every format in turn."""
    g = np.random.default_rng(900 + seed)
    draw = lambda lo, hi, step: max(lo, int(round(np.exp(g.uniform(np.log(lo), np.log(hi))) / step)) * step)
    fmt, group, zeros = FORMATS[seed % len(FORMATS)]
    M, K, N = draw(1, 500, 1), draw(128, 9000, 128), draw(16, 3000, 16)
    say("drawn", M, K, N, fmt, group, zeros)
    w = weight((N,), K, fmt, group, zeros, seed)
    check(r9k, acts(M, K, seed), w, group, packed(r9k, w), f"{fmt} g{group} {M}x{K}x{N}")


@pytest.mark.parametrize("fmt,group,zeros", [("int4", 128, True), ("mxfp4", 32, False)])
@pytest.mark.parametrize("T,k,E,K,N", [(300, 2, 600, 128, 32), (20, 64, 2048, 128, 64), (2000, 4, 300, 256, 64),
                                       (3000, 10, 2048, 128, 32), (4000, 1, 1, 256, 96), (6, 3, 5, 8192, 32),
                                       (60, 2, 3, 8192, 32), (5, 1, 2, 24576, 16 * 3 * 2)])
def test_many_experts_and_long_rows(r9k, fmt, group, zeros, T, k, E, K, N):
    say("experts", T, k, E, K, N, fmt)
    ids = _routing(T, min(k, E), E, "rand", T + 1)
    k = ids.shape[1]
    src, pos, off = ref.sort(ids, E)
    w = weight((E, N), K, fmt, group, zeros, T)
    x = acts(T, K, T)
    c = r9k.moe_gemm_w4(x.cuda(), torch.from_numpy(off).cuda(), *packed(r9k, w), src=torch.from_numpy(src).cuda(), topk=k)
    c = c.cpu().to(ref.F64)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            want, before = ref.product(x[torch.from_numpy(src[lo:hi]).long() // k], w[0][e], w[1][e],
                                       None if w[2] is None else w[2][e], group)
            assert torch.all((c[lo:hi] - want).abs() <= ref.bf16_bound(want, before)), e


@pytest.mark.parametrize("rows", [70000, 140000])
@pytest.mark.parametrize("R", [9, 150])
def test_activations_past_32_bit_offsets(r9k, rows, R):
    """Token rows beyond 2 GiB and beyond 4 GiB, read through the index, by either kernel."""
    K, N, E = 16384, 64, 2
    say("far rows", rows, R)
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    g = np.random.default_rng(rows)
    pick = np.sort(np.append(g.integers(0, rows, R - 2), [0, rows - 1])).astype(np.int32)
    a = acts(R, K, R)
    x[torch.from_numpy(pick).long().cuda()] = a.cuda()      # (a row picked twice holds one of its two)
    a = x[torch.from_numpy(pick).long().cuda()].cpu()
    w = weight((E, N), K, "int4", 64, True, 3)
    off = torch.tensor([0, R // 3, R], dtype=torch.int32)
    c = r9k.moe_gemm_w4(x, off.cuda(), *packed(r9k, w), src=torch.from_numpy(pick).cuda()).cpu().to(ref.F64)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        want, before = ref.product(a[lo:hi], w[0][e], w[1][e], w[2][e], 64)
        assert torch.all((c[lo:hi] - want).abs() <= ref.bf16_bound(want, before)), e


@pytest.mark.parametrize("R", [5, 2000])
def test_weights_past_4_gib(r9k, R):
    """Experts' codes of 4.3 GiB: the first and the last expert's products, on some of their columns."""
    E, N, K, group = 34, 16384, 16384, 128
    say("far weights", R)
    wq = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = (torch.rand((E, N, K // group), device="cuda") * 0.01).to(torch.bfloat16)
    p = r9k.pack_weight_w4(wq, s)
    x = acts(R, K, R)
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = R // 2
    off[E] = R
    c = r9k.moe_gemm_w4(x.cuda(), off.cuda(), *p)
    cols = torch.cat((torch.arange(0, 16), torch.arange(N - 16, N)))
    for e, lo, hi in ((0, 0, R // 2), (E - 1, R // 2, R)):
        rows = torch.unique(torch.tensor([lo, (lo + hi) // 2, hi - 1]))
        want, before = ref.product(x[rows], wq[e][cols.cuda()].cpu(), s[e][cols.cuda()].cpu(), None, group)
        got = c[rows.cuda()][:, cols.cuda()].cpu().to(ref.F64)
        assert torch.all((got - want).abs() <= ref.bf16_bound(want, before)), e
