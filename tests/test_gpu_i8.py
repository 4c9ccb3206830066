"""Products in 8-bit integers: the quantiser, the packed layout and the products, against plain forms."""
import numpy as np
import pytest
import torch

import inputs
from tests import i8_ref as ref
from tests import w4_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


def weight(lead, K, seed, wild=False):
    """Random codes, -128 among them, and scales (`wild`: over many powers of two)."""
    g = np.random.default_rng(seed)
    wq = torch.from_numpy(g.integers(-128, 128, (*lead, K), dtype=np.int8))
    s = np.abs(g.standard_normal(lead)) * 0.001 + 1e-5
    if wild:
        s = s * np.exp2(g.integers(-40, 40, s.shape))
    return wq, torch.from_numpy(s.astype(np.float32))


def acts(M, K, seed):
    return torch.from_numpy(inputs.activations(seed, M, K).view(np.int16)).view(torch.bfloat16)


# ------------------------------------------------------------ quantiser ----

@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (17, 1024), (5, 4096), (9, 4224), (4, 14336), (2, 16384), (3, 20480),
                                    (2, 130944), (1024, 128), (1500, 1152), (2049, 2048), (1100, 2176), (1030, 4096)])
def test_quantiser(r9k, rows, K):
    say("quant_i8", rows, K)
    x = acts(rows, K, rows + K).clone()
    x[0, :] = 0 if rows > 1 else x[0, :]
    if rows > 2:
        x[1] = (torch.arange(K) % 255 - 127).to(torch.bfloat16) / 2      # whole after scaling by 2
        x[2, K // 2] = 3e38
    q, s = r9k.quant_i8(x.cuda())
    rq, rs = ref.quant(x)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(q.cpu(), rq)
    g = torch.full((rows + 1, K), 9, dtype=torch.int8, device="cuda")
    h = torch.full((rows + 1,), 9.0, device="cuda")
    r9k.quant_i8(x.cuda(), q=g[:rows], s=h[:rows])
    assert torch.equal(g[:rows], q) and torch.all(g[rows:] == 9) and float(h[rows]) == 9.0


def test_quantiser_at_the_ends(r9k):
    """Tiny rows, the largest values, ties on both sides, and rows that are not finite."""
    K = 128
    x = torch.zeros((9, K), dtype=torch.bfloat16)
    x[1] = 1e-38
    x[2, ::2] = 1e-10
    x[3] = torch.finfo(torch.bfloat16).max
    x[4] = -torch.finfo(torch.bfloat16).max
    x[5] = torch.linspace(-127, 127, K).to(torch.bfloat16)
    x[5, 0] = 127.0
    x[5, 1:9] = torch.tensor([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5])
    x[6, 77] = float("inf")
    x[7, 3] = float("nan")
    x[8, 127], x[8, 126] = -float("inf"), float("nan")
    q, s = r9k.quant_i8(x.cuda())
    rq, rs = ref.quant(x)
    assert torch.equal(q.cpu(), rq)
    assert torch.equal(s.cpu()[:6], rs[:6]) and torch.isnan(s.cpu()[6:]).all() and torch.all(q.cpu()[6:] == 0)
    assert int(q.min()) == -127 and int(q.max()) == 127
    # the rule in words: the largest value becomes 127, and no value is further than half a step from its code
    back = q.cpu().to(ref.F64) * s.cpu().to(ref.F64)[:, None]
    assert torch.all((back - x.to(ref.F64))[:6].abs() <= (0.5 + 127 * 4 * ref.U) * s.cpu().to(ref.F64)[:6, None])


# ------------------------------------------------------------- products ----

def check(r9k, aq, as_, w, p, what):
    got = r9k.gemm_i8(aq.cuda(), as_.cuda(), p, w[1].cuda())
    want, before = ref.product(aq, as_, *w)
    assert torch.all((got.cpu().to(ref.F64) - want).abs() <= ref.bf16_bound(want, before)), what
    assert torch.equal(got.cpu(), ref.product32(aq, as_, *w).to(torch.bfloat16)), what
    return got


@pytest.mark.parametrize("M,K,N", [(1, 128, 16), (1, 512, 1024), (2, 1280, 48), (5, 256, 272), (16, 896, 128),
                                   (17, 2048, 64), (33, 384, 80), (65, 640, 528), (130, 1024, 144), (257, 256, 400),
                                   (300, 4224, 96), (700, 512, 1040), (64, 4096, 4096), (1, 14336, 4096), (20, 14336, 1024),
                                   (1, 130944, 32), (1500, 2048, 2064), (100, 4096, 4096)])
def test_product(r9k, M, K, N):
    say("gemm_i8", M, K, N)
    w = weight((N,), K, M + K + N, wild=True)
    p = r9k.pack_weight_i8(w[0].cuda())
    a = acts(M, K, M + N)
    aq, as_ = ref.quant(a)
    c = check(r9k, aq, as_, w, p, f"{M}x{K}x{N}")
    assert torch.equal(r9k.gemm_i8(aq.cuda(), as_.cuda(), p, w[1].cuda()), c)        # the same bits again
    assert torch.equal(r9k.gemm_i8_qa(a.cuda(), p, w[1].cuda()), c)                  # and from bf16 activations


def test_largest_sums(r9k):
    """Every product 2^14 at the longest K: the sum is 2145386496 of 2^31."""
    K, N, M = 130944, 16, 2
    wq = torch.full((N, K), -128, dtype=torch.int8)
    wq[1] = 127
    aq = torch.full((M, K), -128, dtype=torch.int8)
    w = (wq, torch.full((N,), 2.0 ** -20))
    check(r9k, aq, torch.ones(M), w, r9k.pack_weight_i8(wq.cuda()), "largest")


def test_packed_copy_holds_the_same_values(r9k):
    """Products with unit rows give the weight's columns, exactly."""
    N, K = 80, 256
    w = weight((N,), K, 3)
    a = torch.eye(K, dtype=torch.int8)
    got = r9k.gemm_i8(a.cuda(), torch.ones(K).cuda(), r9k.pack_weight_i8(w[0].cuda()), torch.ones(N).cuda())
    assert torch.equal(got.cpu().float(), w[0].T.float())


def test_every_row_count_agrees(r9k):
    K, N = 512, 160
    w = weight((N,), K, 9)
    p = r9k.pack_weight_i8(w[0].cuda())
    a = acts(300, K, 4)
    aq, as_ = ref.quant(a)
    want = ref.product32(aq, as_, *w).to(torch.bfloat16)
    for M in (1, 2, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 300):
        say("rows", M)
        c = torch.full((M + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
        r9k.gemm_i8_qa(a[:M].contiguous().cuda(), p, w[1].cuda(), c=c[:M])
        assert torch.equal(c[:M].cpu(), want[:M]), M
        assert torch.all(c[M:] == 7.0), M                         # nothing behind the last row


@pytest.mark.parametrize("M", [7, 33, 150])
def test_a_row_without_a_finite_value_stays_alone(r9k, M):
    K, N = 512, 96
    w = weight((N,), K, 31)
    p, ws, x = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda(), acts(M, K, 4)
    y = x.clone()
    bad = [0, 3, 5, M - 1]
    for r, k, v in zip(bad, (0, 200, K - 1, 77), (float("inf"), float("nan"), -float("inf"), float("inf"))):
        y[r, k] = v
    good = torch.ones(M, dtype=torch.bool)
    good[bad] = False
    fine, got = r9k.gemm_i8_qa(x.cuda(), p, ws).cpu(), r9k.gemm_i8_qa(y.cuda(), p, ws).cpu()
    assert torch.all(torch.isfinite(fine)) and torch.equal(got[good], fine[good])
    assert torch.isnan(got[bad]).all()


def test_streams_workspaces_and_graphs(r9k):
    """A side stream with its own allocations, a caller's workspace with anything in it, and captured graphs
    replayed in turn with other work between them."""
    shapes = [(1, 4096, 1024), (16, 14336, 1024), (48, 2048, 512), (200, 2048, 1024), (600, 1024, 2048)]
    calls = []
    for i, (M, K, N) in enumerate(shapes):
        w = weight((N,), K, i)
        p, ws, a = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda(), acts(M, K, i).cuda()
        c = r9k.gemm_i8_qa(a, p, ws)
        need = r9k.gemm_i8_workspace(M, K, N)
        buf = torch.full((need + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(r9k.gemm_i8_qa(a, p, ws, workspace=buf), c)
        calls.append((a, p, ws, c))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [r9k.gemm_i8_qa(a, p, ws, stream=side) for a, p, ws, _ in calls]
    side.synchronize()
    assert all(torch.equal(o, c) for o, (*_, c) in zip(outs, calls))
    graphs = []
    for a, p, ws, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = r9k.gemm_i8_qa(a, p, ws)
        graphs.append((g, o))
    for _ in range(4):
        for (g, o), (a, p, ws, c) in zip(graphs, calls):
            o.zero_()
            g.replay()
            assert torch.equal(r9k.gemm_i8_qa(a, p, ws), c)
        torch.cuda.synchronize()
        assert all(torch.equal(o, c) for (_, o), (*_, c) in zip(graphs, calls))


def test_refusals(r9k):
    w = weight((32,), 256, 1)
    p, ws = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda()
    a = acts(2, 256, 1).cuda()
    q, s = r9k.quant_i8(a)
    for bad in (lambda: r9k.gemm_i8_qa(a[:, :128].contiguous(), p, ws),                     # another K
                lambda: r9k.gemm_i8_qa(a, p, ws[:16]), lambda: r9k.gemm_i8(q, s[:1], p, ws),
                lambda: r9k.gemm_i8_qa(a.t().contiguous().t(), p, ws),                      # a strided view
                lambda: r9k.gemm_i8_qa(a, p, ws, c=torch.empty((2, 48), dtype=torch.bfloat16, device="cuda")),
                lambda: r9k.gemm_i8_qa(a[0], p, ws), lambda: r9k.gemm_i8_qa(a, p[None], ws),
                lambda: r9k.gemm_i8_qa(a.cpu(), p, ws), lambda: r9k.gemm_i8_qa(a, p.cpu(), ws),
                lambda: r9k.pack_weight_i8(w[0][:24].contiguous().cuda()), lambda: r9k.pack_weight_i8(w[0]),
                lambda: r9k.quant_i8(a.cpu()), lambda: r9k.quant_i8(a, s=s[:1])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: r9k.gemm_i8_qa(a.half(), p, ws), lambda: r9k.gemm_i8_qa(a, p.view(torch.uint8), ws),
                lambda: r9k.gemm_i8_qa(a, p, ws.double()), lambda: r9k.gemm_i8(a, s, p, ws), lambda: r9k.quant_i8(a.float())):
        with pytest.raises(TypeError):
            bad()
    for bad, code in ((lambda: r9k.quant_i8(torch.zeros((2, 96), dtype=torch.bfloat16, device="cuda")), -2),
                      (lambda: r9k.quant_i8(a, q=a.view(torch.int8).view(-1)[:512].view(2, 256)), -7),
                      (lambda: r9k.gemm_i8_qa(acts(100, 256, 1).cuda(), p, ws, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), -6)):
        with pytest.raises(r9k.R9kError) as e:
            bad()
        assert e.value.code == code
    empty = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    assert r9k.gemm_i8_qa(empty, p, ws).shape == (0, 32) and r9k.quant_i8(empty)[1].shape == (0,)


# ------------------------------------------------------ experts' products ----

def routing(T, k, E, kind, seed):
    g = np.random.default_rng(seed)
    if kind == "one":
        return np.full((T, k), E // 2, np.int32)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if kind != "skew" else \
        np.minimum(g.geometric(0.4, (T, k)) - 1, E - 1).astype(np.int32)
    if kind == "drop":
        ids[g.random((T, k)) < 0.4] = -1
    return ids


@pytest.mark.parametrize("T,k,E,K,N,kind", [(1, 1, 1, 128, 32, "rand"), (1, 8, 16, 256, 96, "rand"), (5, 2, 7, 384, 64, "drop"),
                                            (16, 4, 32, 256, 224, "rand"), (40, 2, 3, 256, 160, "rand"),
                                            (90, 3, 6, 128, 64, "skew"), (150, 2, 4, 256, 96, "one"),
                                            (400, 2, 70, 128, 32, "skew"), (700, 2, 3, 256, 288, "drop"),
                                            (1100, 4, 8, 384, 544, "rand"), (30, 2, 300, 128, 64, "rand")])
def test_experts(r9k, T, k, E, K, N, kind):
    say("moe_gemm_i8", T, k, E, K, N, kind)
    ids = routing(T, k, E, kind, T)
    src, pos, off = w4_ref.sort(ids, E)
    n = int(off[E])
    w = weight((E, N), K, T + N)
    p, ws = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda()
    q, s = ref.quant(acts(T, K, T))
    slot = torch.from_numpy(src[:n]).long()
    rq, rs = q[slot // k], s[slot // k]
    val = torch.zeros((n, N))
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            val[lo:hi] = ref.product32(rq[lo:hi], rs[lo:hi], w[0][e], w[1][e])
    offd, srcd = torch.from_numpy(off).cuda(), torch.from_numpy(src).cuda()

    c = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
    r9k.moe_gemm_i8(q.cuda(), s.cuda(), offd, p, ws, src=srcd, topk=k, c=c)
    assert torch.equal(c[:n].cpu(), val.to(torch.bfloat16))
    assert torch.all(c[n:] == 7.0)                                # rows behind the last kept one
    xq, xs = torch.zeros((T * k, K), dtype=torch.int8), torch.zeros(T * k)
    xq[:n], xs[:n] = rq, rs
    c2 = torch.full_like(c, 7.0)
    r9k.moe_gemm_i8(xq.cuda(), xs.cuda(), offd, p, ws, c=c2)      # the sorted copy: the same sums
    assert torch.equal(c2, c)

    h = torch.full((T * k, N // 2), 7.0, dtype=torch.bfloat16, device="cuda")
    r9k.moe_gemm_i8(q.cuda(), s.cuda(), offd, p, ws, src=srcd, topk=k, act="silu_mul", c=h)
    v = val.to(ref.F64)
    none = torch.zeros_like(v[:, :N // 2])                        # gate and up are known to the bit
    wh, bh = w4_ref.silu_mul(v[:, :N // 2], v[:, N // 2:], none, none)
    assert torch.all((h[:n].cpu().to(ref.F64) - wh).abs() <= ref.bf16_bound(wh, bh))
    assert torch.all(h[n:] == 7.0)


def test_bad_offsets_and_indexes_stay_inside(r9k):
    """Device data the host cannot check: offsets beyond the rows are held to them, an index beyond the tokens reads row
    0; the rows of the other experts are right."""
    T, E, K, N = 6, 3, 128, 32
    w = weight((E, N), K, 1)
    p, (q, s) = r9k.pack_weight_i8(w[0].cuda()), ref.quant(acts(T, K, 2))
    off = torch.tensor([-4, 2, 4, 99], dtype=torch.int32).cuda()
    src = torch.tensor([0, 1, 2, 2 ** 31 - 1, -9, 5], dtype=torch.int32).cuda()
    c = torch.full((T + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    r9k.moe_gemm_i8(q.cuda(), s.cuda(), off, p, w[1].cuda(), src=src, c=c[:T])
    r = torch.tensor([0, 1, 2, 0, 0, 5])
    for e, (lo, hi) in enumerate(((0, 2), (2, 4), (4, 6))):
        want = ref.product32(q[r[lo:hi]], s[r[lo:hi]], w[0][e], w[1][e]).to(torch.bfloat16)
        assert torch.equal(c[lo:hi].cpu(), want), e
    assert torch.all(c[T:] == 7.0)


def test_experts_refusals(r9k):
    E, N, K = 2, 32, 128
    w = weight((E, N), K, 1)
    p, ws = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda()
    q, s = r9k.quant_i8(acts(4, K, 1).cuda())
    off = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    src = torch.arange(4, dtype=torch.int32).cuda()
    for bad in (lambda: r9k.moe_gemm_i8(q, s, off[:2], p, ws), lambda: r9k.moe_gemm_i8(q, s[:3], off, p, ws),
                lambda: r9k.moe_gemm_i8(q, s, off, p, ws[:1]), lambda: r9k.moe_gemm_i8(q, s, off, p[0], ws[0]),
                lambda: r9k.moe_gemm_i8(q, s, off, p, ws, act="gelu"), lambda: r9k.moe_gemm_i8(q, s, off, p[:0], ws[:0]),
                lambda: r9k.moe_gemm_i8(q, s, off, p, ws, c=torch.empty((3, N), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: r9k.moe_gemm_i8(q[:1], s[:1], off, p, ws, src=src, topk=3), -2),   # more rows than slots
                      (lambda: r9k.moe_gemm_i8(q, s, off, p, ws, src=src, topk=0), -2)):
        with pytest.raises(r9k.R9kError) as e:
            bad()
        assert e.value.code == code
    assert r9k.moe_gemm_i8(q[:0], s[:0], off, p, ws).shape == (0, N)
