"""Every launch of the 4-bit products, forced one by one: both kernels, every tile and wave shape, K splits, slices
loaded whole and streamed in one and in several LDS segments, and every count of live row tiles, in every format.  The
planner's own choice covers few of them at sizes that a test can afford; each case asserts that the launch it is
written for is the one that runs."""
import contextlib

import numpy as np
import pytest
import torch

from tests import w4_ref as ref
from tests.gpu_util import say
from tests.test_gpu_w4 import FORMATS, acts, packed, weight
from tests.w4_plans import STREAM_CASES, STREAM_EXPERTS, STREAM_SHAPES, TILED_CASES, TILED_EXPERT_COUNTS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


@contextlib.contextmanager
def forced(r9k, *plan):
    r9k.set_w4_plan(*plan)
    try:
        yield
    finally:
        r9k.set_w4_plan()


def _code(r9k, fmt):
    return r9k.W4_INT if fmt == "int4" else r9k.W4_MXFP4


def dense(r9k, a, p, want, bound, what):
    """The product with guard rows behind it, within its bound, and the same bits again."""
    M, N = want.shape
    c = torch.full((M + 3, N), 7.0, dtype=torch.bfloat16, device="cuda")
    r9k.gemm_w4(a, *p, c=c[:M])
    err = (c[:M].cpu().to(ref.F64) - want).abs()
    assert torch.all(err <= bound), f"{what}: {float((err / bound).max()):.3f} of the bound"
    rms = lambda t: float(t.square().mean().sqrt())   # a wrong term is far off: see tests/test_gpu_w4.py
    assert rms(err) <= 2.0 ** -8 * rms(want) + 1e-30, what
    assert torch.all(c[M:] == 7.0), what
    assert torch.equal(r9k.gemm_w4(a, *p), c[:M]), what


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,K,N,splits", TILED_CASES)
def test_tiled(r9k, fmt, group, zeros, M, K, N, splits):
    w = weight((N,), K, fmt, group, zeros, M + K)
    p, a = packed(r9k, w), acts(M, K, N)
    want, before = ref.product(a, *w, group)
    bound = ref.bf16_bound(want, before)
    for tn in (1, 2, 4):
        for ks in splits:
            say("tiled", fmt, group, zeros, M, K, N, "tiles", tn, "split", ks)
            with forced(r9k, r9k.W4_TILED, tn, 0, 0, ks):
                assert r9k.w4_plan(M, K, N, fmt=_code(r9k, fmt), group=group) == (r9k.W4_TILED, tn, 4, 1, ks, 0)
                dense(r9k, a.cuda(), p, want, bound, f"tiles {tn} split {ks}")


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M,K,N,split", STREAM_CASES)
def test_stream(r9k, fmt, group, zeros, M, K, N, split):
    w = weight((N,), K, fmt, group, zeros, M + K)
    p, a = packed(r9k, w), acts(M, K, N)
    want, before = ref.product(a, *w, group)
    bound = ref.bf16_bound(want, before)
    for shape in STREAM_SHAPES:
        with forced(r9k, r9k.W4_STREAM, *shape, split):
            plan = r9k.w4_plan(M, K, N, fmt=_code(r9k, fmt), group=group)
            say("stream", fmt, group, zeros, M, K, N, plan)
            assert plan[:3] == (r9k.W4_STREAM, *shape[:2]) and plan[4] == split
            dense(r9k, a.cuda(), p, want, bound, f"{plan}")


def experts(r9k, fmt, group, zeros, counts, K, N, topk, plan_of):
    """Expert rows by counts, sorted and through the index, plain and with silu, under the plans of plan_of(silu):
    pairs of the forced plan and what the query has to say."""
    E, R = len(counts), sum(counts)
    off = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    T = -(-(R + 2) // topk)
    R2 = T * topk                                            # with rows behind the last sequence
    g = np.random.default_rng(R + K)
    src = np.full(R2, -1, np.int32)
    src[:R] = g.permutation(R2)[:R]
    w = weight((E, N), K, fmt, group, zeros, R + N)
    p, x = packed(r9k, w), acts(T, K, R)
    rows = x[torch.from_numpy(src[:R]).long() // topk]
    want, before = torch.zeros((R, N), dtype=ref.F64), torch.zeros((R, N), dtype=ref.F64)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            want[lo:hi], before[lo:hi] = ref.product(rows[lo:hi], w[0][e], w[1][e], None if w[2] is None else w[2][e], group)
    I = N // 2
    wh, bh = ref.silu_mul(want[:, :I], want[:, I:], before[:, :I], before[:, I:])
    exact = {"none": (want, ref.bf16_bound(want, before)), "silu_mul": (wh, ref.bf16_bound(wh, bh))}
    xs = torch.zeros((R2, K), dtype=torch.bfloat16)
    xs[:R] = rows
    xd, xsd, srcd, offd = x.cuda(), xs.cuda(), torch.from_numpy(src).cuda(), torch.from_numpy(off).cuda()
    for act, (wa, ba) in exact.items():
        for plan, says in plan_of(act == "silu_mul"):
            with forced(r9k, *plan):
                got = r9k.w4_plan(R2, K, N, E, act, _code(r9k, fmt), group)
                say("experts", fmt, group, zeros, "R", R, K, N, act, got)
                assert says(got), got
                c = torch.full((R2, wa.shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
                r9k.moe_gemm_w4(xd, offd, *p, src=srcd, topk=topk, act=act, c=c)
                err = (c[:R].cpu().to(ref.F64) - wa).abs()
                assert torch.all(err <= ba), f"{act} {got}: {float((err / ba).max()):.3f} of the bound"
                assert torch.all(c[R:] == 7.0)
                c2 = torch.full_like(c, 7.0)
                r9k.moe_gemm_w4(xsd, offd, *p, act=act, c=c2)
                assert torch.equal(c2, c)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("K,N", [(128, 32), (640, 96), (1024, 288)])
def test_tiled_experts(r9k, fmt, group, zeros, K, N):
    """One to four live row tiles, blocks of one expert after another, and experts without rows."""
    experts(r9k, fmt, group, zeros, TILED_EXPERT_COUNTS, K, N, 3,
            lambda silu: [((r9k.W4_TILED, tn), lambda p, tn=tn: p == (r9k.W4_TILED, tn, 4, 1, 1, 0)) for tn in (2, 4)])


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("counts,K,N,topk", STREAM_EXPERTS)
def test_stream_experts(r9k, fmt, group, zeros, counts, K, N, topk):
    experts(r9k, fmt, group, zeros, counts, K, N, topk,
            lambda silu: [((r9k.W4_STREAM, *s), lambda p, s=s: p[:3] == (r9k.W4_STREAM, *s[:2]))
                          for s in STREAM_SHAPES if not silu or s[0] == 2])


@pytest.mark.parametrize("tn", [1, 2, 4])
@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
def test_tiled_wide_scales(r9k, fmt, group, zeros, tn):
    """Scales and rows over many powers of two, a row of zeros among them."""
    say("tiled wide", fmt, group, zeros, tn)
    w = weight((64,), 1024, fmt, group, zeros, 21, wild=True)
    a = acts(33, 1024, 2).float() * torch.exp2(torch.arange(33.0)[:, None] * 2 - 32)
    a[4] = 0
    a = a.to(torch.bfloat16)
    want, before = ref.product(a, *w, group)
    for ks in (1, 3):
        with forced(r9k, r9k.W4_TILED, tn, 0, 0, ks):
            got = r9k.gemm_w4(a.cuda(), *packed(r9k, w)).cpu()
        assert torch.all((got.to(ref.F64) - want).abs() <= ref.bf16_bound(want, before))
        assert torch.all(got[4] == 0)


@pytest.mark.parametrize("fmt,group,zeros", FORMATS)
@pytest.mark.parametrize("M", [7, 33, 150])
def test_tiled_row_without_a_finite_value_stays_alone(r9k, fmt, group, zeros, M):
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
    product = lambda t: r9k.gemm_w4(t.cuda(), *one)
    mixed = [lambda t, act=act: r9k.moe_gemm_w4(t.cuda(), off, *p, act=act) for act in ("none", "silu_mul")]
    for tn, ks, f in [(1, 1, product), (1, 2, product), (2, 2, product), (4, 1, product), (2, 1, mixed[0]), (4, 1, mixed[0]),
                      (2, 1, mixed[1]), (4, 1, mixed[1])]:
        say("tiled non-finite", fmt, group, zeros, M, tn, ks)
        with forced(r9k, r9k.W4_TILED, tn, 0, 0, ks):
            fine, got = f(x).cpu(), f(y).cpu()
        assert torch.all(torch.isfinite(fine)) and torch.equal(got[good], fine[good])
        assert not torch.any(torch.isfinite(got[bad]))


@pytest.mark.parametrize("byte", [0, 1, 252, 254])
def test_tiled_mxfp4_every_code_at_the_ends(r9k, byte):
    from tests.test_gpu_w4_ends import E2M1, _mxfp4
    N, K, M = 32, 256, 70
    wq, s = _mxfp4(N, K, byte)
    p = r9k.pack_weight_w4(wq.cuda(), s.cuda())
    scale = 2.0 ** 100 if byte < 100 else 2.0 ** -100
    a = torch.zeros((M, K), dtype=torch.bfloat16)
    a[torch.arange(M), (torch.arange(M) * 37) % K] = scale
    code = torch.arange(N) % 16
    value = E2M1[code % 8] * torch.where(code >= 8, -1.0, 1.0) * 2.0 ** (byte - 127)
    finite = value.abs() < 2.0 ** 128
    for tn in (1, 2, 4):
        say("tiled mxfp4 byte", byte, tn)
        with forced(r9k, r9k.W4_TILED, tn):
            got = r9k.gemm_w4(a.cuda(), *p).cpu().to(ref.F64)
        assert torch.equal(got[:, finite], (value * scale)[finite].expand(M, -1))
        assert torch.all(torch.isnan(got[:, ~finite]))


@pytest.mark.parametrize("kernel,tiles", [("stream", 0), ("tiled", 2), ("tiled", 4)])
@pytest.mark.parametrize("rows", [70000, 140000])
def test_far_activation_rows(r9k, kernel, tiles, rows):
    """Token rows beyond 2 GiB and beyond 4 GiB, read through the index: the tiled kernel's 32-bit lane offsets, and
    from 2^31 activations on its 64-bit addresses."""
    K, N, E, R = 16384, 64, 2, 150
    say("far rows", kernel, tiles, rows)
    x = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    g = np.random.default_rng(rows)
    pick = np.sort(np.append(g.integers(0, rows, R - 2), [0, rows - 1])).astype(np.int32)
    pickd = torch.from_numpy(pick).long().cuda()
    x[pickd] = acts(R, K, R).cuda()                           # (a row picked twice holds one of its two)
    a = x[pickd].cpu()
    off = torch.tensor([0, R // 3, R], dtype=torch.int32)
    for fmt, group, zeros in (("int4", 64, True), ("mxfp4", 32, False)):
        w = weight((E, N), K, fmt, group, zeros, 3)
        with forced(r9k, r9k.W4_TILED if kernel == "tiled" else r9k.W4_STREAM, tiles):
            assert r9k.w4_plan(R, K, N, E, fmt=_code(r9k, fmt), group=group)[0] == (2 if kernel == "tiled" else 1)
            c = r9k.moe_gemm_w4(x, off.cuda(), *packed(r9k, w), src=torch.from_numpy(pick).cuda()).cpu().to(ref.F64)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            want, before = ref.product(a[lo:hi], w[0][e], w[1][e], None if w[2] is None else w[2][e], group)
            assert torch.all((c[lo:hi] - want).abs() <= ref.bf16_bound(want, before)), (fmt, e)


def test_forced_plans_in_graphs(r9k):
    """Launches with splits of either kernel, captured in turn with workspaces of their own and replayed with eager
    calls between."""
    M, K, N = 48, 2048, 272
    w = weight((N,), K, "int4", 64, True, 5)
    p, a = packed(r9k, w), acts(M, K, 1).cuda()
    graphs = []
    for plan in ((r9k.W4_TILED, 1, 0, 0, 8), (r9k.W4_STREAM, 1, 1, 4, 2), (r9k.W4_TILED, 4, 0, 0, 3)):
        say("graph", plan)
        with forced(r9k, *plan):
            eager = r9k.gemm_w4(a, *p)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = r9k.gemm_w4(a, *p)
        graphs.append((g, out, eager))
    for _ in range(3):
        for g, out, eager in graphs:
            out.zero_()
            g.replay()
            r9k.gemm_w4(a, *p)
        torch.cuda.synchronize()
        assert all(torch.equal(out, eager) for _, out, eager in graphs)


@pytest.mark.parametrize("kernel,shape,split", [("tiled", (4, 0, 0), 1), ("stream", (1, 4, 2), 1), ("tiled", (2, 0, 0), 2),
                                                ("stream", (1, 1, 4), 2)])
@pytest.mark.parametrize("M,K,N", [(140000, 256, 16400), (140000, 16384, 16)])
def test_far_dense_rows(r9k, kernel, shape, split, M, K, N):
    """Outputs, partial sums or activations past 4 GiB: rows from either end and the middle, the columns' ends."""
    say("far dense", kernel, shape, split, M, K, N)
    w = weight((N,), K, "int4", 128, True, 7)
    p = packed(r9k, w)
    a = torch.randn((M, K), generator=torch.Generator(device="cuda").manual_seed(M + K), device="cuda", dtype=torch.bfloat16)
    with forced(r9k, r9k.W4_TILED if kernel == "tiled" else r9k.W4_STREAM, *shape, split):
        assert r9k.w4_plan(M, K, N)[4] == split
        c = r9k.gemm_w4(a, *p)
    rows = torch.tensor([0, 1, 31, 64, 65535, 65536, 131071, 131072, M - 65, M - 17, M - 1])
    cols = torch.unique(torch.cat((torch.arange(0, 16), torch.arange(N - 16, N))))
    want, before = ref.product(a[rows.cuda()], *(t[cols] for t in w), 128)
    got = c[rows.cuda()][:, cols.cuda()].cpu().to(ref.F64)
    assert torch.all((got - want).abs() <= ref.bf16_bound(want, before))


def test_two_threads_on_two_streams(r9k):
    """Two threads call products of their own shapes, formats and streams at the same time: each result is to the bit
    what it is alone."""
    import threading
    say("two threads")
    jobs = []
    for i, (M, K, N, fmt, group, zeros) in enumerate([(3, 4096, 512, "int4", 64, True), (150, 1024, 1040, "mxfp4", 32, False)]):
        p, a = packed(r9k, weight((N,), K, fmt, group, zeros, i)), acts(M, K, i).cuda()
        jobs.append((a, p, r9k.gemm_w4(a, *p), torch.cuda.Stream()))
    torch.cuda.synchronize()
    wrong = []

    def work(a, p, want, stream):
        outs = [r9k.gemm_w4(a, *p, stream=stream) for _ in range(50)]
        stream.synchronize()
        wrong.extend(1 for c in outs if not torch.equal(c, want))
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not wrong and not any(t.is_alive() for t in threads)
