"""The 8-bit experts' products where a CTA of the tiled kernel computes tile after tile: with silu(gate) * up, whose instances
store other numbers of rows, with experts on both sides of 256, where the search for a tile's rows changes, and with rows that
are not finite."""
import numpy as np
import pytest
import torch

from tests import i8_ref as ref
from tests import w4_ref
from tests.gpu_util import say
from tests.test_gpu_i8_plans import STREAM, TILES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    yield m
    m.set_i8_plan()


def data(rows, E, N, K, seed):
    """Codes, scales and weights on the GPU; scales so that gates lie around zero and a few far from it."""
    g = torch.Generator("cuda").manual_seed(seed)
    q = torch.randint(-127, 128, (rows, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device="cuda", generator=g)
    s, ws = torch.rand(rows, device="cuda", generator=g), torch.rand((E, N), device="cuda", generator=g)
    return q, s * 2.0 ** -5, w, ws * 2.0 ** -9


def fp32(q, s, w, ws):
    """The product's fp32 value, to the bit: with K * 127^2 < 2^24 any order of the sum gives the integers."""
    assert q.shape[1] * 127 * 127 < 1 << 24
    return (q.float() @ w.float().T) * s[:, None] * ws


def experts(q, s, w, ws, off):
    return torch.cat([fp32(q[a:b], s[a:b], w[e], ws[e]) for e, (a, b) in enumerate(zip(off, off[1:]))])


def same(got, val, act, n, what):
    """The n rows of val, bit for bit, or with silu within its bound; nothing written behind them."""
    assert torch.all(got[n:] == 7.0), what
    if act == "none":
        assert torch.equal(got[:n], val.to(torch.bfloat16)), what
        return
    v = val.to(ref.F64)
    I = v.shape[1] // 2
    none = torch.zeros((), dtype=ref.F64, device=v.device)
    want, before = w4_ref.silu_mul(v[:, :I], v[:, I:], none, none)
    assert torch.all((got[:n].to(ref.F64) - want).abs() <= ref.bf16_bound(want, before)), what


@pytest.mark.parametrize("K", [128, 384, 1024])
def test_many_tiles_a_cta_with_silu(r9k, K):
    """More tiles than CTAs in every shape; chunks in odd numbers, and fewer of them than the ring has stages."""
    M, N, off = 4500, 4128, [0, 700, 700, 2600, 4444]
    q, s, w, ws = data(M, 4, N, K, K)
    p, offd = r9k.pack_weight_i8(w), torch.tensor(off, dtype=torch.int32, device="cuda")
    val = experts(q, s, w, ws, off)
    order = torch.randperm(M, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    back = torch.argsort(order)                                             # row r is row back[r] of the copy
    qr, sr, src = q[order].contiguous(), s[order].contiguous(), (3 * back + 2).int()
    try:
        for tile in TILES:
            say("silu tiles", tile, K)
            r9k.set_i8_plan(r9k.I8_TILED, *tile)
            for x, y, i, k in ((q, s, None, 1), (qr, sr, src, 3)):
                c = torch.full((M, N // 2), 7.0, dtype=torch.bfloat16, device="cuda")
                r9k.moe_gemm_i8(x, y, offd, p, ws, src=i, topk=k, act="silu_mul", c=c)
                same(c, val, "silu_mul", off[-1], (tile, k))
    finally:
        r9k.set_i8_plan()


@pytest.mark.parametrize("E", [255, 256, 257, 300, 700])
def test_many_experts_and_tiles(r9k, E):
    """A third of the experts without rows, ten of several blocks, the first and the last among them; tiled and streaming."""
    K, N = 256, 1056
    g = np.random.default_rng(E)
    sizes = np.where(g.random(E) < 0.33, 0, g.integers(1, 40, E))
    sizes[g.choice(E, 10, replace=False)] = g.integers(250, 700, 10)
    sizes[[0, E - 1]] = 300, 70
    off = np.concatenate(([0], np.cumsum(sizes))).tolist()
    n, M = off[-1], off[-1] + 33
    q, s, w, ws = data(M, E, N, K, E)
    p, offd = r9k.pack_weight_i8(w), torch.tensor(off, dtype=torch.int32, device="cuda")
    val = experts(q, s, w, ws, off)
    src = torch.arange(M, dtype=torch.int32, device="cuda") * 2 + 1
    try:
        for shape in [None] + TILES + STREAM:
            if shape and len(shape) == 2:
                r9k.set_i8_plan(r9k.I8_TILED, *shape)
            elif shape:
                r9k.set_i8_plan(r9k.I8_STREAM, *shape[:3], 0, shape[3])
            for act in ("none", "silu_mul"):
                say("experts", E, M, shape, act)
                for i in (None, src):
                    c = torch.full((M, N if act == "none" else N // 2), 7.0, dtype=torch.bfloat16, device="cuda")
                    r9k.moe_gemm_i8(q, s, offd, p, ws, src=i, topk=1 if i is None else 2, act=act, c=c)
                    same(c, val, act, n, (shape, act, i is None))
    finally:
        r9k.set_i8_plan()


@pytest.mark.parametrize("sizes", [(3, 0, 9, 1), (300, 64, 0, 700)])
def test_a_row_without_a_finite_value_stays_alone_among_experts(r9k, sizes):
    K, N = 384, 160
    off = [0] + np.cumsum(sizes).tolist()
    M = off[-1]
    q, s, w, ws = data(M, len(sizes), N, K, M)
    x = torch.randn((M, K), device="cuda", generator=torch.Generator("cuda").manual_seed(M)).to(torch.bfloat16)
    bad = sorted({0, 2, M // 2, M - 1})
    for r, v in zip(bad, (float("nan"), float("inf"), -float("inf"), float("nan"))):
        x[r, 5 * r % K] = v
    q, s = r9k.quant_i8(x)
    good = torch.ones(M, dtype=torch.bool, device="cuda")
    good[bad] = False
    val, s0 = experts(q, torch.where(good, s, torch.ones_like(s)), w, ws, off), s[good]
    assert torch.isnan(s[~good]).all() and torch.isfinite(s0).all()
    p, offd = r9k.pack_weight_i8(w), torch.tensor(off, dtype=torch.int32, device="cuda")
    src = torch.arange(M, dtype=torch.int32, device="cuda")
    try:
        for shape in [None] + TILES + STREAM:
            if shape and len(shape) == 2:
                r9k.set_i8_plan(r9k.I8_TILED, *shape)
            elif shape:
                r9k.set_i8_plan(r9k.I8_STREAM, *shape[:3], 0, shape[3])
            for act in ("none", "silu_mul"):
                say("bad rows", sizes, shape, act)
                for i in (None, src):
                    c = r9k.moe_gemm_i8(q, s, offd, p, ws, src=i, act=act)
                    assert torch.isnan(c[~good]).all(), (shape, act)
                    same(c[good], val[good], act, int(good.sum()), (shape, act))
    finally:
        r9k.set_i8_plan()
