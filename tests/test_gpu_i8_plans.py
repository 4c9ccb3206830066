"""Every launch of the 8-bit products, forced: each instance of the streaming and the tiled kernel, with and without a K
split, on shapes that end inside its tiles.  Integer sums are exact, so every launch gives the same bits."""
import numpy as np
import pytest
import torch

from tests import i8_ref as ref
from tests import w4_ref
from tests.gpu_util import say
from tests.test_gpu_i8 import acts, routing, weight

pytestmark = pytest.mark.gpu
TILES = [(256, 256), (256, 128), (128, 128), (128, 64), (64, 128), (64, 64)]
# column tiles a wave, waves along the columns and along K, row tiles a CTA
STREAM = [(1, 1, 4, 1), (1, 1, 8, 1), (1, 1, 16, 1), (2, 1, 4, 1), (2, 1, 8, 1), (2, 2, 2, 1), (1, 1, 4, 2), (1, 1, 8, 2), (2, 1, 4, 2),
          (2, 1, 8, 2), (2, 2, 2, 2), (2, 1, 4, 4), (2, 1, 8, 4)]


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    yield m
    m.set_i8_plan()


@pytest.fixture(scope="module")
def dense(r9k):
    out = []
    for M, K, N in [(1, 128, 16), (1, 4096, 48), (3, 640, 272), (16, 2048, 144), (18, 1152, 96), (67, 896, 400), (200, 384, 528),
                    (300, 1280, 272)]:
        w = weight((N,), K, M + N)
        a = acts(M, K, M)
        want = ref.product32(*ref.quant(a), *w).to(torch.bfloat16).cuda()
        out.append((M, K, N, a.cuda(), r9k.pack_weight_i8(w[0].cuda()), w[1].cuda(), want))
    return out


def run_dense(r9k, dense, what):
    for M, K, N, a, p, ws, want in dense:
        say(what, M, K, N, r9k.i8_plan(M, K, N))
        c = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
        r9k.gemm_i8_qa(a, p, ws, c=c[:M])
        assert torch.equal(c[:M], want) and torch.all(c[M:] == 7.0), (what, M, K, N)
        q, s = r9k.quant_i8(a)
        assert torch.equal(r9k.gemm_i8(q, s, p, ws), want), (what, M, K, N)


@pytest.mark.parametrize("shape", STREAM)
def test_streaming_dense(r9k, dense, shape):
    nt, wn, wk, mt = shape
    for ks in (1, 2, 5):
        r9k.set_i8_plan(r9k.I8_STREAM, nt, wn, wk, ks, mt)
        run_dense(r9k, dense, f"stream {shape} split {ks}")


@pytest.mark.parametrize("tile", TILES)
def test_tiled_dense(r9k, dense, tile):
    for ks in (1, 2, 3):
        r9k.set_i8_plan(r9k.I8_TILED, *tile, 0, ks)
        run_dense(r9k, dense, f"tiled {tile} split {ks}")


@pytest.fixture(scope="module")
def experts(r9k):
    out = []
    for T, k, E, K, N, kind in [(1, 1, 1, 128, 32, "rand"), (9, 3, 7, 384, 96, "drop"), (60, 2, 3, 256, 544, "rand"),
                                (400, 2, 5, 640, 288, "skew"), (90, 4, 300, 128, 64, "rand"), (33, 2, 2, 4096, 64, "one")]:
        ids = routing(T, k, E, kind, T) if kind != "one" else np.full((T, k), 1, np.int32)
        src, pos, off = w4_ref.sort(ids, E)
        n = int(off[E])
        w = weight((E, N), K, T)
        q, s = ref.quant(acts(T, K, T))
        slot = torch.from_numpy(src[:n]).long()
        val = torch.zeros((n, N))
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            if lo < hi:
                val[lo:hi] = ref.product32(q[slot[lo:hi] // k], s[slot[lo:hi] // k], w[0][e], w[1][e])
        out.append((T, k, E, K, N, n, q.cuda(), s.cuda(), torch.from_numpy(off).cuda(), torch.from_numpy(src).cuda(),
                    r9k.pack_weight_i8(w[0].cuda()), w[1].cuda(), val))
    return out


def run_experts(r9k, experts, what):
    for T, k, E, K, N, n, q, s, off, src, p, ws, val in experts:
        say(what, T, k, E, K, N)
        c = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device="cuda")
        r9k.moe_gemm_i8(q, s, off, p, ws, src=src, topk=k, c=c)
        assert torch.equal(c[:n].cpu(), val.to(torch.bfloat16)) and torch.all(c[n:] == 7.0), (what, T, E)
        h = torch.full((T * k, N // 2), 7.0, dtype=torch.bfloat16, device="cuda")
        r9k.moe_gemm_i8(q, s, off, p, ws, src=src, topk=k, act="silu_mul", c=h)
        v = val.to(ref.F64)
        none = torch.zeros_like(v[:, :N // 2])
        wh, bh = w4_ref.silu_mul(v[:, :N // 2], v[:, N // 2:], none, none)
        assert torch.all((h[:n].cpu().to(ref.F64) - wh).abs() <= ref.bf16_bound(wh, bh)) and torch.all(h[n:] == 7.0)


@pytest.mark.parametrize("shape", STREAM)
def test_streaming_experts(r9k, experts, shape):
    nt, wn, wk, mt = shape
    r9k.set_i8_plan(r9k.I8_STREAM, nt, wn, wk, 0, mt)
    run_experts(r9k, experts, f"stream {shape}")


@pytest.mark.parametrize("tile", TILES)
def test_tiled_experts(r9k, experts, tile):
    r9k.set_i8_plan(r9k.I8_TILED, *tile)
    run_experts(r9k, experts, f"tiled {tile}")


def test_a_product_from_codes_allocates_its_output_alone(r9k):
    r9k.set_i8_plan()
    M, K, N = 2048, 4096, 512
    w = weight((N,), K, 1)
    p, ws = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda()
    q, s = r9k.quant_i8(acts(M, K, 2).cuda())
    want = r9k.gemm_i8(q, s, p, ws)
    split = r9k.gemm_i8_workspace(M, K, N, quant=False)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    c = r9k.gemm_i8(q, s, p, ws)
    assert torch.cuda.max_memory_allocated() - before <= c.numel() * 2 + split + 1024 < M * K + split
    assert torch.equal(c, want)
