"""silu(gate) * up of the 8-bit experts' products at gates far from zero: exp(-|gate|) leaves fp32's normal numbers below gate =
-87.3, and a large up brings the output back into them."""
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


GATES = [-1.0, -20.0, -79.5, -80.0, -86.0, -87.0, -87.25, -87.3, -87.33, -87.34, -87.5, -88.0, -88.7, -88.8, -90.0, -95.0, -100.0,
         -104.0, -110.0, -120.0, -131.0, -150.0, -170.0, -176.0, -180.0, -190.0, -199.0, -200.0, -201.0, -230.0, -300.0, -301.0,
         -1000.0, -1e10, -3e38, 1e-40, 0.5, 5.0, 20.0, 87.5, 95.0, 200.0, 1e10]
UPS = [1.0, -3.0, 1e10, -1e20, 3e30, 3.3e38, -3.3e38, 1e-10, 1e-30, 1e-38, -1e-42]


def pairs(K=128):
    """A weight whose first column is 1 and all else 0, with the gates and ups as its scales: row r of the product with a row
    whose first code is r and whose scale is 1 / r gives them to the bit for r a power of two."""
    g, u = (torch.tensor(v, dtype=torch.float32) for v in zip(*[(g, u) for g in GATES for u in UPS]))
    n = (len(g) + 15) // 16 * 16
    g, u = (torch.cat((v, torch.ones(n - len(v)))) for v in (g, u))
    w = torch.zeros((1, 2 * n, K), dtype=torch.int8)
    w[:, :, 0] = 1
    return g, u, w, torch.cat((g, u))[None]


@pytest.mark.parametrize("shape", [None] + [("stream", *s) for s in STREAM if s[0] > 1] + [("tiled", *t) for t in TILES])
@pytest.mark.parametrize("M", [1, 40, 300])
def test_far_gates(r9k, M, shape):
    """The bound: exp, its correction, the sum, its reciprocal and the products lose at most 8 * 2^-24 of the value, a
    product that leaves the normal numbers half of fp32's smallest step before it is multiplied by at most |gate| < 2^9 (from
    gate = -300 on the output is 0 whatever up), and bf16 its own rounding."""
    K = 128
    g, u, w, ws = pairs(K)
    q = torch.zeros((M, K), dtype=torch.int8)
    q[:, 0] = torch.pow(2, torch.arange(M) % 7).to(torch.int8)
    s = 1.0 / q[:, 0].float()
    if shape:
        kernel, a, b, *more = shape
        r9k.set_i8_plan(r9k.I8_STREAM, a, b, more[0], 0, more[1]) if kernel == "stream" else r9k.set_i8_plan(r9k.I8_TILED, a, b)
    say("silu", M, shape)
    try:
        off = torch.tensor([0, M], dtype=torch.int32).cuda()
        got = r9k.moe_gemm_i8(q.cuda(), s.cuda(), off, r9k.pack_weight_i8(w.cuda()), ws.cuda(), act="silu_mul").cpu()
    finally:
        r9k.set_i8_plan()
    none = torch.zeros(len(g), dtype=ref.F64)
    want, bound = w4_ref.silu_mul(g.to(ref.F64), u.to(ref.F64), none, none)
    bound = ref.bf16_bound(want, bound + 2.0 ** -150 * 2.0 ** 9)
    large = want.abs() > 3.39e38                                   # past bf16's largest value
    err = (got.to(ref.F64) - want).abs()
    bad = (err > bound) & ~large
    assert not bad.any(), [(float(g[j]), float(u[j]), float(want[j]), float(got[i, j])) for i, j in bad.nonzero().tolist()[:4]]
    assert torch.all(torch.isinf(got[:, large])) and torch.equal(got, got[:1].expand_as(got))


@pytest.mark.parametrize("M", [3, 200])
def test_what_is_not_finite_stays_so(r9k, M):
    """A NaN gate or up gives NaN beside far gates that are right, an infinite up an infinity."""
    g, u, w, ws = pairs()
    at = [i * len(UPS) + UPS.index(3.3e38) for i in range(len(GATES))]
    ws[0, at[0]], ws[0, len(g) + at[1]], ws[0, len(g) + at[9]] = float("nan"), float("nan"), float("inf")
    q = torch.zeros((M, 128), dtype=torch.int8)
    q[:, 0] = 1
    off = torch.tensor([0, M], dtype=torch.int32).cuda()
    p = r9k.pack_weight_i8(w.cuda())
    fine = r9k.moe_gemm_i8(q.cuda(), torch.ones(M).cuda(), off, p, torch.cat((g, u))[None].cuda(), act="silu_mul").cpu()
    got = r9k.moe_gemm_i8(q.cuda(), torch.ones(M).cuda(), off, p, ws.cuda(), act="silu_mul").cpu()
    assert torch.isnan(got[:, at[0]]).all() and torch.isnan(got[:, at[1]]).all()
    assert torch.all(got[:, at[9]] == -float("inf"))
    rest = torch.ones(len(g), dtype=torch.bool)
    rest[[at[0], at[1], at[9]]] = False
    assert torch.equal(got[:, rest], fine[:, rest])
