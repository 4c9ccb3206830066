"""4-bit weights at the ends of their formats' ranges: scale bytes, infinities and NaN."""
import numpy as np
import pytest
import torch

from tests import w4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


def _mxfp4(N, K, byte):
    """Row n of the weight holds code n % 16 everywhere, with the scale byte `byte` in every group."""
    code = (torch.arange(N) % 16).to(torch.uint8)
    return (code | code << 4)[:, None].expand(N, K // 2).contiguous(), torch.full((N, K // 32), byte, dtype=torch.uint8)


E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=ref.F64)


@pytest.mark.parametrize("M", [1, 20, 150, 1100])
@pytest.mark.parametrize("byte", [0, 1, 2, 127, 252, 253, 254])
def test_mxfp4_every_code_at_the_ends(r9k, M, byte):
    """One activation a row is not zero, so the product is one value of the weight times a power of two: exact.  From
    2^128 on a value is an infinity, and times the row's zeros NaN."""
    say("mxfp4 byte", byte, M)
    N, K = 32, 256
    wq, s = _mxfp4(N, K, byte)
    p = r9k.pack_weight_w4(wq.cuda(), s.cuda())
    scale = 2.0 ** 100 if byte < 100 else 1.0 if byte < 200 else 2.0 ** -100
    a = torch.zeros((M, K), dtype=torch.bfloat16)
    a[torch.arange(M), (torch.arange(M) * 37) % K] = scale
    got = r9k.gemm_w4(a.cuda(), *p).cpu().to(ref.F64)
    code = torch.arange(N) % 16
    value = E2M1[code % 8] * torch.where(code >= 8, -1.0, 1.0) * 2.0 ** (byte - 127)
    finite = value.abs() < 2.0 ** 128
    assert torch.equal(got[:, finite], (value * scale)[finite].expand(M, -1))
    assert torch.all(torch.isnan(got[:, ~finite]))


@pytest.mark.parametrize("M", [1, 20, 150, 1100])
def test_mxfp4_byte_255_is_nan(r9k, M):
    """The format's NaN scale: its rows of the weight are NaN, the others are to the bit what they are without it."""
    say("mxfp4 byte 255", M)
    N, K = 48, 256
    wq, s = _mxfp4(N, K, 120)
    a = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
    fine = r9k.gemm_w4(a, *r9k.pack_weight_w4(wq.cuda(), s.cuda()))
    s[5, 3] = s[16, 0] = 255
    got = r9k.gemm_w4(a, *r9k.pack_weight_w4(wq.cuda(), s.cuda()))
    keep = torch.ones(N, dtype=torch.bool)
    keep[[5, 16]] = False
    assert torch.all(torch.isnan(got.cpu()[:, ~keep])) and torch.equal(got.cpu()[:, keep], fine.cpu()[:, keep])


def test_quantiser_at_the_widest_ranges(r9k):
    """Groups that reach from one end of bf16 to the other: hi - lo passes fp32's largest value, the scale does not.
    Bit for bit the rule, with the difference taken of the halves (a power of two: exact)."""
    say("quant_weight_w4 wide")
    top = torch.finfo(torch.bfloat16).max
    w = (torch.rand((16, 256), generator=torch.Generator().manual_seed(3)) * 2 - 1)
    w = (w * torch.linspace(0.4, 1, 16)[:, None] * top).to(torch.bfloat16)
    w[0, 0], w[0, 1], w[1] = top, -top, 0
    for group in (32, 64, 128):
        q, s, z = r9k.quant_weight_w4(w.cuda(), group, r9k.W4_INT, True)
        g = w.float().numpy().reshape(16, -1, group)
        f32 = np.float32
        lo, hi = np.minimum(g.min(2), f32(0)), np.maximum(g.max(2), f32(0))
        want_s = torch.from_numpy(np.maximum(hi * f32(0.5) - lo * f32(0.5), f32(0.5e-10)) / f32(15) * f32(2)).to(torch.bfloat16)
        ss = want_s.float().numpy()
        want_z = np.clip(np.rint(-lo / ss), 0, 15)
        want_q = np.clip(np.rint(g / ss[..., None]) + want_z[..., None], 0, 15).reshape(16, -1)
        assert torch.equal(s.cpu(), want_s)
        assert np.array_equal(z.cpu().numpy(), want_z) and np.array_equal(ref.codes_of(q).numpy(), want_q)
        value, _ = ref.dequant(q, s, z, group)
        # half a step of rounding, half of the zero point's, and the codes that the range's ends are clamped to
        # (the scale's own rounding, 2^-8 of 15 steps)
        step = s.cpu().to(ref.F64).repeat_interleave(group, 1)
        assert torch.all((value - w.to(ref.F64)).abs() <= (1 + 15 * 2.0 ** -8) * step)


@pytest.mark.parametrize("fmt,group,zeros", [("int4", 32, False), ("int4", 64, True), ("int4", 128, True), ("mxfp4", 32, False)])
def test_quantiser_keeps_what_is_not_finite(r9k, fmt, group, zeros):
    """A group with an infinity or a NaN has no finite value; every other group is to the bit what it is without it;
    and the product's columns show both."""
    say("quant_weight_w4 non-finite", fmt, group, zeros)
    N, K = 48, 512
    code = r9k.W4_INT if fmt == "int4" else r9k.W4_MXFP4
    w = (torch.randn((N, K), generator=torch.Generator().manual_seed(group)) * 0.02).to(torch.bfloat16)
    bad = w.clone()
    where = [(0, 0, float("nan")), (5, K - 1, float("inf")), (6, 100, -float("inf")), (47, 300, float("nan"))]
    for n, k, v in where:
        bad[n, k] = v
    fine, got = r9k.quant_weight_w4(w.cuda(), group, code, zeros), r9k.quant_weight_w4(bad.cuda(), group, code, zeros)
    groups = torch.zeros((N, K // group), dtype=torch.bool)
    for n, k, _ in where:
        groups[n, k // group] = True
    s = got[1].cpu()
    assert torch.equal(s == 255 if fmt == "mxfp4" else torch.isnan(s), groups)
    assert torch.equal(s[~groups], fine[1].cpu()[~groups])
    each = groups.repeat_interleave(group, 1)
    assert torch.equal(ref.codes_of(got[0])[~each], ref.codes_of(fine[0])[~each])
    if zeros:
        assert torch.equal(got[2].cpu()[~groups], fine[2].cpu()[~groups])
    rows = groups.any(1)
    for M in (3, 90):
        a = torch.randn((M, K), generator=torch.Generator().manual_seed(M)).to(torch.bfloat16).cuda()
        for plan in ((), (r9k.W4_TILED, 1), (r9k.W4_TILED, 4)):
            r9k.set_w4_plan(*plan)
            try:
                c, d = r9k.gemm_w4(a, *r9k.pack_weight_w4(*fine)).cpu(), r9k.gemm_w4(a, *r9k.pack_weight_w4(*got)).cpu()
            finally:
                r9k.set_w4_plan()
            assert torch.all(torch.isnan(d[:, rows])) and torch.equal(d[:, ~rows], c[:, ~rows])
