"""The 8-bit products' planner on the host (plans are made without a device): every plan is one that the kernels have, the
workspace covers it, every launch is somebody's; the plan control's refusals; and the wait states before the tiled kernel's
loads into LDS."""
import ctypes
import math
import os
import random

import pytest

import block_scaled_fp8_r9k_amd as r9k
from tests.test_abi import _gpu_present
from tests.test_i8_host import _need
from tests.test_isa_lds_loads import short_waits
from tests.test_isa_mfma_exec import CSRC, HIPCC, _device_asm

TILES = [(256, 256), (256, 128), (128, 128), (128, 64), (64, 128), (64, 64)]


@pytest.fixture(autouse=True)
def auto_plan():
    r9k.set_i8_plan()
    yield
    r9k.set_i8_plan()


def sizes(rng, lo, hi, step=1):
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(x / step)) * step))


def test_plans_are_launches_and_fit_their_workspace():
    rng, seen = random.Random(3), set()
    for _ in range(6000):
        M, K, N = sizes(rng, 1, 1 << 17), sizes(rng, 128, 130944, 128), sizes(rng, 16, 1 << 17, 16)
        rc, need = _need(r9k.lib(), M, K, N)
        assert rc == 0 and need % 256 == 0
        for quant in (False, True):
            kernel, a, b, c, ks, rows, fused = r9k.i8_plan(M, K, N, quant=quant)
            assert 1 <= ks <= min(K // 128, 8) and (quant or not fused)
            split = ks * M * N * 4 if ks > 1 else 0
            assert need >= split + (M * (K + 4) if quant and not fused else 0), (M, K, N)
            assert not fused or (kernel == r9k.I8_STREAM and M <= 16 and ks == 1)
            if kernel == r9k.I8_TILED:
                assert (a, b) in TILES and c == rows == 0 and M > 16
                assert math.ceil(N / a) * math.ceil(M / b) * ks <= max(600, math.ceil(N / a) * math.ceil(M / b))
            else:
                assert M <= 256 and a in (1, 2) and b == 1 and c in (4, 8, 16) and rows in (1, 2, 4) and (rows == 1) == (M <= 16)
            seen.add((kernel, a, b, c, rows))
        E, act = sizes(rng, 1, 2048), rng.choice(["none", "silu_mul"])
        plan = r9k.i8_plan(sizes(rng, 1, 1 << 20), sizes(rng, 128, 16384, 128), sizes(rng, 32, 1 << 15, 32), E, act)
        assert plan[4] == 1 and plan[6] == 0 and (act == "none" or plan[0] == r9k.I8_TILED or plan[1] == 2)
        seen.add(plan[:4] + plan[5:6])
    assert {p[1:3] for p in seen if p[0] == r9k.I8_TILED} == set(TILES)
    for plan in seen - {p for p in seen if p[0] == r9k.I8_TILED}:
        r9k.set_i8_plan(plan[0], *plan[1:4], 1, plan[4])               # what a plan names can be asked for


def test_a_plan_follows_its_setting():
    auto = r9k.i8_plan(100, 4096, 4096)
    r9k.set_i8_plan(r9k.I8_TILED, 256, 128, 0, 7)
    assert r9k.i8_plan(100, 4096, 4096) == (r9k.I8_TILED, 256, 128, 0, 7, 0, 0)
    assert r9k.gemm_i8_workspace(100, 4096, 4096) >= 7 * 100 * 4096 * 4
    assert r9k.i8_plan(100, 384, 4096)[4] == 3                         # no split without chunks
    assert r9k.i8_plan(100, 4096, 4096, 8)[4] == 1                     # nor of experts
    r9k.set_i8_plan(r9k.I8_STREAM)
    assert r9k.i8_plan(100, 4096, 4096)[0] == r9k.I8_STREAM
    r9k.set_i8_plan(r9k.I8_STREAM, 2, 1, 8, 3, 4)
    assert r9k.i8_plan(100, 4096, 4096) == (r9k.I8_STREAM, 2, 1, 8, 3, 4, 0)
    r9k.set_i8_plan()
    assert r9k.i8_plan(100, 4096, 4096) == auto


def test_queries_and_control_refuse():
    for M, K, N, E, act, quant, code in ((-1, 128, 16, 0, "none", False, -2), ((1 << 24) + 1, 128, 16, 0, "none", False, -2),
                                         (1, 100, 16, 0, "none", False, -2), (1, 128, 24, 0, "none", False, -2),
                                         (1, 128, 48, 4, "silu_mul", False, -2), (1, 128, 32, 0, "silu_mul", False, -7),
                                         (1, 128, 32, 4, "none", True, -7), (1, 128, 16, 2049, "none", False, -2)):
        with pytest.raises(r9k.R9kError) as e:
            r9k.i8_plan(M, K, N, E, act, quant)
        assert e.value.code == code, (M, K, N, E, act, quant)
    assert r9k.i8_plan(0, 128, 16) == (0,) * 7
    for bad in ((3,), (-1,), (r9k.I8_AUTO, 1), (r9k.I8_AUTO, 0, 0, 0, 2), (r9k.I8_STREAM, 1, 1, 4, 0, 3), (r9k.I8_STREAM, 0, 0, 0, 2),
                (r9k.I8_STREAM, 1, 1, 4), (r9k.I8_TILED, 32, 64), (r9k.I8_TILED, 128, 64, 1), (r9k.I8_TILED, 128, 128, 0, -1)):
        with pytest.raises(r9k.R9kError) as e:
            r9k.set_i8_plan(*bad)
        assert e.value.code == -7, bad


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")
def test_tiled_loads_wait_for_their_address(tmp_path):
    with open(_device_asm(os.path.join(CSRC, "gemm_i8_tiled.hip"), str(tmp_path))) as f:
        loads, bad = short_waits(f.read())
    assert loads > 100 and not bad, bad[:3]


def test_codes_need_no_room_for_codes():
    """The workspace of a product from codes holds a split's sums alone, and what the query says is what the call takes."""
    assert r9k.gemm_i8_workspace(4096, 4096, 12288, quant=False) == 0
    assert r9k.gemm_i8_workspace(4096, 4096, 12288) >= 4096 * (4096 + 4)
    rng = random.Random(5)
    P = [ctypes.c_void_p(i << 40) for i in range(1, 7)]
    for n in range(600):
        if n % 3 == 0:
            r9k.set_i8_plan(r9k.I8_TILED, *rng.choice(TILES), 0, rng.randint(0, 5))
        M, K, N = sizes(rng, 1, 1 << 14), sizes(rng, 128, 130944, 128), sizes(rng, 16, 1 << 15, 16)
        need, ks = r9k.gemm_i8_workspace(M, K, N, quant=False), r9k.i8_plan(M, K, N)[4]
        assert need == (0 if ks == 1 else (ks * M * N * 4 + 255) // 256 * 256), (M, K, N, ks)
        assert need <= r9k.gemm_i8_workspace(M, K, N)
        call = lambda room: r9k.lib().r9k_gemm_i8(P[0], P[1], M, K, P[2], P[3], N, P[4], P[5], room, None)
        if need:
            assert call(need - 1) == -6, (M, K, N)
        if not _gpu_present():
            assert call(need) == -4, (M, K, N)
    f = r9k.lib().r9k_gemm_i8_codes_workspace
    b = ctypes.c_size_t(7)
    assert f(1, 128, 16, None) == -1 and f(1, 100, 16, ctypes.byref(b)) == -2 and f(0, 128, 16, ctypes.byref(b)) == 0 == b.value
