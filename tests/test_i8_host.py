"""The 8-bit integer products and the router's training operators on the host: argument checks and their codes, before any
device is touched; workspace queries; loads into LDS."""
import ctypes
import os
from ctypes import c_size_t, c_void_p

import numpy as np
import pytest
import torch

from tests import i8_ref as ref
from tests.test_abi import A16, B16, C16, NUL, ODD, S, _gpu_present

D16, E16, F16, G16 = (c_void_p(i << 40) for i in range(4, 8))   # far from each other: no overlap
NO_DEVICE = 0 if _gpu_present() else -4


@pytest.fixture(scope="module")
def L():
    import block_scaled_fp8_r9k_amd as r9k
    return r9k.lib()


def test_quant_and_pack_checks(L):
    f = L.r9k_quant_i8
    X, Q, P = D16, E16, F16
    assert f(NUL, 1, 128, Q, P, S) == f(X, 1, 128, NUL, P, S) == f(X, 1, 128, Q, NUL, S) == -1
    for rows, K in ((-1, 128), (1 << 31, 128), (1, 0), (1, 100), (1, -128), (1, 1 << 17), (1, (1 << 17) + 128)):
        assert f(X, rows, K, Q, P, S) == -2, (rows, K)
    assert f(ODD, 1, 128, Q, P, S) == f(X, 1, 128, ODD, P, S) == f(X, 1, 128, Q, ODD, S) == -3
    assert f(X, 4, 128, X, P, S) == -7                                          # in place
    assert f(X, 4, 128, c_void_p((4 << 40) + 1008), P, S) == -7                 # the codes begin on the last values
    assert f(X, 4, 128, Q, c_void_p((5 << 40) + 496), S) == -7                  # the scales on the last codes
    assert f(X, 0, 128, Q, P, S) == 0
    g = L.r9k_pack_weight_i8
    assert g(NUL, 16, 128, Q, S) == g(X, 16, 128, NUL, S) == -1
    for N, K in ((0, 128), (8, 128), (24, 128), (16, 64), (16, 1 << 17), (1 << 29, 128), (-16, 128)):
        assert g(X, N, K, Q, S) == -2, (N, K)
    assert g(ODD, 16, 128, Q, S) == g(X, 16, 128, ODD, S) == -3
    assert g(X, 16, 128, X, S) == -7


def _need(L, M, K, N):
    b = c_size_t(7)
    return L.r9k_gemm_i8_workspace(M, K, N, ctypes.byref(b)), b.value


def test_workspace_queries(L):
    assert L.r9k_gemm_i8_workspace(1, 128, 16, None) == -1
    assert _need(L, 0, 128, 16) == (0, 0)
    for M, K, N in ((-1, 128, 16), ((1 << 24) + 1, 128, 16), (1, 64, 16), (1, 1 << 17, 16), (1, 128, 8), (1, 128, (1 << 24) + 16)):
        assert _need(L, M, K, N)[0] == -2
    for M, K, N in ((100, 4096, 4096), (4096, 4096, 12288)):
        rc, b = _need(L, M, K, N)
        assert rc == 0 and b >= M * K + 4 * M and b % 256 == 0
    assert _need(L, 1, 512, 1024) == (0, 0)                                     # quantised inside the product, no split
    b = c_size_t(0)
    q = L.r9k_moe_balance_loss_workspace
    assert q(1, 1, 1, None) == -1
    for T, E, k in ((-1, 8, 2), (1 << 24, 8, 2), (8, 0, 2), (8, 2049, 2), (8, 8, 0), (8, 8, 65)):
        assert q(T, E, k, ctypes.byref(b)) == -2
    assert q((1 << 24) - 1, 2048, 64, ctypes.byref(b)) == 0 and 0 < b.value < 1 << 24
    assert q(64, 8, 2, ctypes.byref(b)) == 0 and b.value == 0                   # one launch


def test_product_checks(L):
    big = 1 << 38
    W = c_void_p(9 << 40)
    f = L.r9k_gemm_i8
    ok = [D16, E16, 4, 256, F16, G16, 32, A16, W, big, S]
    for i in (0, 1, 4, 5, 7):
        bad = list(ok)
        bad[i] = NUL
        assert f(*bad) == -1, i
        bad[i] = ODD
        assert f(*bad) == -3, i
    for i, v in ((2, -1), (2, (1 << 24) + 1), (3, 0), (3, 192), (3, 1 << 17), (6, 0), (6, 8), (6, (1 << 24) + 16)):
        bad = list(ok)
        bad[i] = v
        assert f(*bad) == -2, (i, v)
    for i in (0, 1, 4, 5):                                                      # the output on an input
        bad = list(ok)
        bad[7] = ok[i]
        assert f(*bad) == -7, i
    bad = list(ok)
    bad[2] = 0
    assert f(*bad) == 0
    g = L.r9k_gemm_i8_qa
    ok = [D16, 100, 256, F16, G16, 32, A16, W, big, S]
    for i in (0, 3, 4, 6, 7):
        bad = list(ok)
        bad[i] = NUL
        assert g(*bad) == -1, i
        bad[i] = ODD
        assert g(*bad) == -3, i
    bad = list(ok)
    bad[8] = _need(L, 100, 256, 32)[1] - 1
    assert g(*bad) == -6
    for i in (0, 3, 4, 6):                                                      # the workspace on a tensor
        bad = list(ok)
        bad[7] = ok[i]
        assert g(*bad) == -7, i
    bad = list(ok)
    bad[1] = 0
    assert g(*bad) == 0


def test_experts_checks(L):
    f = L.r9k_moe_gemm_i8
    ok = [D16, E16, 4, F16, 2, G16, 3, 8, 256, c_void_p(9 << 40), c_void_p(10 << 40), 64, 0, A16, S]
    for i in (0, 1, 5, 9, 10, 13):
        bad = list(ok)
        bad[i] = NUL
        assert f(*bad) == -1, i
    for i in (0, 1, 3, 5, 9, 10, 13):
        bad = list(ok)
        bad[i] = ODD
        assert f(*bad) == -3, i
    for i, v in ((2, 0), (2, -1), (4, 0), (4, 1), (6, 0), (6, 2049), (7, -1), (7, 9), (7, 1 << 31), (8, 100), (8, 1 << 17), (11, 8)):
        bad = list(ok)
        bad[i] = v
        assert f(*bad) == -2, (i, v)
    bad = list(ok)
    bad[3], bad[7] = NUL, 5                                                     # without an index, more rows than there are
    assert f(*bad) == -2
    bad = list(ok)
    bad[11], bad[12] = 48, 1                                                    # silu: columns in pairs of tiles
    assert f(*bad) == -2
    bad[11], bad[12] = 64, 2
    assert f(*bad) == -7
    for i in (0, 1, 3, 5, 9, 10):
        bad = list(ok)
        bad[13] = ok[i]
        assert f(*bad) == -7, i
    bad = list(ok)
    bad[7] = 0
    assert f(*bad) == 0


def test_router_checks(L):
    big = 1 << 38
    f = L.r9k_moe_balance_loss
    V = [c_void_p(i << 40) for i in range(1, 9)]
    ok = [V[0], 1, 2000, 16, V[1], 2, V[2], V[3], V[4], V[5], V[6], big, S]
    for i in (0, 4, 7, 8, 9, 10):
        bad = list(ok)
        bad[i] = NUL
        assert f(*bad) == -1, i
    for i in (0, 4, 6, 7, 8, 9, 10):
        bad = list(ok)
        bad[i] = ODD
        assert f(*bad) == -3, i
    for i, v in ((2, -1), (2, 1 << 24), (3, 0), (3, 2049), (5, 0), (5, 65)):
        bad = list(ok)
        bad[i] = v
        assert f(*bad) == -2, (i, v)
    bad = list(ok)
    bad[1] = 2
    assert f(*bad) == -7
    bad = list(ok)
    bad[11] = 16
    assert f(*bad) == -6
    for i in (0, 4, 6, 8, 9, 10):
        bad = list(ok)
        bad[7] = ok[i]
        assert f(*bad) == -7, i
    g = L.r9k_moe_balance_loss_backward
    ok = [V[0], V[1], 0, 20, 16, 2, V[2], V[3], V[4], V[5], V[6], V[7], S]
    for i in (0, 1, 6, 8, 9, 10, 11):                                           # one of the routing's three alone too
        bad = list(ok)
        bad[i] = NUL
        assert g(*bad) == -1, i
    for i in (0, 1, 6, 7, 8, 9, 10, 11):
        bad = list(ok)
        bad[i] = ODD
        assert g(*bad) == -3, i
    for i in (0, 1, 6, 7, 8, 9, 10):
        bad = list(ok)
        bad[11] = ok[i]
        assert g(*bad) == -7, i
    for i, v in ((3, -1), (3, 1 << 24), (4, 0), (4, 2049), (5, 0), (5, 65)):
        bad = list(ok)
        bad[i] = v
        assert g(*bad) == -2, (i, v)
    bad = list(ok)
    bad[3] = 0
    assert g(*bad) == 0
    h = L.r9k_moe_route_backward
    ok = [V[0], V[1], V[2], 20, 16, 2, V[3], S]
    for i in (0, 1, 2, 6):
        bad = list(ok)
        bad[i] = NUL
        assert h(*bad) == -1, i
        bad[i] = ODD
        assert h(*bad) == -3, i
        if i < 3:
            bad = list(ok)
            bad[6] = ok[i]
            assert h(*bad) == -7, i
    for i, v in ((3, -1), (3, 1 << 24), (4, 0), (4, 65537), (5, 0), (5, 65)):
        bad = list(ok)
        bad[i] = v
        assert h(*bad) == -2, (i, v)
    bad = list(ok)
    bad[3] = 0
    assert h(*bad) == 0


@pytest.mark.skipif(_gpu_present(), reason="valid arguments would reach a real device")
def test_no_device_is_reported(L):
    V = [c_void_p(i << 40) for i in range(1, 9)]
    big = 1 << 38
    assert L.r9k_quant_i8(V[0], 1, 128, V[1], V[2], S) == -4
    assert L.r9k_pack_weight_i8(V[0], 16, 128, V[1], S) == -4
    assert L.r9k_gemm_i8(V[0], V[1], 1, 128, V[2], V[3], 16, V[4], V[5], big, S) == -4
    assert L.r9k_gemm_i8_qa(V[0], 1, 128, V[2], V[3], 16, V[4], V[5], big, S) == -4
    assert L.r9k_moe_gemm_i8(V[0], V[1], 4, V[2], 2, V[3], 3, 8, 256, V[4], V[5], 64, 1, V[6], S) == -4
    assert L.r9k_moe_balance_loss(V[0], 1, 0, 16, V[1], 2, NUL, V[3], V[4], V[5], V[6], big, S) == -4
    assert L.r9k_moe_balance_loss_backward(V[0], V[1], 0, 4, 16, 2, V[2], NUL, NUL, NUL, NUL, V[7], S) == -4
    assert L.r9k_moe_route_backward(V[0], V[1], V[2], 4, 16, 2, V[3], S) == -4


def test_binding_refuses_host_tensors():
    import block_scaled_fp8_r9k_amd as r9k
    q, f = torch.zeros((16, 128), dtype=torch.int8), torch.zeros(16)
    for call in (lambda: r9k.quant_i8(q.to(torch.bfloat16)), lambda: r9k.pack_weight_i8(q), lambda: r9k.gemm_i8(q, f, q, f),
                 lambda: r9k.gemm_i8_qa(q.to(torch.bfloat16), q, f),
                 lambda: r9k.moe_gemm_i8(q, f, torch.zeros(2, dtype=torch.int32), q[None], f[None]),
                 lambda: r9k.moe_balance_loss(torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)),
                 lambda: r9k.moe_balance_loss_backward(f[0], torch.zeros((4, 8)), torch.zeros(9, dtype=torch.int32), 2),
                 lambda: r9k.moe_route_backward(torch.zeros((4, 2)), torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)), 8)):
        with pytest.raises(ValueError):
            call()


def test_rounding_by_a_sum_is_rint():
    """x * inv + 1.5 * 2^23 leaves rint(x * inv) in its low byte for every |x * inv| <= 127 (1 + 2^-23): all halves, and the
    fp32 values next to them."""
    v = np.arange(-254, 255, dtype=np.float32) / 2
    v = np.concatenate([v, np.nextafter(v, np.float32(1e9)), np.nextafter(v, np.float32(-1e9)),
                        np.linspace(-127, 127, 100001, dtype=np.float32)])
    low = (v + np.float32(12582912.0)).view(np.uint32) & 0xFF
    assert np.array_equal(low.astype(np.uint8).view(np.int8), np.rint(v).astype(np.int8))


def test_largest_code_is_127():
    """amax * (127 / amax) in fp32 rounds to 127 for every bf16 amax from 1e-10 on, so that no code leaves the range."""
    bits = np.arange(0x2EDB, 0x7F80, dtype=np.uint32)          # 1e-10 lies between 0x2EDB and 0x2EDC
    x = (bits << 16).view(np.float32)
    b = np.maximum(x, np.float32(1e-10))
    assert np.all(np.rint(x * (np.float32(127) / b)) <= 127)
    assert np.all(np.rint(x[1:] * (np.float32(127) / b[1:])) == 127)
    q, s = ref.quant(torch.from_numpy(x[:, None]).to(torch.bfloat16))
    assert q.max() == 127 and np.array_equal(s.numpy(), b / np.float32(127))
