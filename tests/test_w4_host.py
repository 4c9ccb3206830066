"""The 4-bit weight and row-sorting calls on the host: every check of arguments, before any device is touched."""
import ctypes
from ctypes import c_size_t, c_void_p

import pytest

from tests.test_abi import _gpu_present

A, B, C, D, E16 = (c_void_p(0x100000000 * i) for i in range(1, 6))  # aligned, far apart, never dereferenced
ODD, NUL, S = c_void_p(0x100000008), c_void_p(None), c_void_p(None)
INT, MX = 0, 1


@pytest.fixture(scope="module")
def L():
    import block_scaled_fp8_r9k_amd as r9k
    return r9k.lib()


def test_constants():
    import block_scaled_fp8_r9k_amd as r9k
    from tests.test_abi import _defines
    d = _defines()
    assert (r9k.W4_INT, r9k.W4_MXFP4) == (d["R9K_W4_INT"], d["R9K_W4_MXFP4"]) == (INT, MX)
    assert (r9k.ACT_NONE, r9k.ACT_SILU_MUL) == (d["R9K_ACT_NONE"], d["R9K_ACT_SILU_MUL"])
    assert sorted(r9k._ROWS.values()) == [d["R9K_BF16"], d["R9K_F32"]]


def test_quant_checks(L):
    f = L.r9k_quant_weight_w4
    ok = [A, 16, 128, INT, 128, B, C, NUL, S]

    def with_(i, v):
        x = list(ok)
        x[i] = v
        return f(*x)
    for i in (0, 5, 6):
        assert with_(i, NUL) == -1
    for N in (0, -16, 8, 100):
        assert with_(1, N) == -2
    for K in (0, 64, 130, -128):
        assert with_(2, K) == -2
    assert with_(3, 2) == -7 and with_(3, -1) == -7
    for g in (0, 16, 48, 256):
        assert with_(4, g) == -7
    assert f(A, 16, 128, MX, 128, B, C, NUL, S) == -7        # mxfp4 has one group size
    assert f(A, 16, 128, MX, 32, B, C, D, S) == -7           # and no zeros
    for i in (0, 5, 6, 7):
        assert with_(i, ODD) == -3


def test_pack_checks(L):
    f = L.r9k_pack_weight_w4
    ok = [A, B, NUL, 16, 128, INT, 128, C, D, NUL, S]

    def with_(**kw):
        x = list(ok)
        for k, v in kw.items():
            x[int(k[1:])] = v
        return f(*x)
    for i in (0, 1, 7, 8):
        assert with_(**{f"_{i}": NUL}) == -1
    assert with_(_3=24) == -2 and with_(_4=64) == -2
    assert with_(_5=3) == -7 and with_(_6=96) == -7 and with_(_5=MX) == -7
    assert with_(_2=E16) == -7 and with_(_9=E16) == -7       # zeros in without out, and out without in
    assert with_(_7=A) == -7 and with_(_8=B) == -7           # in place
    for i in (0, 1, 7, 8):
        assert with_(**{f"_{i}": ODD}) == -3


def _ws(fn, *shape):
    b = c_size_t(1 << 40)
    return fn(*shape, ctypes.byref(b)), b.value


def test_gemm_checks(L):
    f = L.r9k_gemm_w4
    big = 1 << 40
    ok = [A, 3, 256, B, C, NUL, INT, 64, 48, D, E16, big, S]

    def with_(**kw):
        x = list(ok)
        for k, v in kw.items():
            x[int(k[1:])] = v
        return f(*x)
    for i in (0, 3, 4, 9):
        assert with_(**{f"_{i}": NUL}) == -1
    assert with_(_1=-1) == -2 and with_(_1=1 << 25) == -2
    assert with_(_2=64) == -2 and with_(_2=0) == -2 and with_(_8=8) == -2 and with_(_8=0) == -2
    assert with_(_6=5) == -7 and with_(_7=100) == -7 and with_(_6=MX) == -7
    assert with_(_6=MX, _7=32, _5=E16) == -7
    for i in (0, 3, 4, 5, 9, 10):
        assert with_(**{f"_{i}": ODD}) == -3
    assert with_(_1=0) == 0
    assert L.r9k_gemm_w4_workspace(1, 128, 16, None) == -1
    assert _ws(L.r9k_gemm_w4_workspace, -1, 128, 16)[0] == -2
    assert _ws(L.r9k_gemm_w4_workspace, 1, 100, 16)[0] == -2
    assert _ws(L.r9k_gemm_w4_workspace, 1, 128, 20)[0] == -2
    assert _ws(L.r9k_gemm_w4_workspace, 0, 128, 16) == (0, 0)
    for M in (1, 5, 64, 300, 4096):       # a workspace smaller than the query's is refused, and NULL where one is needed
        rc, need = _ws(L.r9k_gemm_w4_workspace, M, 4096, 4096)
        assert rc == 0 and need % 256 == 0
        if need:
            x = dict(_1=M, _2=4096, _8=4096)
            assert with_(_11=need - 1, **x) == -6 and with_(_10=NUL, **x) == -1


def test_moe_gemm_checks(L):
    f = L.r9k_moe_gemm_w4
    ok = [A, 8, B, 2, C, 4, 16, 256, D, E16, NUL, INT, 128, 64, 1, c_void_p(6 << 32), S]

    def with_(**kw):
        x = list(ok)
        for k, v in kw.items():
            x[int(k[1:])] = v
        return f(*x)
    for i in (0, 4, 8, 9, 15):
        assert with_(**{f"_{i}": NUL}) == -1
    assert with_(_1=0) == -2 and with_(_1=-1) == -2
    assert with_(_2=NUL) == -2                               # 16 rows from 8 without an index
    assert with_(_3=0) == -2
    assert with_(_5=0) == -2 and with_(_5=2049) == -2
    assert with_(_6=-1) == -2
    assert with_(_7=100) == -2 and with_(_13=16) == -2       # silu needs whole tiles in either half
    assert with_(_13=24, _14=0) == -2
    assert with_(_11=2) == -7 and with_(_12=16) == -7 and with_(_14=2) == -7
    for i in (0, 2, 4, 8, 9, 10, 15):
        assert with_(**{f"_{i}": ODD}) == -3
    assert with_(_6=0) == 0


def test_permute_checks(L):
    f = L.r9k_moe_permute
    F = c_void_p(6 << 32)
    G = c_void_p(7 << 32)
    ok = [A, 0, 4096, 64, B, 2, 8, C, D, E16, F, G, 1 << 30, S]  # slots enough to need a workspace

    def with_(**kw):
        x = list(ok)
        for k, v in kw.items():
            x[int(k[1:])] = v
        return f(*x)
    for i in (0, 4, 7, 8, 9, 10, 11):
        assert with_(**{f"_{i}": NUL}) == -1
    assert with_(_1=2) == -7
    assert with_(_2=-1) == -2 and with_(_2=1 << 25) == -2
    assert with_(_3=0) == -2 and with_(_3=4) == -2 and with_(_3=63) == -2
    assert with_(_3=2, _1=1) == -2                           # 8 bytes of fp32
    assert with_(_5=0) == -2 and with_(_5=65) == -2
    assert with_(_6=0) == -2 and with_(_6=2049) == -2
    assert with_(_7=A) == -7                                 # rows on top of their source
    assert with_(_12=0) == -6
    for i in (0, 4, 7, 8, 9, 10, 11):
        assert with_(**{f"_{i}": ODD}) == -3
    assert L.r9k_moe_permute_workspace(4, 8, 2, None) == -1
    assert _ws(L.r9k_moe_permute_workspace, 4, 0, 2)[0] == -2
    assert _ws(L.r9k_moe_permute_workspace, 4, 8, 0)[0] == -2
    assert _ws(L.r9k_moe_permute_workspace, -4, 8, 2)[0] == -2
    rc, need = _ws(L.r9k_moe_permute_workspace, 4, 8, 2)
    assert rc == 0 and need % 256 == 0


def test_unpermute_checks(L):
    for f, ok, ptrs, out in (
            (L.r9k_moe_unpermute, [A, 0, 4, 64, B, C, 2, D, S], (0, 4, 7), 7),
            (L.r9k_moe_permute_backward, [A, 0, 4, 64, B, 2, D, S], (0, 4, 6), 6)):
        def with_(i, v):
            x = list(ok)
            x[i] = v
            return f(*x)
        for i in ptrs:
            assert with_(i, NUL) == -1 and with_(i, ODD) == -3
        assert with_(1, 3) == -7 and with_(out, A) == -7
        assert with_(2, -1) == -2 and with_(3, 20) == -2 and with_(3, 0) == -2
        assert with_(2, 0) == 0
    f = L.r9k_moe_unpermute_backward
    ok = [A, B, 1, 4, 64, C, D, 2, E16, c_void_p(6 << 32), S]

    def with_(i, v):
        x = list(ok)
        x[i] = v
        return f(*x)
    for i in (0, 1, 5, 6, 8, 9):
        assert with_(i, NUL) == -1 and with_(i, ODD) == -3
    assert with_(8, A) == -7 and with_(8, B) == -7
    assert with_(2, 2) == -7 and with_(3, -1) == -2 and with_(4, 2) == -2 and with_(7, 0) == -2
    assert with_(3, 0) == 0


def test_outputs_on_top_of_inputs(L):
    """An output that lies on what other threads of the call still read is refused, whole or by its last bytes."""
    F, G, H = (c_void_p(i << 32) for i in (6, 7, 8))

    def at(p, off):
        return c_void_p(p.value + off)
    # c [3, 48] against a [3, 256]
    for c in (A, at(A, 2 * 3 * 256 - 16), at(A, -2 * 3 * 48 + 16)):
        assert L.r9k_gemm_w4(A, 3, 256, B, C, NUL, INT, 64, 48, c, E16, 1 << 40, S) == -7
        assert L.r9k_gemm_w4(A, 0, 256, B, C, NUL, INT, 64, 48, c, E16, 1 << 40, S) == 0
    # c [16, 64 or 32] against a [8, 256]
    for act, width in ((0, 64), (1, 32)):
        for c in (A, at(A, 2 * 8 * 256 - 16), at(A, -2 * 16 * width + 16)):
            assert L.r9k_moe_gemm_w4(A, 8, B, 2, C, 4, 16, 256, D, E16, NUL, INT, 128, 64, act, c, S) == -7
    # src, pos [4, 2] and offsets [9] against the ids [4, 2]
    for i in (8, 9, 10):
        for p in (B, at(B, 16)):
            x = [A, 0, 4, 64, B, 2, 8, C, D, E16, F, G, 1 << 30, S]
            x[i] = p
            assert L.r9k_moe_permute(*x) == -7
    # gw [4, 2] against gout, y, w
    for p in (A, B, D, at(B, 4 * 2 * 64 * 4 - 16), at(D, 16)):
        assert L.r9k_moe_unpermute_backward(A, B, 1, 4, 64, C, D, 2, H, p, S) == -7


def test_sizes_past_a_launch(L):
    """Sizes whose launch would hold 2^32 threads are refused before anything is launched, and the workspace queries
    refuse what their calls refuse."""
    T = 1 << 24
    F, G = c_void_p(6 << 40), c_void_p(7 << 40)
    far = c_void_p(1 << 46)
    assert L.r9k_quant_weight_w4(A, 1 << 20, 1 << 15, INT, 128, B, C, D, S) == -2
    assert L.r9k_pack_weight_w4(A, B, NUL, 1 << 22, 1 << 15, INT, 128, far, F, NUL, S) == -2
    assert _ws(L.r9k_moe_permute_workspace, T, 8, 1)[0] == -2 and _ws(L.r9k_moe_permute_workspace, T - 1, 8, 1)[0] == 0
    assert L.r9k_moe_permute(A, 0, T, 64, B, 1, 8, far, D, E16, F, G, 1 << 40, S) == -2
    assert L.r9k_moe_unpermute(A, 0, T, 64, B, C, 1, far, S) == -2
    assert L.r9k_moe_permute_backward(A, 0, T, 64, B, 1, far, S) == -2
    assert L.r9k_moe_unpermute_backward(A, F, 0, T, 64, B, C, 1, far, G, S) == -2
    assert _ws(L.r9k_gemm_w4_workspace, 1, 128, (1 << 24) + 16)[0] == -2
    assert L.r9k_gemm_w4(A, 1, 128, B, C, NUL, INT, 128, (1 << 24) + 16, D, E16, 1 << 40, S) == -2


@pytest.mark.skipif(_gpu_present(), reason="valid arguments would reach a real device")
def test_no_device_is_reported(L):
    big, F, G = 1 << 40, c_void_p(6 << 32), c_void_p(7 << 32)
    assert L.r9k_quant_weight_w4(A, 16, 128, INT, 32, B, C, D, S) == -4
    assert L.r9k_pack_weight_w4(A, B, NUL, 16, 128, MX, 32, C, D, NUL, S) == -4
    assert L.r9k_gemm_w4(A, 1, 128, B, C, NUL, INT, 128, 16, D, E16, big, S) == -4
    assert L.r9k_moe_gemm_w4(A, 8, B, 2, C, 4, 16, 256, D, E16, NUL, INT, 128, 64, 1, F, S) == -4
    assert L.r9k_moe_permute(A, 0, 4, 64, B, 2, 8, C, D, E16, F, G, big, S) == -4
    assert L.r9k_moe_unpermute(A, 0, 4, 64, B, C, 2, D, S) == -4
    assert L.r9k_moe_permute_backward(A, 0, 4, 64, B, 2, D, S) == -4
    assert L.r9k_moe_unpermute_backward(A, B, 1, 4, 64, C, D, 2, E16, F, S) == -4


def test_binding_refuses_host_tensors():
    import torch
    import block_scaled_fp8_r9k_amd as r9k
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    with pytest.raises(ValueError):
        r9k.quant_weight_w4(torch.zeros((16, 128), dtype=bf))
    with pytest.raises(ValueError):
        r9k.pack_weight_w4(torch.zeros((16, 64), dtype=u8), torch.zeros((16, 1), dtype=bf))
    with pytest.raises(ValueError):
        r9k.gemm_w4(torch.zeros((1, 128), dtype=bf), torch.zeros((16, 64), dtype=u8), torch.zeros((16, 1), dtype=bf))
    with pytest.raises(ValueError):
        r9k.moe_permute(None, torch.zeros((2, 2), dtype=i32), 4)
    with pytest.raises(ValueError):
        r9k.moe_unpermute(torch.zeros((4, 64)), torch.zeros((2, 2), dtype=i32))


def test_plans_of_drawn_shapes(L):
    """The workspace query over 3000 drawn shapes: whole fp32 partial outputs, at most eight of them, and the same
    answer again."""
    import random
    rng = random.Random(11)
    for _ in range(3000):
        M = int(2 ** rng.uniform(0, 14))
        K, N = 128 * int(2 ** rng.uniform(0, 9)), 16 * int(2 ** rng.uniform(0, 12))
        rc, need = _ws(L.r9k_gemm_w4_workspace, M, K, N)
        assert rc == 0 and need % 256 == 0
        per = 4 * M * N
        assert any(need == (per * s + 255) // 256 * 256 for s in range(2, 9)) or need == 0, (M, K, N, need)
        assert _ws(L.r9k_gemm_w4_workspace, M, K, N) == (0, need)


@pytest.mark.parametrize("c", [False, True])
@pytest.mark.parametrize("workspace", [False, True])
def test_gemm_refuses_host_tensors_in_every_form(monkeypatch, c, workspace):
    """All operands on the host, with and without the output and the workspace: refused, and no call is made with a
    host address (the library is replaced by one that counts its calls)."""
    import torch
    import block_scaled_fp8_r9k_amd as r9k
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or 0
    monkeypatch.setattr(r9k, "lib", Lib)
    monkeypatch.setattr(r9k, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(r9k, "gemm_w4_workspace", lambda M, K, N: 0)
    bf, u8 = torch.bfloat16, torch.uint8
    a, wp, sp, zp = torch.zeros((1, 128), dtype=bf), torch.zeros((16, 64), dtype=u8), torch.zeros((16, 1), dtype=bf), None
    kw = dict(c=torch.zeros((1, 16), dtype=bf)) if c else {}
    if workspace:
        kw["workspace"] = torch.zeros(256, dtype=u8)
    for zp in (None, torch.zeros((16, 1), dtype=u8)):
        with pytest.raises(ValueError, match="current device"):
            r9k.gemm_w4(a, wp, sp, zp, **kw)
    assert not calls


def test_moe_gemm_refuses_an_index_that_does_not_go_with_the_rows(L):
    """src numbers slots of arows tokens with topk each: more rows than slots cannot be such an index (topk left at 1
    with a top-8 sort would read row 0 for most of them)."""
    F = c_void_p(6 << 32)

    def call(arows, topk, R, src=B, act=1):
        return L.r9k_moe_gemm_w4(A, arows, src, topk, C, 4, R, 256, D, E16, NUL, INT, 128, 64, act, F, S)
    for arows, topk, R in ((8, 1, 16), (8, 2, 17), (16, 8, 129), (1, 1, 2), (8, 1, 1 << 30)):
        assert call(arows, topk, R) == -2 and call(arows, topk, R, act=0) == -2
    if not _gpu_present():  # every slot, or some of them, is an index
        for arows, topk, R in ((8, 2, 16), (8, 2, 9), (16, 8, 128), (1 << 20, 1 << 20, 1 << 20)):
            assert call(arows, topk, R) == -4


def _clashes(f, args, sizes, outs, ins):
    """Places every output of a call on the first and on the last 16 bytes of every input and of every other output
    and yields (what, code).  sizes: bytes by argument index; args: pointers far apart."""
    for o in outs:
        for i in ins + [x for x in outs if x != o]:
            for at in (args[i].value, args[i].value + (sizes[i] - 1) // 16 * 16, args[i].value - (sizes[o] - 1) // 16 * 16):
                x = list(args)
                x[o] = c_void_p(at)
                yield f"argument {o} on argument {i}", f(*x)


def test_every_output_on_every_input_and_output(L):
    """Every call: outputs and workspaces on top of any input or of each other are refused, whole or by their ends."""
    P = [c_void_p(i << 33) for i in range(1, 14)]
    N, K, M, E, R, T, H, k = 64, 256, 40, 3, 24, 512, 64, 6
    wq, s2, z = N * K // 2, N * K // 64 * 2, N * K // 64
    cases = [
        (L.r9k_quant_weight_w4, [P[0], N, K, INT, 64, P[1], P[2], P[3], S], {0: 2 * N * K, 5: wq, 6: s2, 7: z}, [5, 6, 7], [0]),
        (L.r9k_pack_weight_w4, [P[0], P[1], P[2], N, K, INT, 64, P[3], P[4], P[5], S],
         {0: wq, 1: s2, 2: z, 7: wq, 8: s2, 9: z}, [7, 8, 9], [0, 1, 2]),
        (L.r9k_gemm_w4, [P[0], M, K, P[1], P[2], P[3], INT, 64, N, P[4], P[5], 1 << 40, S],
         {0: 2 * M * K, 3: wq, 4: s2, 5: z, 9: 2 * M * N}, [9], [0, 3, 4, 5]),
        (L.r9k_moe_gemm_w4, [P[0], 8, P[1], 3, P[2], E, R, K, P[3], P[4], P[5], INT, 64, N, 1, P[6], S],
         {0: 2 * 8 * K, 2: 4 * R, 4: 4 * (E + 1), 8: E * wq, 9: E * s2, 10: E * z, 15: R * N}, [15], [0, 2, 4, 8, 9, 10]),
        (L.r9k_moe_permute, [P[0], 1, T, H, P[1], k, 8, P[2], P[3], P[4], P[5], P[6], 1 << 40, S],
         {0: 4 * T * H, 4: 4 * T * k, 7: 4 * T * k * H, 8: 4 * T * k, 9: 4 * T * k, 10: 36,
          11: _ws(L.r9k_moe_permute_workspace, T, 8, k)[1]}, [7, 8, 9, 10, 11], [0, 4]),
        (L.r9k_moe_unpermute, [P[0], 0, T, H, P[1], P[2], k, P[3], S],
         {0: 2 * T * k * H, 4: 4 * T * k, 5: 4 * T * k, 7: 2 * T * H}, [7], [0, 4, 5]),
        (L.r9k_moe_permute_backward, [P[0], 0, T, H, P[1], k, P[2], S], {0: 2 * T * k * H, 4: 4 * T * k, 6: 2 * T * H}, [6], [0, 4]),
        (L.r9k_moe_unpermute_backward, [P[0], P[1], 0, T, H, P[2], P[3], k, P[4], P[5], S],
         {0: 2 * T * H, 1: 2 * T * k * H, 5: 4 * T * k, 6: 4 * T * k, 8: 2 * T * k * H, 9: 4 * T * k}, [8, 9], [0, 1, 5, 6]),
    ]
    for f, args, sizes, outs, ins in cases:
        assert sizes.get(11) is None or sizes[11] > 0
        for what, rc in _clashes(f, args, sizes, outs, ins):
            assert rc == -7, (f.__name__, what, rc)
    # a product that splits K: its workspace against everything
    M, K, N = 1, 14336, 1024
    need = _ws(L.r9k_gemm_w4_workspace, M, K, N)[1]
    if need:
        args = [P[0], M, K, P[1], P[2], P[3], INT, 128, N, P[4], P[5], need, S]
        sizes = {0: 2 * M * K, 3: N * K // 2, 4: N * K // 64, 5: N * K // 128, 9: 2 * M * N, 10: need}
        for what, rc in _clashes(L.r9k_gemm_w4, args, sizes, [9, 10], [0, 3, 4, 5]):
            assert rc == -7, (what, rc)


@pytest.mark.skipif(_gpu_present(), reason="valid arguments would reach a real device")
def test_neighbours_do_not_overlap(L):
    """Outputs that end where an input begins, and empty ones anywhere, are fine."""
    N, K, M = 16, 128, 1
    base = 1 << 33
    at = lambda off: c_void_p(base + off)
    # a [1, 128] 256 bytes, wp 1024, sp 32, c 32
    assert L.r9k_gemm_w4(at(0), M, K, at(256), at(1280), NUL, INT, 128, N, at(1312), NUL, 0, S) == -4
    assert L.r9k_gemm_w4(at(32), M, K, at(288), at(1312), NUL, INT, 128, N, at(0), NUL, 0, S) == -4
    assert L.r9k_gemm_w4(at(0), 0, K, at(256), at(1280), NUL, INT, 128, N, at(512), NUL, 0, S) == 0
    assert L.r9k_moe_unpermute(at(0), 0, 0, 64, at(0), at(0), 2, at(0), S) == 0
    assert L.r9k_moe_permute(NUL, 0, 0, 64, at(0), 2, 8, NUL, at(0), at(0), at(0), NUL, 0, S) == -4


@pytest.mark.skipif(_gpu_present(), reason="valid arguments would reach a real device")
def test_planning_does_not_grow_with_the_rows(L):
    """A call's plan costs the same for a few rows and for the most (it was a step for every block of rows: half a
    second at 2^31 - 1)."""
    import time
    P = [c_void_p(1 << b) for b in range(49, 56)]

    def us(R, E):
        best = 1e9
        for i in range(5):  # a new shape each time, so that it is planned
            t = time.perf_counter()
            assert L.r9k_moe_gemm_w4(P[0], R, None, 1, P[1], E, R - i, 256, P[2], P[3], None, INT, 128, 64, 0, P[4], S) == -4
            best = min(best, 1e6 * (time.perf_counter() - t))
        return best
    for R, E in ((1 << 17, 1), (1 << 20, 1), (1 << 24, 2), ((1 << 31) - 1, 1), ((1 << 31) - 1, 2048)):
        assert us(R, E) < 4 * us(16, 1) + 10, (R, E)


FORMS = [(INT, 32), (INT, 64), (INT, 128), (MX, 32)]


@pytest.fixture
def plans():
    import block_scaled_fp8_r9k_amd as r9k
    yield r9k
    r9k.set_w4_plan()


def test_plan_query_and_control_checks(L, plans):
    out = (ctypes.c_int * 6)()
    assert L.r9k_w4_plan(1, 128, 16, 0, 0, INT, 128, None) == -1
    for M, K, N, E in ((-1, 128, 16, 0), (1, 100, 16, 0), (1, 128, 8, 0), (1, 128, 16, -1), (1, 128, 16, 2049)):
        assert L.r9k_w4_plan(M, K, N, E, 0, INT, 128, out) == -2
    assert L.r9k_w4_plan(1, 128, 16, 4, 1, INT, 128, out) == -2        # silu needs whole tiles in either half
    for act, fmt, g in ((1, INT, 128), (2, INT, 128), (0, 2, 32), (0, INT, 16), (0, MX, 64)):
        assert L.r9k_w4_plan(1, 128, 32, 0, act, fmt, g, out) == -7    # an act with a dense product, unknown ones
    assert L.r9k_w4_plan(0, 128, 16, 0, 0, INT, 128, out) == 0 and list(out) == [0] * 6
    for bad in ((3, 0, 0, 0, 0), (-1, 0, 0, 0, 0), (0, 1, 0, 0, 0), (0, 0, 0, 0, 2), (1, 1, 1, 1, 0), (1, 2, 0, 0, 0),
                (1, 0, 0, 0, 2), (1, 3, 1, 4, 0), (2, 3, 0, 0, 0), (2, 2, 1, 0, 0), (2, 2, 0, 1, 0), (2, 2, 0, 0, -1)):
        assert L.r9k_set_w4_plan(*bad) == -7, bad


def test_control_is_followed_and_lifted(L, plans):
    """A forced launch is the one planned, the workspace query follows it, and the planner's choice comes back; the
    calls of one thread see a change at once."""
    shape = (100, 4096, 4096)
    auto, ws = plans.w4_plan(*shape, group=32), plans.gemm_w4_workspace(*shape)
    plans.set_w4_plan(plans.W4_TILED, 4, 0, 0, 8)
    assert plans.w4_plan(*shape, group=32) == (plans.W4_TILED, 4, 4, 1, 8, 0)
    assert plans.gemm_w4_workspace(*shape) == 8 * 4 * 100 * 4096
    assert plans.w4_plan(100, 256, 4096)[4] == 2                       # the split clamped to K / 128
    assert plans.w4_plan(64, 4096, 4096, 8) == (plans.W4_TILED, 4, 4, 1, 1, 0)  # experts take none
    plans.set_w4_plan(plans.W4_TILED, 1)
    assert plans.w4_plan(64, 4096, 4096, 8)[0] == plans.W4_STREAM      # nor one tile a wave
    plans.set_w4_plan(plans.W4_STREAM, 1, 2, 4, 3)
    assert plans.w4_plan(*shape)[:5] == (plans.W4_STREAM, 1, 2, 4, 3)
    assert plans.w4_plan(64, 4096, 4096, 8, "silu_mul")[:5] == (plans.W4_STREAM, 2, 2, 4, 1)
    plans.set_w4_plan()
    assert plans.w4_plan(*shape, group=32) == auto and plans.gemm_w4_workspace(*shape) == ws


def test_forced_cases_reach_every_launch(plans):
    """The cases that the GPU tests run, on the CPU: each is planned as it is forced, and together they reach every
    instance of either kernel: one and two row tiles, one and two column tiles, slices loaded whole and streamed in
    one and in several segments, with a split and without."""
    from tests.w4_plans import STREAM_CASES, STREAM_EXPERTS, STREAM_SHAPES, TILED_CASES, TILED_EXPERT_COUNTS
    every = {(mt, nt, seg) for mt in (1, 2) for nt in (1, 2) for seg in (0, 1, 2)}
    for fmt, group in FORMS:
        seen = set()
        for M, K, N, ks in STREAM_CASES:
            for sh in STREAM_SHAPES:
                plans.set_w4_plan(plans.W4_STREAM, *sh, ks)
                p = plans.w4_plan(M, K, N, fmt=fmt, group=group)
                assert p[:3] == (plans.W4_STREAM, *sh[:2]) and p[4] == ks, (M, K, N, sh, p)
                seen.add((1 if M <= 16 else 2, p[1], min(p[5], 2), ks > 1))
        assert seen == {(*x, split) for x in every for split in (False, True)}
        for act in ("none", "silu_mul"):
            seen = set()
            for counts, K, N, topk in STREAM_EXPERTS:
                R = -(-(sum(counts) + 2) // topk) * topk
                for sh in STREAM_SHAPES:
                    if act == "none" or sh[0] == 2:
                        plans.set_w4_plan(plans.W4_STREAM, *sh)
                        p = plans.w4_plan(R, K, N, len(counts), act, fmt, group)
                        assert p[:3] == (plans.W4_STREAM, *sh[:2])
                        seen.add((1 if R <= 12 * len(counts) else 2, p[1], min(p[5], 2)))
            assert seen == {x for x in every if act == "none" or x[1] == 2}
        live = set()
        for M, K, N, splits in TILED_CASES:
            live.add((min(M, 64) + 15) // 16)
            for tn in (1, 2, 4):
                for ks in splits:
                    plans.set_w4_plan(plans.W4_TILED, tn, 0, 0, ks)
                    assert plans.w4_plan(M, K, N, fmt=fmt, group=group) == (plans.W4_TILED, tn, 4, 1, ks, 0)
        assert live == {1, 2, 3, 4}
    assert {(min(c, 64) + 15) // 16 for c in TILED_EXPERT_COUNTS} == {0, 1, 2, 3, 4}


def test_planned_launches(plans):
    """The kernel and the shape that the planner picks for sizes in use: a change of its constants shows here."""
    S, T = plans.W4_STREAM, plans.W4_TILED
    for args, kw, want in (
            ((1, 512, 1024), {}, (S, 1, 1, 4, 1, 0)),
            ((1, 4096, 14336), {}, (S, 1, 1, 4, 1, 0)),
            ((16, 14336, 4096), dict(fmt=MX, group=32), (S, 1, 4, 2, 4, 1)),
            ((100, 4096, 4096), dict(group=32), (T, 2, 4, 1, 4, 0)),
            ((4096, 4096, 12288), {}, (T, 4, 4, 1, 1, 0)),
            ((33, 14336, 2048), {}, (T, 1, 4, 1, 8, 0)),
            ((128, 2048, 1536, 128, "silu_mul"), {}, (S, 2, 4, 2, 1, 1)),
            ((16384, 768, 2048, 128), dict(fmt=MX, group=32), (T, 4, 4, 1, 1, 0))):
        assert plans.w4_plan(*args, **kw) == want, (args, kw, plans.w4_plan(*args, **kw))


@pytest.fixture
def on_host(monkeypatch):
    """The binding with host tensors let through its device check, and no call that reaches the library's launches."""
    import block_scaled_fp8_r9k_amd as r9k
    monkeypatch.setattr(r9k, "_dev", lambda t, name: -1)
    monkeypatch.setattr(r9k, "_raw", lambda stream, dev: 0)
    return r9k


def test_permute_refuses_expert_counts_before_it_allocates(on_host):
    import torch
    for E in (0, -1, -5, 2049, 1 << 40):
        with pytest.raises(on_host.R9kError) as e:
            on_host.moe_permute(None, torch.zeros((2, 2), dtype=torch.int32), E)
        assert e.value.code == -2, E


def test_weights_without_columns_are_refused(on_host):
    """Codes of no columns with scales of some: a refusal of their shape, in every call that takes a weight."""
    import torch
    bf, u8 = torch.bfloat16, torch.uint8
    for lead in ((16,), (2, 16)):
        wq, s = torch.zeros((*lead, 0), dtype=u8), torch.zeros((*lead, 2), dtype=bf)
        with pytest.raises(ValueError, match="K = 0"):
            on_host.pack_weight_w4(wq, s)
    with pytest.raises(ValueError, match="K = 0"):
        on_host.gemm_w4(torch.zeros((1, 0), dtype=bf), torch.zeros((16, 0), dtype=u8), torch.zeros((16, 2), dtype=bf))
    with pytest.raises(ValueError, match="K = 0"):
        on_host.moe_gemm_w4(torch.zeros((1, 0), dtype=bf), torch.zeros(3, dtype=torch.int32), wq, s)
    with pytest.raises(ValueError, match="K = 0"):
        on_host.quant_weight_w4(torch.zeros((16, 0), dtype=bf))


def test_unpermute_backward_without_weights_is_refused(on_host):
    """moe_unpermute takes no weights to mean 1; its gradient has a result for them and needs them."""
    import torch
    y, pos, g = torch.zeros((4, 64)), torch.zeros((2, 2), dtype=torch.int32), torch.zeros((2, 64))
    with pytest.raises(TypeError, match="w: .*ones"):
        on_host.moe_unpermute_backward(g, y, pos, None)
