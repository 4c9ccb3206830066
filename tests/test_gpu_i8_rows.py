"""The 8-bit experts' products at the most rows that they take, 2^31 - 1, nearly all of them one expert's."""
import pytest
import torch

from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


@pytest.mark.parametrize("E", [2, 300])
def test_the_most_rows(r9k, E):
    """79 GB.  Row blocks are counted up, and 2^31 - 4 rows and a block's less one pass 2^31."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB")
    T, k, K, N, big, last = 1 << 25, 64, 128, 16, E // 2, E - 1
    R = T * k - 1
    g = torch.Generator("cuda").manual_seed(E)
    q = torch.randint(-127, 128, (T, K), dtype=torch.int8, device="cuda", generator=g)
    s = torch.rand(T, device="cuda", generator=g)
    w = torch.randint(-127, 128, (E, N, K), dtype=torch.int8, device="cuda", generator=g)
    ws = torch.rand((E, N), device="cuda", generator=g)
    p = r9k.pack_weight_i8(w)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[big + 1:] = R - 3
    off[last + 1:] = R
    src = torch.arange(R, dtype=torch.int32, device="cuda")
    c = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    say("moe_gemm_i8", R, K, N, E)
    r9k.moe_gemm_i8(q, s, off, p, ws, src=src, topk=k, c=c)
    step = 1 << 20
    for t in range(0, T, step):
        n = min(step, T - t - 1)                                            # the last token has an expert's three rows
        want = r9k.gemm_i8(q[t:t + n], s[t:t + n], p[big], ws[big])
        assert torch.equal(c[t * k:(t + n) * k].view(n, k, N), want[:, None].expand(n, k, N)), t
    tail = r9k.gemm_i8(q[-1:], s[-1:].clone(), p[big], ws[big]), r9k.gemm_i8(q[-1:], s[-1:].clone(), p[last], ws[last])
    assert torch.equal(c[R - 63:R - 3], tail[0].expand(60, N)) and torch.equal(c[R - 3:], tail[1].expand(3, N))
    del q, s, src, c
    torch.cuda.empty_cache()
