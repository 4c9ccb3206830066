"""The sort and the way back at the largest counts they take."""
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


@pytest.mark.parametrize("T,k,E", [((1 << 24) - 1, 1, 2048), (1 << 20, 64, 300), ((1 << 22) + 5, 3, 1)])
def test_most_slots(r9k, T, k, E):
    """Against torch's stable sort of the same keys, with ids on either side of the range; and rows of the narrowest
    width moved there, back and through both gradients (small whole numbers: every sum is exact)."""
    say("most slots", T, k, E)
    gen = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.randint(-2, E + 2, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    x = torch.randint(-3, 4, (T, 8), generator=gen, device="cuda").to(torch.bfloat16)
    xs = torch.full((T * k, 8), 7.0, dtype=torch.bfloat16, device="cuda")
    _, src, pos, off = r9k.moe_permute(x, ids, E, xs=xs)
    flat = ids.reshape(-1)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    n = int((key < E).sum())
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key.long(), minlength=E + 1)[:E]
    assert torch.equal(off[1:].long(), torch.cumsum(counts, 0)) and int(off[0]) == 0
    assert torch.equal(src[:n].long(), order[:n]) and bool((src[n:] == -1).all())
    want = torch.full_like(order, -1)
    want[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(pos.reshape(-1).long(), want)
    del key, want
    assert torch.equal(xs[:n], x[order[:n] // k]) and bool((xs[n:] == 7.0).all())
    kept = (pos >= 0).sum(1, keepdim=True).to(torch.float32)
    w = torch.full((T, k), 2.0, device="cuda")
    assert torch.equal(r9k.moe_unpermute(xs, pos, w).float(), (2 * x.float() * kept).to(torch.bfloat16).float())
    assert torch.equal(r9k.moe_permute_backward(xs, pos).float(), (x.float() * kept).to(torch.bfloat16).float())
    gy, gw = r9k.moe_unpermute_backward(x, xs, pos, w, gy=xs.clone())
    assert torch.equal(gy[:n], 2 * xs[:n]) and torch.equal(gy[n:], xs[n:])
    assert torch.equal(gw, x.float().square().sum(1, keepdim=True) * (pos >= 0))
