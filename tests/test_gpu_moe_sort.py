"""Rows sorted by expert and back, and both gradients, against plain 64-bit forms."""
import numpy as np
import pytest
import torch

from tests import w4_ref as ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


def _ids(T, k, E, kind, seed):
    g = np.random.default_rng(seed)
    if kind == "one":                     # every slot to one expert: the same id twice in a row, the rest empty
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    ids = g.integers(0, E, (T, k))
    if kind == "drop":                    # ids on either side of the range, some tokens wholly dropped
        ids = np.where(g.random((T, k)) < 0.3, g.choice([-1, -7, E, E + 5, 2 ** 31 - 1, -2 ** 31], (T, k)), ids)
        ids[g.random(T) < 0.2] = -1
    return ids.astype(np.int32)


def _rows(n, H, dtype, seed):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((n, H), dtype=np.float32)).to(dtype)


SHAPES = [(1, 1, 1, 8, "rand"), (1, 8, 128, 2048, "rand"), (3, 2, 5, 64, "drop"), (16, 8, 128, 2048, "rand"),
          (16, 8, 128, 512, "one"), (7, 4, 9, 136, "none"), (64, 64, 64, 72, "drop"), (255, 6, 60, 264, "drop"),
          (300, 8, 128, 256, "rand"), (512, 8, 2048, 128, "drop"), (1025, 5, 33, 96, "drop"), (3001, 8, 257, 64, "rand"),
          (4097, 10, 128, 40, "one"), (40000, 8, 512, 16, "drop")]


@pytest.mark.parametrize("T,k,E,H,kind", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_permute(r9k, T, k, E, H, kind, dtype):
    say("permute", T, k, E, H, kind, dtype)
    ids = _ids(T, k, E, kind, T + E)
    x = _rows(T, H, dtype, T)
    src, pos, off = ref.sort(ids, E)
    xs = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    got = r9k.moe_permute(x.cuda(), torch.from_numpy(ids).cuda(), E, xs=xs)
    assert got[0] is xs
    for g, w, name in zip(got[1:], (src, pos, off), ("src", "pos", "offsets")):
        assert np.array_equal(g.cpu().numpy(), w), name
    want = torch.full((T * k, H), 7.0, dtype=dtype)           # rows behind the last kept one keep what they held
    n = off[E]
    want[:n] = x[torch.from_numpy(src[:n]).long() // k]
    assert torch.equal(xs.cpu(), want)
    alone = r9k.moe_permute(None, torch.from_numpy(ids).cuda(), E)
    assert alone[0] is None and all(torch.equal(a, b) for a, b in zip(alone[1:], got[1:]))


def _bound(dtype, want, mag, n):
    """n additions of fp32 terms, each rounded once more when it is weighted, then one rounding to the rows' type."""
    before = (n + 1) * 2.0 ** -23 * mag
    return before + torch.finfo(dtype).eps / 2 * (want.abs() + before)


@pytest.mark.parametrize("T,k,E,H,kind", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_unpermute_and_gradients(r9k, T, k, E, H, kind, dtype):
    say("unpermute", T, k, E, H, kind, dtype)
    ids = _ids(T, k, E, kind, T + E)
    src, pos, off = ref.sort(ids, E)
    n = int(off[E])
    y = _rows(T * k, H, dtype, T + 1)
    y[n:] = float("nan")                                      # nobody's rows: never read
    w = torch.from_numpy(np.random.default_rng(T + 2).random((T, k), dtype=np.float32))
    g = _rows(T, H, dtype, T + 3)
    yd, posd, wd, gd = y.cuda(), torch.from_numpy(pos).cuda(), w.cuda(), g.cuda()

    clean = torch.nan_to_num(y)
    want, mag = ref.unpermute(clean, pos, w)
    got = r9k.moe_unpermute(yd, posd, wd).cpu().to(ref.F64)
    assert torch.all((got - want).abs() <= _bound(dtype, want, mag, k))
    want, mag = ref.unpermute(clean, pos, None)
    got = r9k.moe_unpermute(yd, posd).cpu()
    assert torch.all((got.to(ref.F64) - want).abs() <= _bound(dtype, want, mag, k))
    assert torch.equal(r9k.moe_permute_backward(yd, posd).cpu(), got)

    gy = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    gy2, gw = r9k.moe_unpermute_backward(gd, yd, posd, wd, gy=gy)
    assert gy2 is gy
    s = torch.from_numpy(src[:n]).long()
    want = torch.full((T * k, H), 7.0, dtype=ref.F64)
    want[:n] = g.to(ref.F64)[s // k] * w.to(ref.F64).reshape(-1)[s][:, None]
    err = (gy.cpu().to(ref.F64) - want).abs()
    assert torch.all(err[:n] <= _bound(dtype, want, want.abs(), 0)[:n]) and torch.all(err[n:] == 0)
    term = torch.zeros(T * k, H, dtype=ref.F64)
    term[s] = g.to(ref.F64)[s // k] * clean.to(ref.F64)[:n]
    want, mag = term.sum(1).view(T, k), term.abs().sum(1).view(T, k)
    assert torch.all((gw.cpu().to(ref.F64) - want).abs() <= (H + 1) * 2.0 ** -23 * mag)


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_against_differences(r9k, dtype):
    """Both maps are linear in the rows and in the weights, so a central difference of the 64-bit forward along a
    direction is the derivative itself, with no error of its own."""
    T, k, E, H = 37, 4, 11, 200
    ids = _ids(T, k, E, "drop", 5)
    src, pos, off = ref.sort(ids, E)
    n = int(off[E])
    rnd = lambda *s, seed: torch.from_numpy(np.random.default_rng(seed).standard_normal(s))
    y, w, g = rnd(T * k, H, seed=1).to(dtype), rnd(T, k, seed=2).float(), rnd(T, H, seed=3).to(dtype)
    vy, vw = rnd(T * k, H, seed=4), rnd(T, k, seed=5)
    loss = lambda yy, ww: (ref.unpermute(yy, pos, ww)[0] * g.to(ref.F64)).sum()
    dy = (loss(y.to(ref.F64) + vy, w) - loss(y.to(ref.F64) - vy, w)) / 2
    dw = (loss(y, w.to(ref.F64) + vw) - loss(y, w.to(ref.F64) - vw)) / 2
    posd = torch.from_numpy(pos).cuda()
    gy, gw = r9k.moe_unpermute_backward(g.cuda(), y.cuda(), posd, w.cuda())
    gy = gy.cpu().to(ref.F64)[:n]
    half = torch.finfo(dtype).eps / 2
    assert abs((gy * vy[:n]).sum() - dy) <= (half + 2.0 ** -23) / (1 - half) * (gy * vy[:n]).abs().sum()
    s = torch.from_numpy(src[:n]).long()
    mag = torch.zeros(T * k, dtype=ref.F64)
    mag[s] = (g.to(ref.F64)[s // k] * y.to(ref.F64)[:n]).abs().sum(1)
    assert abs((gw.cpu().to(ref.F64) * vw).sum() - dw) <= (H + 1) * 2.0 ** -23 * (mag.view(T, k) * vw.abs()).sum() + 1e-12 * abs(dw)
    # the sort's gradient: loss(x) = <sorted rows of x, g2>
    g2 = rnd(T * k, H, seed=6).to(dtype)
    vx = rnd(T, H, seed=7)
    sorted_loss = lambda x: (x[s // k] * g2.to(ref.F64)[:n]).sum()
    dx = (sorted_loss(vx) - sorted_loss(-vx)) / 2
    gx = r9k.moe_permute_backward(g2.cuda(), posd).cpu().to(ref.F64)
    _, mag = ref.unpermute(g2, pos, None)
    assert abs((gx * vx).sum() - dx) <= ((half + (k + 1) * 2.0 ** -22) * mag * vx.abs()).sum()


def test_zero_weight_and_infinite_rows(r9k):
    """A dropped slot's weight and rows, whatever they hold, reach nothing; a kept slot's infinity stays one."""
    pos = torch.tensor([[0, -1], [-1, -1], [2, 1]], dtype=torch.int32).cuda()
    y = torch.ones((6, 16), dtype=torch.float32)
    y[3:] = float("nan")
    y[2, 5] = float("inf")
    w = torch.tensor([[0.5, float("nan")], [float("inf"), 1.0], [2.0, 3.0]])
    out = r9k.moe_unpermute(y.cuda(), pos, w.cuda()).cpu()
    want = torch.stack((torch.full((16,), 0.5), torch.zeros(16), torch.full((16,), 5.0)))
    want[2, 5] = float("inf")
    assert torch.equal(out, want)
    gy, gw = r9k.moe_unpermute_backward(torch.ones((3, 16)).cuda(), y.cuda(), pos, w.cuda(), gy=torch.zeros((6, 16)).cuda())
    assert torch.equal(gw.cpu()[0], torch.tensor([16.0, 0.0])) and torch.equal(gw.cpu()[1], torch.zeros(2))
    assert torch.equal(gy.cpu()[:, 0], torch.tensor([0.5, 3.0, 2.0, 0.0, 0.0, 0.0]))


def test_positions_out_of_range_count_as_dropped(r9k):
    pos = torch.tensor([[0, 6], [2 ** 31 - 1, -5]], dtype=torch.int32).cuda()
    y = torch.arange(4, dtype=torch.float32)[:, None].expand(4, 8).contiguous() + 1
    assert torch.equal(r9k.moe_unpermute(y.cuda(), pos).cpu()[:, 0], torch.tensor([1.0, 0.0]))


def test_empty_batch(r9k):
    ids = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    x = torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")
    xs, src, pos, off = r9k.moe_permute(x, ids, 6)
    assert xs.shape == (0, 64) and src.shape == (0,) and pos.shape == (0, 4) and torch.equal(off.cpu(), torch.zeros(7, dtype=torch.int32))
    assert r9k.moe_unpermute(xs, pos, torch.zeros((0, 4), device="cuda")).shape == (0, 64)
    gy, gw = r9k.moe_unpermute_backward(x, xs, pos, torch.zeros((0, 4), device="cuda"))
    assert gy.shape == (0, 64) and gw.shape == (0, 4)


def test_refusals(r9k):
    dev = dict(device="cuda")
    ids = torch.zeros((4, 2), dtype=torch.int32, **dev)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, **dev)
    ys, pos = torch.zeros((8, 64), dtype=torch.bfloat16, **dev), torch.zeros((4, 2), dtype=torch.int32, **dev)
    w = torch.zeros((4, 2), **dev)
    with pytest.raises(TypeError):
        r9k.moe_permute(x.half(), ids, 4)
    with pytest.raises(TypeError):
        r9k.moe_permute(x, ids.long(), 4)
    with pytest.raises(ValueError):
        r9k.moe_permute(x[:3], ids, 4)
    with pytest.raises(ValueError):
        r9k.moe_permute(x.t(), ids, 4)
    with pytest.raises(ValueError):
        r9k.moe_permute(x, ids.t().contiguous().t(), 4)
    with pytest.raises(ValueError):
        r9k.moe_permute(x, ids, 4, xs=torch.zeros((7, 64), dtype=torch.bfloat16, **dev))
    with pytest.raises(ValueError):
        r9k.moe_permute(x.cpu(), ids, 4)
    with pytest.raises(r9k.R9kError) as e:
        r9k.moe_permute(x, ids, 4096)
    assert e.value.code == -2
    with pytest.raises(r9k.R9kError) as e:
        r9k.moe_permute(torch.zeros((4, 4), dtype=torch.bfloat16, **dev), ids, 4)
    assert e.value.code == -2
    with pytest.raises(ValueError):
        r9k.moe_unpermute(ys[:7], pos)
    with pytest.raises(ValueError):
        r9k.moe_unpermute(ys, pos, w[:, :1].contiguous())
    with pytest.raises(TypeError):
        r9k.moe_unpermute(ys, pos, w.bfloat16())
    with pytest.raises(TypeError):
        r9k.moe_unpermute_backward(x.float(), ys, pos, w)
    with pytest.raises(r9k.R9kError) as e:
        r9k.moe_unpermute_backward(x, ys, pos, w, gy=ys)
    assert e.value.code == -7


def test_rows_past_4_gib(r9k):
    """Sorted rows of 4.4 GiB: every row is its token's, and the way back gives each token topk times itself."""
    T, k, E, H = 36000, 8, 64, 8192
    ids = torch.from_numpy(_ids(T, k, E, "rand", 1)).cuda()
    x = torch.randn((T, H), device="cuda").to(torch.bfloat16)
    xs, src, pos, off = r9k.moe_permute(x, ids, E)
    for lo in range(0, T * k, 40000):
        hi = min(T * k, lo + 40000)
        assert torch.equal(xs[lo:hi], x[src[lo:hi].long() // k])
    assert torch.equal(r9k.moe_permute_backward(xs, pos), x * 8)      # a power of two: exact
    gy, gw = r9k.moe_unpermute_backward(x, xs, pos, torch.full((T, k), 0.5, device="cuda"))
    for lo in range(0, T * k, 40000):
        hi = min(T * k, lo + 40000)
        assert torch.equal(gy[lo:hi], xs[lo:hi] * 0.5)


def test_graphs_and_streams(r9k):
    """Two sorts of different sizes captured and replayed in turn with eager work between, and a side stream."""
    cases = []
    for T, k, E, H in ((40, 4, 16, 256), (3000, 6, 50, 512)):
        ids = torch.from_numpy(_ids(T, k, E, "drop", T)).cuda()
        x, w = _rows(T, H, torch.bfloat16, T).cuda(), torch.rand((T, k), device="cuda")

        def step(x=x, ids=ids, w=w, E=E, xs=torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda"),
                 gy=torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda"), **kw):
            _, src, pos, off = r9k.moe_permute(x, ids, E, xs=xs, **kw)
            out = r9k.moe_unpermute(xs, pos, w, **kw)
            return [src, pos, off, out, *r9k.moe_unpermute_backward(x, xs, pos, w, gy=gy, **kw)]
        want = [t.clone() for t in step()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = step(stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = step()
        cases.append((g, outs, want, step))
    for _ in range(4):
        for g, outs, want, step in cases:
            for t in outs:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
            assert all(torch.equal(a, b) for a, b in zip(step(), want))
