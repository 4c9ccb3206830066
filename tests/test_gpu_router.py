"""The router's training operators: the balance loss with its counts, and the gradients of the logits, against 64-bit
forms and against differences; and a training step's pass through router, sort and 8-bit experts."""
import numpy as np
import pytest
import torch

import inputs
from tests import i8_ref as ref
from tests import w4_ref
from tests.gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


SHAPES = [(1, 1, 1), (8193, 3, 1), (300, 520, 33), (1, 8, 2), (3, 2, 2), (5, 7, 3), (64, 8, 2), (100, 128, 8), (257, 60, 4), (1000, 256, 8), (333, 129, 5),
          (77, 512, 10), (50, 1000, 6), (130, 2048, 8), (31, 2047, 64), (2100, 16, 4), (9000, 64, 6), (40000, 10, 2)]


def batch(T, E, k, kind, bf16=False, seed=0):
    """Logits, ids and mask.  kinds: plain; mask (a third of the tokens out); drop (ids outside the range);
    closed (half the logits -inf, one token's all); lowest (half the logits the type's lowest value); far (logits
    hundreds apart); same (an expert several times in a row)."""
    g = np.random.default_rng(T * 31 + E + seed)
    dt = torch.bfloat16 if bf16 else torch.float32
    x = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32))
    if kind == "far":
        x = x * 100
    if kind in ("closed", "lowest"):
        low = -float("inf") if kind == "closed" else torch.finfo(dt).min
        x[torch.from_numpy(g.random((T, E)) < 0.5)] = low
        x[T // 2] = low
    ids = torch.from_numpy(g.integers(0, E, (T, k)).astype(np.int32))
    if kind != "same" and k <= E:
        ids = torch.from_numpy(np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32))
    if kind == "drop":
        ids[torch.from_numpy(g.random((T, k)) < 0.3)] = -1
        ids[0, 0] = E
    mask = torch.from_numpy(g.random(T) < 0.66) if kind == "mask" else None
    return x.to(dt), ids, mask


def on_gpu(*ts):
    return tuple(None if t is None else t.cuda() for t in ts)


@pytest.mark.parametrize("kind", ["plain", "mask", "drop", "closed", "lowest", "far", "same"])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_balance_loss(r9k, T, E, k, kind):
    for bf16 in (False, True):
        say("balance", T, E, k, kind, bf16)
        x, ids, mask = batch(T, E, k, kind, bf16)
        (loss, counts, psum), (bl, bp) = ref.balance(x, ids, mask)
        got = r9k.moe_balance_loss(*on_gpu(x, ids, mask))
        assert torch.equal(got[1].cpu(), counts)
        assert torch.all((got[2].cpu().to(ref.F64) - psum).abs() <= bp)
        assert abs(float(got[0]) - float(loss)) <= float(bl)
        again = r9k.moe_balance_loss(*on_gpu(x, ids, mask))
        assert all(torch.equal(a, b) for a, b in zip(got, again))          # the same bits again


@pytest.mark.parametrize("kind", ["plain", "mask", "drop", "closed", "lowest", "far", "same"])
@pytest.mark.parametrize("T,E,k", [s for s in SHAPES if s[0] <= 1000])
def test_gradients(r9k, T, E, k, kind):
    g = np.random.default_rng(T + E)
    gw, w = (torch.from_numpy(g.standard_normal((T, k)).astype(np.float32)) for _ in range(2))
    w = torch.softmax(w, 1)
    for bf16 in (False, True):
        say("gradients", T, E, k, kind, bf16)
        x, ids, mask = batch(T, E, k, kind, bf16)
        if mask is not None:
            x[~mask] = float("nan")                                        # padding may hold anything
        _, counts, _ = ref.balance(torch.nan_to_num(x.float()), ids, mask)[0]
        gloss = torch.tensor(0.37 * T)
        want, err = ref.balance_grad(gloss, x, counts, k, mask)
        rw, rerr = ref.route_grad(gw, ids, w, E)
        half = lambda v, e: e + (2.0 ** -8 * (v.abs() + e) + 2.0 ** -134 if bf16 else 0.0)
        out = r9k.moe_balance_loss_backward(*on_gpu(gloss, x, counts), k, mask=on_gpu(mask)[0])
        assert out.dtype == x.dtype
        assert torch.all((out.cpu().to(ref.F64) - want).abs() <= half(want, err))
        out = r9k.moe_balance_loss_backward(*on_gpu(gloss, x, counts), k, mask=on_gpu(mask)[0], route=on_gpu(gw, ids, w))
        both, berr = want + rw, err + rerr + 2 * ref.U * (want.abs() + rw.abs()) * (k + 1)
        assert torch.all((out.cpu().to(ref.F64) - both).abs() <= half(both, berr))
    out = r9k.moe_route_backward(*on_gpu(gw, ids, w), E)
    assert torch.all((out.cpu().to(ref.F64) - rw).abs() <= rerr)


def test_route_gradient_of_many_experts(r9k):
    for T, E, k in ((3, 65536, 64), (70, 5000, 8), (2, 65535, 1)):
        g = np.random.default_rng(E)
        ids = torch.from_numpy(g.integers(0, E, (T, k)).astype(np.int32))
        ids[0, 0], ids[-1, -1] = E - 1, 0
        gw = torch.from_numpy(g.standard_normal((T, k)).astype(np.float32))
        w = torch.softmax(gw * 0.3, 1)
        out = r9k.moe_route_backward(*on_gpu(gw, ids, w), E)
        want, err = ref.route_grad(gw, ids, w, E)
        assert torch.all((out.cpu().to(ref.F64) - want).abs() <= err)


def test_no_tokens_and_no_kept_tokens(r9k):
    E, k = 8, 2
    loss, counts, psum = r9k.moe_balance_loss(torch.empty((0, E)).cuda(), torch.empty((0, k), dtype=torch.int32).cuda())
    assert float(loss) == 0 and not counts.any() and not psum.any()
    x, ids, _ = batch(5, E, k, "plain")
    x[1] = float("nan")
    none = torch.zeros(5, dtype=torch.bool)
    loss, counts, psum = r9k.moe_balance_loss(*on_gpu(x, ids, none))
    assert float(loss) == 0 and not counts.any() and not psum.any()
    g = r9k.moe_balance_loss_backward(torch.tensor(1.0).cuda(), x.cuda(), counts, k, mask=none.cuda())
    assert torch.all(g == 0)
    assert r9k.moe_balance_loss_backward(torch.tensor(1.0).cuda(), x[:0].cuda(), counts, k).shape == (0, E)
    assert r9k.moe_route_backward(torch.empty((0, k)).cuda(), ids[:0].cuda(), torch.empty((0, k)).cuda(), E).shape == (0, E)


def test_logits_that_are_not_finite_show(r9k):
    x, ids, _ = batch(40, 16, 2, "plain")
    for v in (float("nan"), float("inf")):
        y = x.clone()
        y[7, 3] = v
        loss, counts, _ = r9k.moe_balance_loss(*on_gpu(y, ids))
        assert torch.isnan(loss)
        g = r9k.moe_balance_loss_backward(torch.tensor(1.0).cuda(), y.cuda(), counts, 2).cpu()
        fine = r9k.moe_balance_loss_backward(torch.tensor(1.0).cuda(), x.cuda(), counts, 2).cpu()
        rows = torch.arange(40) != 7
        assert torch.isnan(g[7]).any() and torch.equal(g[rows], fine[rows])


def test_gradients_against_differences(r9k):
    """Central differences of the forward pass.  With a step of h the difference is off by h^2 / 6 of the third derivative: at
    most 1/8 for a probability p (of p (1 - p) (1 - 6 p + 6 p^2)) and as much for all others together, so 1/4 of the largest
    factor, E / k for the loss and max |gw| for the routing weights; and by the error of the fp32 loss over h."""
    T, E, k, h = 6, 8, 2, 2.0 ** -6
    x, _, mask = batch(T, E, k, "mask", seed=3)
    mask[:2] = torch.tensor([True, False])
    x, mask = x.cuda(), mask.cuda()
    ids, w = r9k.moe_route(x, k)
    loss, counts, _ = r9k.moe_balance_loss(x, ids, mask=mask)
    gw = torch.randn((T, k), generator=torch.Generator().manual_seed(1)).cuda()
    gloss = torch.tensor(3.0).cuda()
    g = r9k.moe_balance_loss_backward(gloss, x, counts, k, mask=mask, route=(gw, ids, w)).cpu()

    def value(y):
        l, c, _ = r9k.moe_balance_loss(y, ids, mask=mask)
        z = torch.gather(y, 1, ids.long()).double()
        return 3.0 * float(l) + float((torch.softmax(z, 1) * gw.double()).sum())
    for t in range(T):
        for e in range(E):
            up, dn = x.clone(), x.clone()
            up[t, e] += h
            dn[t, e] -= h
            d = (value(up) - value(dn)) / float(up[t, e].double() - dn[t, e].double())
            bound = h * h / 24 * (3.0 * E / k + float(gw[t].abs().max())) + 3.0 * float(loss) * 64 * ref.U / h
            assert abs(d - float(g[t, e])) <= bound, (t, e, d, float(g[t, e]))


def test_counts_of_two_shards_add_up(r9k):
    """The gradient with counts added over two shards is the whole batch's."""
    x, ids, mask = batch(300, 32, 4, "mask")
    whole = r9k.moe_balance_loss(*on_gpu(x, ids, mask))
    parts = [r9k.moe_balance_loss(*on_gpu(x[s].contiguous(), ids[s].contiguous(), mask[s].clone())) for s in (slice(0, 112), slice(112, 300))]
    counts = parts[0][1] + parts[1][1]
    assert torch.equal(counts, whole[1])
    gl = torch.tensor(2.0).cuda()
    g = r9k.moe_balance_loss_backward(gl, x.cuda(), whole[1], 4, mask=mask.cuda())
    for s in (slice(0, 112), slice(112, 300)):
        assert torch.equal(r9k.moe_balance_loss_backward(gl, x[s].contiguous().cuda(), counts, 4, mask=mask[s].clone().cuda()), g[s])


def test_streams_outputs_and_graphs(r9k):
    cases = [batch(T, E, k, kind) + (k,) for T, E, k, kind in ((64, 8, 2, "plain"), (5000, 128, 8, "mask"), (300, 60, 4, "drop"))]
    runs = []
    for x, ids, mask, k in cases:
        x, ids, mask = on_gpu(x, ids, mask)
        E = x.shape[1]
        ref_out = r9k.moe_balance_loss(x, ids, mask=mask)
        ws = torch.full((r9k.moe_balance_loss_workspace(x.shape[0], E, k) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        own = [torch.full((), 9.0).cuda(), torch.full((E + 1,), 9, dtype=torch.int32).cuda(), torch.full((E,), 9.0).cuda()]
        out = r9k.moe_balance_loss(x, ids, mask=mask, loss=own[0], counts=own[1], psum=own[2], workspace=ws)
        assert all(a is b and torch.equal(a, c) for a, b, c in zip(out, own, ref_out))
        gl = torch.tensor(1.5).cuda()
        grad = r9k.moe_balance_loss_backward(gl, x, ref_out[1], k, mask=mask)
        runs.append((x, ids, mask, k, gl, ref_out, grad))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, ids, mask, k, gl, want, grad in runs:
        out = r9k.moe_balance_loss(x, ids, mask=mask, stream=side)
        g = r9k.moe_balance_loss_backward(gl, x, out[1], k, mask=mask, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(g, grad)
    graphs = []
    for x, ids, mask, k, gl, want, grad in runs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = r9k.moe_balance_loss(x, ids, mask=mask)
            g = r9k.moe_balance_loss_backward(gl, x, out[1], k, mask=mask)
        graphs.append((gr, out, g))
    for _ in range(4):
        for (gr, out, g), (x, ids, mask, k, gl, want, grad) in zip(graphs, runs):
            g.zero_()
            gr.replay()
            assert torch.equal(r9k.moe_balance_loss_backward(gl, x, want[1], k, mask=mask), grad)
        torch.cuda.synchronize()
        for (gr, out, g), (*_, want, grad) in zip(graphs, runs):
            assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(g, grad)


def test_refusals(r9k):
    x, ids, mask = on_gpu(*batch(20, 16, 2, "mask"))
    loss, counts, psum = r9k.moe_balance_loss(x, ids, mask=mask)
    gl = torch.tensor(1.0).cuda()
    gw, w = torch.ones((20, 2)).cuda(), torch.ones((20, 2)).cuda()
    for bad in (lambda: r9k.moe_balance_loss(x, ids[:5]), lambda: r9k.moe_balance_loss(x, ids, mask=mask[:5]),
                lambda: r9k.moe_balance_loss(x[0], ids), lambda: r9k.moe_balance_loss(x.t(), ids),
                lambda: r9k.moe_balance_loss(x.cpu(), ids), lambda: r9k.moe_balance_loss(x, ids.cpu()),
                lambda: r9k.moe_balance_loss(x, ids, loss=torch.empty(1).cuda()),
                lambda: r9k.moe_balance_loss(x, ids, counts=counts[:16]),
                lambda: r9k.moe_balance_loss_backward(gl, x, counts[:16], 2),
                lambda: r9k.moe_balance_loss_backward(gl[None], x, counts, 2),
                lambda: r9k.moe_balance_loss_backward(gl, x, counts, 2, route=(gw, ids, w[:5])),
                lambda: r9k.moe_balance_loss_backward(gl, x, counts, 3, route=(gw, ids, w)),
                lambda: r9k.moe_route_backward(gw, ids, w[:5], 16), lambda: r9k.moe_route_backward(gw[0], ids, w, 16)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: r9k.moe_balance_loss(x.half(), ids), lambda: r9k.moe_balance_loss(x, ids.long()),
                lambda: r9k.moe_balance_loss(x, ids, mask=mask.float()),
                lambda: r9k.moe_balance_loss_backward(gl.double(), x, counts, 2),
                lambda: r9k.moe_balance_loss_backward(gl, x, counts, 2, glogits=torch.empty_like(x, dtype=torch.bfloat16))):
        with pytest.raises(TypeError):
            bad()
    big = torch.zeros((2, 4096)).cuda()
    for bad, code in ((lambda: r9k.moe_balance_loss(big, ids[:2]), -2),
                      (lambda: r9k.moe_balance_loss(x, torch.zeros((20, 65), dtype=torch.int32).cuda()), -2),
                      (lambda: r9k.moe_balance_loss(*on_gpu(*batch(2100, 16, 2, "plain")[:2]), workspace=torch.empty(16, dtype=torch.uint8).cuda()), -6),
                      (lambda: r9k.moe_balance_loss_backward(gl, x, counts, 2, glogits=x), -7),     # in place
                      (lambda: r9k.moe_balance_loss_backward(gl, x, counts, 0), -2),
                      (lambda: r9k.moe_route_backward(gw, ids, w, 2, glogits=gw), -7),
                      (lambda: r9k.moe_route_backward(gw, ids, w, 0), -2),
                      (lambda: r9k.moe_route_backward(gw, ids, w, 1 << 40), -2)):
        with pytest.raises(r9k.R9kError) as e:
            bad()
        assert e.value.code == code


def test_a_training_step_through_router_and_experts(r9k):
    """Routing, sort, 8-bit experts, the way back, and the gradients back to the router's logits, each stage against its
    plain form on the stage before."""
    T, H, I, E, k = 150, 256, 128, 16, 4
    g = np.random.default_rng(5)
    x = torch.from_numpy(inputs.activations(1, T, H).view(np.int16)).view(torch.bfloat16)
    logits, _, mask = batch(T, E, k, "mask")
    w13 = torch.from_numpy((0.02 * g.standard_normal((E, 2 * I, H))).astype(np.float32)).to(torch.bfloat16)
    w2 = torch.from_numpy((0.02 * g.standard_normal((E, H, I))).astype(np.float32)).to(torch.bfloat16)
    (q13, s13), (q2, s2) = r9k.quant_i8(w13.cuda()), r9k.quant_i8(w2.cuda())
    p13, p2 = r9k.pack_weight_i8(q13), r9k.pack_weight_i8(q2)
    ld, md = logits.cuda(), mask.cuda()

    ids, tw = r9k.moe_route(ld, k)
    loss, counts, psum = r9k.moe_balance_loss(ld, ids, mask=md)
    _, src, pos, off = r9k.moe_permute(None, ids, E)
    xq, xs = r9k.quant_i8(x.cuda())
    h = r9k.moe_gemm_i8(xq, xs, off, p13, s13, src=src, topk=k, act="silu_mul")
    hq, hs = r9k.quant_i8(h)
    y = r9k.moe_gemm_i8(hq, hs, off, p2, s2)
    out = r9k.moe_unpermute(y, pos, tw)
    gout = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).cuda()
    gy, gw = r9k.moe_unpermute_backward(gout, y, pos, tw)
    gloss = torch.tensor(0.01 * T).cuda()
    gl = r9k.moe_balance_loss_backward(gloss, ld, counts, k, mask=md, route=(gw, ids, tw))

    cpu = lambda *t: [v.cpu() for v in t]
    ids, tw, src, pos, off, h, y, gw, counts = cpu(ids, tw, src, pos, off, h, y, gw, counts)
    rsrc, rpos, roff = w4_ref.sort(ids.numpy(), E)
    assert np.array_equal(src.numpy(), rsrc) and np.array_equal(off.numpy(), roff)
    rows = src.long() // k
    rq, rs = ref.quant(x)
    wq13, ws13, wq2, ws2 = cpu(q13, s13, q2, s2)
    hq_ref, hs_ref = ref.quant(h)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        v = ref.product32(rq[rows[lo:hi]], rs[rows[lo:hi]], wq13[e], ws13[e]).to(ref.F64)
        none = torch.zeros_like(v[:, :I])
        wh, bh = w4_ref.silu_mul(v[:, :I], v[:, I:], none, none)
        assert torch.all((h[lo:hi].to(ref.F64) - wh).abs() <= ref.bf16_bound(wh, bh))
        assert torch.equal(y[lo:hi], ref.product32(hq_ref[lo:hi], hs_ref[lo:hi], wq2[e], ws2[e]).to(torch.bfloat16))
    want, mag = w4_ref.unpermute(y, pos.numpy(), tw)
    assert torch.all((out.cpu().to(ref.F64) - want).abs() <= w4_ref.bf16_bound(want, (k + 1) * 2.0 ** -23 * mag))
    (wl, wc, wp), (bl, bp) = ref.balance(logits, ids, mask)
    assert torch.equal(counts, wc) and abs(float(loss) - float(wl)) <= float(bl)
    a, ea = ref.balance_grad(gloss.cpu(), logits, counts, k, mask)
    b, eb = ref.route_grad(gw, ids, tw, E)
    assert torch.all((gl.cpu().to(ref.F64) - a - b).abs() <= ea + eb + 2 * ref.U * (a.abs() + b.abs()) * (k + 1))
    # the tokens' experts got the slots that were counted, and the sort's ranges are as long as the unmasked counts
    assert int(counts[E]) == int(mask.sum()) and int(counts[:E].sum()) == k * int(mask.sum())
