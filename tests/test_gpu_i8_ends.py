"""The 8-bit products and the router's training operators where sizes and use end: many tiles a CTA, offsets past 32 bits,
calls from two threads and on two streams at once, graphs that share a workspace, and the checks of calls with every
output given."""
import threading

import pytest
import torch

from tests import i8_ref as ref
from tests import w4_ref
from tests.gpu_util import say
from tests.test_gpu_i8 import acts, routing, weight
from tests.test_gpu_i8_plans import TILES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def r9k():
    import block_scaled_fp8_r9k_amd as m
    assert torch.cuda.is_available()
    m.lib()
    yield m
    m.set_i8_plan()


def on_device(q, s, w, ws):
    """ref.product32 on the GPU.  With K * 127^2 < 2^24 every partial sum is a whole number that fp32 holds, so that
    any order of the sum gives the integers."""
    assert q.shape[1] * 127 * 127 < 1 << 24
    return ((q.float() @ w.float().T) * s[:, None] * ws).to(torch.bfloat16)


@pytest.mark.parametrize("K", [128, 384, 1024])
def test_many_tiles_a_cta(r9k, K):
    """More tiles than CTAs in every shape, so that a CTA's next stages are under way while it stores; chunks in odd
    numbers, and fewer of them than the ring has stages."""
    M, N = 4500, 4112
    g = torch.Generator("cuda").manual_seed(K)
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    s, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    p, want = r9k.pack_weight_i8(w), on_device(q, s, w, ws)
    off = torch.tensor([0, 700, 700, 2600, 4444], dtype=torch.int32, device="cuda")
    wE = torch.stack([w.roll(e, 0) for e in range(4)])
    pE, wsE = r9k.pack_weight_i8(wE), ws.expand(4, N).contiguous()
    wantE = torch.cat([on_device(q[a:b], s[a:b], wE[e], ws) for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:]))])
    try:
        for tile in TILES:
            for ks in (1, 2):
                say("tiles", tile, K, "split", ks)
                r9k.set_i8_plan(r9k.I8_TILED, *tile, 0, ks)
                c = torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device="cuda")
                r9k.gemm_i8(q, s, p, ws, c=c[:M])
                assert torch.equal(c[:M], want) and torch.all(c[M:] == 7.0), (tile, ks)
            c = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
            r9k.moe_gemm_i8(q, s, off, pE, wsE, c=c)
            assert torch.equal(c[:4444], wantE) and torch.all(c[4444:] == 7.0), tile
    finally:
        r9k.set_i8_plan()


def test_outputs_past_32_bits(r9k):
    """2.3e9 outputs, 4.6 GB: the last rows are as right as the first."""
    M, N, K = 70001, 32768, 128
    g = torch.Generator("cuda").manual_seed(1)
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    s, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    p = r9k.pack_weight_i8(w)
    say("gemm_i8", M, K, N)
    c = r9k.gemm_i8(q, s, p, ws)
    for lo in (0, 32700, 65500, M - 300):
        assert torch.equal(c[lo:lo + 300], on_device(q[lo:lo + 300], s[lo:lo + 300], w, ws)), lo
    off = torch.tensor([0, M - 5, M], dtype=torch.int32, device="cuda")
    pE = torch.stack([p, p])
    say("moe_gemm_i8", M, K, N)
    r9k.moe_gemm_i8(q, s, off, pE, torch.stack([ws, 2 * ws]), c=c)
    for lo, hi, f in ((0, 300, 1), (65500, 65800, 1), (M - 300, M - 5, 1), (M - 5, M, 2)):
        assert torch.equal(c[lo:hi], on_device(q[lo:hi], s[lo:hi], w, f * ws)), lo


def test_activations_past_32_bits(r9k):
    """Tokens' rows that take 4.3 GB, read through the sort's index, and the same rows read in their order."""
    K, N, rows = 16384, 32, (1 << 18) + 40
    q = torch.zeros((rows, K), dtype=torch.int8, device="cuda")
    at = torch.tensor([0, 1, 77, 131071, 131072, 262143, 262144, 262183], device="cuda")
    g = torch.Generator("cuda").manual_seed(2)
    small = torch.randint(-31, 32, (len(at), K), dtype=torch.int8, device="cuda", generator=g)
    q[at] = small
    s = torch.zeros(rows, device="cuda")
    s[at] = torch.rand(len(at), device="cuda", generator=g) + 0.5
    w = torch.randint(-31, 32, (2, N, K), dtype=torch.int8, device="cuda", generator=g)
    ws = torch.rand((2, N), device="cuda", generator=g)
    p = r9k.pack_weight_i8(w)
    src = (2 * at + 1).int()                                                 # the second slot of each token
    off = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    want = torch.cat([((small[a:b].double() @ w[e].double().T).float() * s[at][a:b, None] * ws[e]).to(torch.bfloat16)
                      for e, (a, b) in enumerate(((0, 3), (3, 8)))])
    say("moe_gemm_i8 through an index", rows, K)
    assert torch.equal(r9k.moe_gemm_i8(q, s, off, p, ws, src=src, topk=2), want)
    say("gemm_i8", rows, K)
    c = r9k.gemm_i8(q, s, p[1], ws[1])
    assert torch.equal(c[at[3:]], want[3:]) and not torch.any(c[2:77])


def test_router_past_32_bits(r9k):
    """2.25e9 logits."""
    T, E, k = 1_100_001, 2048, 2
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=g)
    last = torch.randn((1000, E), device="cuda", generator=g).to(torch.bfloat16)
    x[-1000:] = last
    say("moe_balance_loss", T, E)
    loss, counts, psum = r9k.moe_balance_loss(x, ids)
    assert torch.equal(counts[:E].long(), torch.bincount(ids.flatten().long(), minlength=E)) and int(counts[E]) == T
    p, err = ref.probs(last.cpu())
    want, err = p.sum(0) + (T - 1000) / E, err.sum(0) + (T - 1000) / E * (E + 8) * ref.U
    # at most 256 parts of rows: 4298 of them added up in any order, then the parts
    assert torch.all((psum.cpu().to(ref.F64) - want).abs() <= err + (want + err) * (4298 + 256) * ref.U)
    say("moe_balance_loss_backward", T, E)
    gl = torch.tensor(float(T), device="cuda")
    gx = r9k.moe_balance_loss_backward(gl, x, counts, k)
    want, bad = ref.balance_grad(float(T), last[-3:].cpu(), counts.cpu(), k)
    assert torch.all((gx[-3:].cpu().to(ref.F64) - want).abs() <= ref.bf16_bound(want, bad))
    del x, gx
    gw, tw = torch.randn((T, k), device="cuda", generator=g), torch.rand((T, k), device="cuda", generator=g)
    say("moe_route_backward", T, E)
    gr = r9k.moe_route_backward(gw, ids, tw, E)
    tail = r9k.moe_route_backward(gw[-100:].clone(), ids[-100:].clone(), tw[-100:].clone(), E)
    assert torch.equal(gr[-100:], tail) and torch.count_nonzero(gr[T // 2]) <= k


def test_two_threads(r9k):
    """Calls of different shapes from two threads, each on a stream of its own."""
    shapes = [[(1, 4096, 1024), (48, 2048, 512), (200, 2048, 1024)], [(16, 2048, 512), (600, 1024, 2048), (3, 640, 272)]]
    work = []
    for t in range(2):
        calls = []
        for M, K, N in shapes[t]:
            w = weight((N,), K, M + t)
            a, p, ws = acts(M, K, M).cuda(), r9k.pack_weight_i8(w[0].cuda()), w[1].cuda()
            x, ids = torch.randn(M, 64, device="cuda"), torch.randint(0, 64, (M, 4), dtype=torch.int32, device="cuda")
            calls.append((a, p, ws, x, ids, r9k.gemm_i8_qa(a, p, ws), r9k.moe_balance_loss(x, ids)))
        work.append(calls)
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream() for _ in work]

    def go(t):
        try:
            with torch.cuda.stream(streams[t]):
                for i in range(30):
                    for a, p, ws, x, ids, c, bal in work[t]:
                        same = torch.equal(r9k.gemm_i8_qa(a, p, ws), c)
                        same &= all(torch.equal(u, v) for u, v in zip(r9k.moe_balance_loss(x, ids), bal))
                        if not same:
                            wrong.append((t, i, tuple(a.shape)))
        except Exception as e:  # noqa: BLE001 - a thread's error belongs to the test
            wrong.append(e)

    threads = [threading.Thread(target=go, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_streams_and_shared_workspaces(r9k):
    """Experts and the router's gradient on a side stream; graphs that were captured with one workspace, replayed in turn."""
    T, k, E, K, N = 90, 4, 16, 256, 96
    ids = routing(T, k, E, "rand", 1)
    src, pos, off = w4_ref.sort(ids, E)
    w = weight((E, N), K, 5)
    p, ws = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda()
    q, s = r9k.quant_i8(acts(T, K, 6).cuda())
    srcd, offd = torch.from_numpy(src).cuda(), torch.from_numpy(off).cuda()
    idsd, gw, tw = torch.from_numpy(ids).cuda(), torch.randn(T, k, device="cuda"), torch.rand(T, k, device="cuda")
    c, gr = r9k.moe_gemm_i8(q, s, offd, p, ws, src=srcd, topk=k), r9k.moe_route_backward(gw, idsd, tw, E)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = [r9k.moe_gemm_i8(q, s, offd, p, ws, src=srcd, topk=k, stream=side), r9k.moe_route_backward(gw, idsd, tw, E, stream=side),
           r9k.quant_i8(acts(T, K, 6).cuda(), stream=torch.cuda.current_stream())[0]]
    side.synchronize()
    assert torch.equal(out[0], c) and torch.equal(out[1], gr) and torch.equal(out[2], q)

    shapes = [(16, 14336, 1024), (48, 2048, 512), (200, 2048, 1024)]
    buf = torch.full((max(r9k.gemm_i8_workspace(*x) for x in shapes) + (1 << 20),), 0xFF, dtype=torch.uint8, device="cuda")
    graphs = []
    for M, K2, N2 in shapes:
        wd = weight((N2,), K2, M)
        a, pd, wsd = acts(M, K2, M).cuda(), r9k.pack_weight_i8(wd[0].cuda()), wd[1].cuda()
        want, o = r9k.gemm_i8_qa(a, pd, wsd), torch.empty((M, N2), dtype=torch.bfloat16, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r9k.gemm_i8_qa(a, pd, wsd, c=o, workspace=buf)
        graphs.append((g, o, want, (a, pd, wsd)))
    x, xi = torch.randn(3000, 60, device="cuda"), torch.randint(0, 60, (3000, 3), dtype=torch.int32, device="cuda")
    bal = r9k.moe_balance_loss(x, xi)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o = r9k.moe_balance_loss(x, xi, workspace=buf)
    for _ in range(3):
        for gi, oi, want, _keep in graphs:
            oi.zero_()
            gi.replay()
            g.replay()
            gi.replay()
        buf.fill_(0x5A)
        torch.cuda.synchronize()
        assert all(torch.equal(oi, want) for _, oi, want, _ in graphs) and all(torch.equal(u, v) for u, v in zip(o, bal))


def test_refusals_with_every_output_given(r9k):
    """The one-expression checks of calls with their output given let nothing through that the named ones refuse."""
    M, K, N = 4, 256, 32
    w = weight((N,), K, 1)
    p, ws, a = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda(), acts(M, K, 2).cuda()
    q, s = r9k.quant_i8(a)
    c = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    wide = torch.empty((M, 2 * N), dtype=torch.bfloat16, device="cuda")[:, ::2]
    for bad in (dict(c=wide), dict(c=c[:2]), dict(c=c.cpu()), dict(c=c.t()), dict(ws=ws[:16]), dict(ws=ws.cpu()), dict(ws=ws[None]),
                dict(p=p[:16]), dict(p=p.t()), dict(p=p.cpu()), dict(p=p[None]), dict(s=s[:2]), dict(s=s.cpu()), dict(q=q.t())):
        v = dict(q=q, s=s, p=p, ws=ws, c=c) | bad
        with pytest.raises(ValueError):
            r9k.gemm_i8(v["q"], v["s"], v["p"], v["ws"], c=v["c"])
        if "s" not in bad and "q" not in bad:
            with pytest.raises(ValueError):
                r9k.gemm_i8_qa(a, v["p"], v["ws"], c=v["c"])
    for bad in (dict(c=c.float()), dict(ws=ws.half()), dict(p=p.float()), dict(s=s.double()), dict(q=q.float())):
        v = dict(q=q, s=s, p=p, ws=ws, c=c) | bad
        with pytest.raises(TypeError):
            r9k.gemm_i8(v["q"], v["s"], v["p"], v["ws"], c=v["c"])
    with pytest.raises(ValueError):
        r9k.gemm_i8_qa(a.t(), p, ws, c=c)
    with pytest.raises(TypeError):
        r9k.gemm_i8_qa(a.float(), p, ws, c=c)
    with pytest.raises(r9k.R9kError):                                        # the output on an input
        r9k.gemm_i8_qa(a, p, ws, c=a.view(-1)[:M * N].view(M, N))
    assert torch.equal(r9k.gemm_i8(q, s, p, ws, c=c), r9k.gemm_i8(q, s, p, ws))
    gw, tw, ids = torch.randn(M, 2).cuda(), torch.rand(M, 2).cuda(), torch.zeros((M, 2), dtype=torch.int32).cuda()
    for args, err in (((gw, ids, tw[:2]), ValueError), ((gw, ids[:, :1], tw), ValueError), ((gw.t(), ids, tw), ValueError),
                      ((gw, ids.cpu(), tw), ValueError), ((gw, ids.long(), tw), TypeError), ((gw, ids, tw.half()), TypeError)):
        with pytest.raises(err):
            r9k.moe_route_backward(*args, 8)


def test_refusals_of_quantiser_and_experts_with_outputs_given(r9k):
    T, K, E, N = 6, 256, 3, 32
    x = acts(T, K, 1).cuda()
    q, s = r9k.quant_i8(x)
    for bad, err in ((dict(q=q[:2]), ValueError), (dict(q=q.t()), ValueError), (dict(q=q.cpu()), ValueError), (dict(q=q.float()), TypeError),
                     (dict(s=s[:2]), ValueError), (dict(s=s[:, None]), ValueError), (dict(s=s.half()), TypeError), (dict(x=x.t()), ValueError),
                     (dict(x=x.float()), TypeError)):
        v = dict(x=x, q=q, s=s) | bad
        with pytest.raises(err):
            r9k.quant_i8(v["x"], q=v["q"], s=v["s"])
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    assert r9k.quant_i8(x, q=q2, s=s2)[0] is q2 and torch.equal(q2, q) and torch.equal(s2, s)
    w = weight((E, N), K, 2)
    p, ws = r9k.pack_weight_i8(w[0].cuda()), w[1].cuda()
    off, src = torch.tensor([0, 2, 3, 6], dtype=torch.int32).cuda(), torch.tensor([3, 1, 0, 5, 4, 2], dtype=torch.int32).cuda()
    c = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    ok = dict(xq=q, xs=s, offsets=off, wp=p, ws=ws, src=src, c=c)
    for bad, err in ((dict(c=c[:2]), ValueError), (dict(c=c[:, :16]), ValueError), (dict(c=c.cpu()), ValueError), (dict(c=c.half()), TypeError),
                     (dict(xs=s[:2]), ValueError), (dict(xs=s.half()), TypeError), (dict(offsets=off[:3]), ValueError),
                     (dict(offsets=off.long()), TypeError), (dict(offsets=off.cpu()), ValueError), (dict(ws=ws[:2]), ValueError),
                     (dict(ws=ws.t()), ValueError), (dict(wp=p[:, :, :128].contiguous()), ValueError), (dict(wp=p[:2]), ValueError),
                     (dict(src=src.long()), TypeError), (dict(src=src.cpu()), ValueError), (dict(src=src[::2], c=c[:3]), ValueError),
                     (dict(xq=q.t()), ValueError), (dict(act="silu_mul"), ValueError)):
        with pytest.raises(err):
            r9k.moe_gemm_i8(**(ok | bad))
    assert torch.equal(r9k.moe_gemm_i8(**ok), r9k.moe_gemm_i8(**(ok | dict(c=None))))
    assert torch.equal(r9k.moe_gemm_i8(**(ok | dict(src=None))), r9k.moe_gemm_i8(**(ok | dict(c=None, src=None))))
