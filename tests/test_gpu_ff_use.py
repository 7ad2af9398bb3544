"""The feed-forward operators as they are used: large sizes, offsets past 32 bits, run together, under autograd, on
other streams, captured into graphs, and refused.  Tolerances: ff_ref.py."""
import numpy as np
import pytest

import ff_ref as ref

pytestmark = pytest.mark.gpu


def _randn(seed, shape, dt, scale=1.0):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(ref.torch_type(dt))


def _ok():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    torch.cuda.synchronize()
    st, word = tg.device_status()
    assert st == tg.Status.OK, hex(word)


def _some(n, seed, count=24):
    """Indices at both ends, around tile borders and at random."""
    rng = np.random.default_rng(seed)
    picks = {0, 1, n - 1, n - 2, 127, 128, 255, 256, n // 2} | {int(i) for i in rng.integers(0, n, size=count)}
    return np.array(sorted(i for i in picks if 0 <= i < n))


# ---------------------------------------------------------------------------
# Large sizes: several waves of tiles, the last one of half tiles or not
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K,dt,save", [(2048, 7680, 4096, "f16", False), (2000, 7681, 4104, "bf16", True),
                                           (2304, 8192, 2560, "bf16", False), (3001, 5003, 1021, "f16", True)])
def test_gated_large(M, N, K, dt, save):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, wg, wu = _randn(1, (M, K), dt), _randn(2, (N, K), dt, K ** -0.5), _randn(3, (N, K), dt, K ** -0.5)
    got = tg.gated(x, wg, wu, act="silu", save=save)
    got = got if save else (got,)
    _ok()
    rows, cols = _some(M, M), _some(N, N, 200)
    ri, ci = torch.from_numpy(rows).cuda(), torch.from_numpy(cols).cuda()
    outs, tols = ref.gated(ref.f64(x[ri]), ref.f64(wg[ci]), ref.f64(wu[ci]), "silu", dt)
    for t, o, tol in zip(got, outs, tols):
        ref.check(ref.f64(t[ri][:, ci]), o, tol, "gated")


@pytest.mark.parametrize("M,N,K", [(4096, 2048, 3848), (4096, 2048, 15360)])
def test_gated_backward_large(M, N, K):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    dt = "bf16"
    x, wg, wu = _randn(1, (M, K), dt), _randn(2, (N, K), dt, K ** -0.5), _randn(3, (N, K), dt, K ** -0.5)
    dh = _randn(4, (M, N), dt, 0.1)
    _, g, u = tg.gated(x, wg, wu, act="gelu", save=True)
    dx, dwg, dwu = tg.gated_backward(dh, x, wg, wu, g, u, act="gelu")
    _ok()
    rows, ks, ns = _some(M, 5), _some(K, 6, 100), _some(N, 7)
    ri, ki, ni = (torch.from_numpy(i).cuda() for i in (rows, ks, ns))
    outs, tols = ref.gated_backward(ref.f64(dh[ri]), ref.f64(x[ri][:, ki]), ref.f64(wg[:, ki]), ref.f64(wu[:, ki]), ref.f64(g[ri]),
                                    ref.f64(u[ri]), "gelu", dt)
    ref.check(ref.f64(dx[ri][:, ki]), outs[0], tols[0], "dX")
    outs, tols = ref.gated_backward(ref.f64(dh[:, ni]), ref.f64(x[:, ki]), ref.f64(wg[ni][:, ki]), ref.f64(wu[ni][:, ki]),
                                    ref.f64(g[:, ni]), ref.f64(u[:, ni]), "gelu", dt)
    ref.check(ref.f64(dwg[ni][:, ki]), outs[1], tols[1], "dWg")
    ref.check(ref.f64(dwu[ni][:, ki]), outs[2], tols[2], "dWu")


def _codes(seed, rows, K):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    full = torch.randint(-128, 128, (rows, (K + 15) // 16 * 16), generator=gen, device="cuda", dtype=torch.int8)
    return full[:, :K], torch.rand(rows, generator=gen, device="cuda") * 0.01 + 0.005


@pytest.mark.parametrize("M,N,K", [(2048, 15360, 8192), (8192, 5003, 1021), (200, 8192, 8192), (256, 1000, 7000)])
def test_gemm_i8_large(M, N, K):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    a, sa = _codes(1, M, K)
    w, sw = _codes(2, N, K)
    got = tg.gemm_i8(a, sa, w, sw, dtype=torch.bfloat16)
    _ok()
    ri, ci = (torch.from_numpy(_some(n, n, 100)).cuda() for n in (M, N))
    c, err = ref.i8_product(a[ri].cpu().numpy(), sa[ri].cpu().numpy(), w[ci].cpu().numpy(), sw[ci].cpu().numpy())
    ref.check(ref.f64(got[ri][:, ci]), c, err + ref.round_error(c, "bf16"), "C")


@pytest.mark.parametrize("M,N,K", [(4096, 4096, 8192), (3001, 5003, 1021), (256, 8192, 1024)])
def test_gated_i8_large(M, N, K):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    a, sa = _codes(1, M, K)
    (wg, sg), (wu, su) = _codes(2, N, K), _codes(3, N, K)
    sa = sa * 1e-3
    got = tg.gated_i8(a, sa, wg, sg, wu, su, act="gelu", dtype=torch.bfloat16)
    _ok()
    ri, ci = (torch.from_numpy(_some(n, n, 100)).cuda() for n in (M, N))
    rows = (a[ri].cpu().numpy(), sa[ri].cpu().numpy())
    g, dg = ref.i8_product(*rows, wg[ci].cpu().numpy(), sg[ci].cpu().numpy())
    u, du = ref.i8_product(*rows, wu[ci].cpu().numpy(), su[ci].cpu().numpy())
    outs, tols = ref.gate(g, u, dg, du, "gelu", "bf16")
    ref.check(ref.f64(got[ri][:, ci]), outs[0], tols[0], "H")


# ---------------------------------------------------------------------------
# Offsets past 2^31 elements
# ---------------------------------------------------------------------------

def test_offsets_past_32_bits_gated():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K, dt = 66000, 32776, 64, "bf16"
    assert M * N > 1 << 31
    x, wg, wu = _randn(1, (M, K), dt), _randn(2, (N, K), dt, 0.2), _randn(3, (N, K), dt, 0.2)
    h, g, u = tg.gated(x, wg, wu, save=True)
    dh = h  # any gradient will do
    dx, dwg, dwu = tg.gated_backward(dh, x, wg, wu, g, u)
    _ok()
    rows = np.unique(np.concatenate([_some(M, 1, 8), [M - 129, M - 128, (1 << 31) // N, (1 << 31) // N + 1]]))
    ri = torch.from_numpy(rows).cuda()
    outs, tols = ref.gated(ref.f64(x[ri]), ref.f64(wg), ref.f64(wu), "silu", dt)
    for name, t, o, tol in zip("HGU", (h, g, u), outs, tols):
        ref.check(ref.f64(t[ri]), o, tol, name)
    args = [ref.f64(t[ri]) for t in (dh, x)] + [ref.f64(wg), ref.f64(wu)] + [ref.f64(t[ri]) for t in (g, u)]
    outs, tols = ref.gated_backward(*args, "silu", dt)
    ref.check(ref.f64(dx[ri]), outs[0], tols[0], "dX")
    ni = torch.tensor([0, 1, 255, N - 1], device="cuda")
    args = [ref.f64(dh[:, ni]), ref.f64(x), ref.f64(wg[ni]), ref.f64(wu[ni]), ref.f64(g[:, ni]), ref.f64(u[:, ni])]
    outs, tols = ref.gated_backward(*args, "silu", dt)
    ref.check(ref.f64(dwg[ni]), outs[1], tols[1], "dWg")
    ref.check(ref.f64(dwu[ni]), outs[2], tols[2], "dWu")


def test_offsets_past_32_bits_i8():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, K, N = 66000, 32776, 136
    assert M * K > 1 << 31
    x = _randn(5, (M, K), "f16")
    q, s = tg.quantize_i8(x)
    _ok()
    rows = np.unique(np.concatenate([_some(M, 1, 8), [(1 << 31) // K, (1 << 31) // K + 1]]))
    ri = torch.from_numpy(rows).cuda()
    want_q, want_s = ref.quantize(ref.f64(x[ri]))
    assert np.array_equal(q[ri].cpu().numpy(), want_q) and np.array_equal(s[ri].cpu().numpy(), want_s)
    w, sw = _codes(2, N, K)
    got = tg.gemm_i8(q, s, w, sw * 1e-3)
    _ok()
    c, err = ref.i8_product(want_q, want_s, w.cpu().numpy(), (sw * 1e-3).cpu().numpy())
    ref.check(ref.f64(got[ri]), c, err + ref.round_error(c, "f16"), "C")


# ---------------------------------------------------------------------------
# Run together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 37, 300])
def test_served_block(M):
    """Quantize, gated block, quantize, down projection with bias: the block as it is served, in 8 bits."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    K, N, dt = 264, 520, "bf16"
    x = _randn(1, (2, M, K), dt)
    weights = [_randn(i, s, dt, s[1] ** -0.5) for i, s in ((2, (N, K)), (3, (N, K)), (4, (K, N)))]
    (wg, sg), (wu, su), (wd, sd) = (tg.quantize_i8(w) for w in weights)
    bias = _randn(5, (K,), dt)
    q, s = tg.quantize_i8(x)
    h = tg.gated_i8(q, s, wg, sg, wu, su, dtype=torch.bfloat16)
    q2, s2 = tg.quantize_i8(h)
    y = tg.gemm_i8(q2, s2, wd, sd, bias=bias, dtype=torch.bfloat16)
    _ok()
    assert q.shape == x.shape and s.shape == (2, M) and h.shape == (2, M, N) and y.shape == x.shape

    def flat(t):
        return t.cpu().numpy().reshape(-1, t.shape[-1])

    qr, sr = ref.quantize(ref.f64(x).reshape(-1, K))
    assert np.array_equal(flat(q), qr) and np.array_equal(s.cpu().numpy().ravel(), sr)
    g, dg = ref.i8_product(qr, sr, wg.cpu().numpy(), sg.cpu().numpy())
    u, du = ref.i8_product(qr, sr, wu.cpu().numpy(), su.cpu().numpy())
    outs, tols = ref.gate(g, u, dg, du, "silu", dt)
    ref.check(ref.f64(h).reshape(-1, N), outs[0], tols[0], "H")
    qh, sh = ref.quantize(ref.f64(h).reshape(-1, N))
    assert np.array_equal(flat(q2), qh) and np.array_equal(s2.cpu().numpy().ravel(), sh)
    c, err = ref.i8_product(qh, sh, wd.cpu().numpy(), sd.cpu().numpy())
    c = c + ref.f64(bias)
    ref.check(ref.f64(y).reshape(-1, K), c, err + np.abs(c) * 2.0 ** -24 + ref.round_error(c, dt), "Y")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_autograd_block(act):
    """A block of three weights under autograd: gradients of the gated half against the formulas, and of the whole
    against difference quotients of its 64-bit form."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K, dt = 70, 136, 72, "f16"
    x = _randn(1, (2, M // 2, K), dt).requires_grad_()
    w = _randn(2, (2 * N, K), dt, K ** -0.5).requires_grad_()  # gate and up in one weight
    dh = _randn(4, (2, M // 2, N), dt, 0.5)
    h = tg.gated_block(x, w[:N], w[N:], act=act)
    h.backward(dh)
    _ok()
    x2, w2, dh2 = ref.f64(x).reshape(M, K), ref.f64(w), ref.f64(dh).reshape(M, N)
    outs, tols = ref.gated(x2, w2[:N], w2[N:], act, dt)
    ref.check(ref.f64(h).reshape(M, N), outs[0], tols[0], "H")
    _, g, u = tg.gated(x.detach(), w.detach()[:N], w.detach()[N:], act=act, save=True)
    want, wtol = ref.gated_backward(dh2, x2, w2[:N], w2[N:], ref.f64(g).reshape(M, N), ref.f64(u).reshape(M, N), act, dt)
    ref.check(ref.f64(x.grad).reshape(M, K), want[0], wtol[0], "dX")
    ref.check(ref.f64(w.grad)[:N], want[1], wtol[1], "dWg")
    ref.check(ref.f64(w.grad)[N:], want[2], wtol[2], "dWu")


def test_gradient_against_differences():
    """<dX, v> against the difference quotient of <H, dH> along v, both taken with the library's calls.

    The quotient of the library's H differs from that of the 64-bit H by at most the sum of H's tolerances at
    both ends over the step; the 64-bit quotient differs from the derivative by what its halved step shows
    (central differences: the error falls to a quarter, so it is at most 4/3 of the change; 2 is taken)."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K, dt, act = 40, 64, 24, "f16", "gelu"
    x, wg, wu, dh = _randn(1, (M, K), dt), _randn(2, (N, K), dt, 0.2), _randn(3, (N, K), dt, 0.2), _randn(4, (M, N), dt)
    v = (torch.randint(0, 2, (M, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)) * 2 - 1).to(x.dtype)
    x = (x * 64).round() / 64  # so that x +- v / 16 is exact
    step = 1 / 16
    plus, minus = (x + step * v), (x - step * v)
    assert torch.equal(plus.double() - x.double(), step * v.double())
    _, g, u = tg.gated(x, wg, wu, act=act, save=True)
    dx, _, _ = tg.gated_backward(dh, x, wg, wu, g, u, act=act, needs=(True, False, False))
    ends = [tg.gated(t, wg, wu, act=act) for t in (plus, minus)]
    _ok()
    dh64, v64 = ref.f64(dh), ref.f64(v)
    quotient = float(((ref.f64(ends[0]) - ref.f64(ends[1])) * dh64).sum() / (2 * step))
    sides = [ref.gated(ref.f64(t), ref.f64(wg), ref.f64(wu), act, dt) for t in (plus, minus)]
    noise = float(sum((tol[0] * np.abs(dh64)).sum() for _, tol in sides) / (2 * step))

    def exact_quotient(e):
        a, b = (ref.gated(ref.f64(x) + d * e * v64, ref.f64(wg), ref.f64(wu), act, dt)[0][0] for d in (1, -1))
        return float(((a - b) * dh64).sum() / (2 * e))

    curve = 2 * abs(exact_quotient(step) - exact_quotient(step / 2))
    _, tol_dx = ref.gated_backward(dh64, ref.f64(x), ref.f64(wg), ref.f64(wu), ref.f64(g), ref.f64(u), act, dt)
    # The stored G and U are rounded: the formula at them is off by half a step of each, times the second
    # derivatives, at most 1.2 in all, carried through the weights.
    stored = ((1.2 * np.abs(dh64) * (np.abs(ref.f64(u)) * np.abs(ref.f64(g)) + np.abs(ref.f64(u)) + np.abs(ref.f64(g))) * ref.HALF[dt])
              @ (np.abs(ref.f64(wg)) + np.abs(ref.f64(wu)))).sum()
    slope = float((ref.f64(dx) * v64).sum())
    assert abs(slope - quotient) <= noise + curve + float(tol_dx[0].sum()) + float(stored), (slope, quotient, noise, curve)
    assert abs(quotient) > 10 * curve  # the direction says something


def test_autograd_shapes_of_gradients():
    """An expanded gradient, gradients for some leaves only, inference without storing, rows with gaps."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K, dt = 33, 40, 24, "bf16"
    x = _randn(1, (M, 2 * K), dt)[:, :K]
    wg, wu = _randn(2, (N, K), dt).requires_grad_(), _randn(3, (N, K), dt)
    h = tg.gated_block(x, wg, wu)
    h.sum().backward()  # an expanded gradient of stride 0
    _ok()
    ones = torch.ones((M, N), dtype=x.dtype, device="cuda")
    _, g, u = tg.gated(x, wg.detach(), wu, save=True)
    want = tg.gated_backward(ones, x, wg.detach(), wu, g, u, needs=(False, True, False))[1]
    assert torch.equal(wg.grad, want) and wu.grad is None and x.grad is None
    with torch.no_grad():
        assert torch.equal(tg.gated_block(x, wg, wu), h)
    assert tg.gated_block(x, wg.detach(), wu).grad_fn is None
    # A column-major x and an odd-strided weight are copied or taken as they are.
    xt = _randn(4, (K, M), dt).t().requires_grad_()
    h = tg.gated_block(xt, wg, wu)
    h.backward(ones)
    _ok()
    assert torch.equal(h, tg.gated(xt.detach().contiguous(), wg.detach(), wu)) and xt.grad.shape == xt.shape


# ---------------------------------------------------------------------------
# Streams, graphs, repeats
# ---------------------------------------------------------------------------

def _all_operators(seed=1, M=150, N=131, K=265):
    """Calls of every operator on fixed inputs, as (inputs, function of a stream -> outputs)."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    dt = "f16"  # odd sizes: padded copies and unaligned results too
    x, wg, wu, dh = (_randn(seed + i, s, dt, sc) for i, (s, sc) in
                     enumerate((((M, K), 1.0), ((N, K), 0.06), ((N, K), 0.06), ((M, N), 0.1))))
    qg, sg = tg.quantize_i8(wg)
    qu, su = tg.quantize_i8(wu)

    def run(stream=None):
        h, g, u = tg.gated(x, wg, wu, save=True, stream=stream)
        grads = tg.gated_backward(dh, x, wg, wu, g, u, stream=stream)
        q, s = tg.quantize_i8(x, stream=stream)
        return (h, g, u, *grads, q, s, tg.gemm_i8(q, s, qg, sg, stream=stream),
                tg.gated_i8(q, s, qg, sg, qu, su, dtype=torch.bfloat16, stream=stream))

    return (x, dh), run


def test_repeats_are_equal():
    import torch
    for M in (9, 150, 700):
        _, run = _all_operators(M=M)
        first = run()
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, run()))
    _ok()


def test_another_stream():
    """A call on a stream runs there: it waits for what the stream holds, not for the current stream."""
    import torch
    (x, _), run = _all_operators()
    want = run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = x.clone()
    x.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
        x.copy_(keep)  # on the side stream, after a while
    got = run(stream=side)  # from the main stream's context: ordered after the copy
    side.synchronize()
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_two_streams_at_once():
    import torch
    (_, run_a), (_, run_b) = _all_operators(seed=1), _all_operators(seed=50, M=301)
    want_a, want_b = run_a(), run_b()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(run_a(stream=s1), run_b(stream=s2)) for _ in range(10)]
    torch.cuda.synchronize()
    _ok()
    for a, b in got:
        assert all(torch.equal(p, q) for p, q in zip(want_a, a)) and all(torch.equal(p, q) for p, q in zip(want_b, b))


def test_graphs():
    """Captured calls replay on new inputs; two graphs that share a memory pool replay one after the other."""
    import torch
    (x, dh), run = _all_operators()
    (x2, _), run2 = _all_operators(seed=50, M=301)
    run(), run2()
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        out1 = run()
    with torch.cuda.graph(g2, pool=g1.pool()):
        out2 = run2()
    for seed in (7, 8):
        x.copy_(_randn(seed, x.shape, "f16"))
        dh.copy_(_randn(seed + 10, dh.shape, "f16", 0.1))
        x2.copy_(_randn(seed + 20, x2.shape, "f16"))
        want1, want2 = run(), run2()
        g1.replay()
        first = [t.clone() for t in out1]
        g2.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want1, first))
        assert all(torch.equal(a, b) for a, b in zip(want2, out2))
    _ok()
    del g1, g2


def test_long_sums_in_streams_and_graphs():
    """Products whose K is split over clusters: two streams at once, one captured, repeated."""
    import torch
    (x, dh), run_a = _all_operators(seed=1, M=300, N=136, K=2104)
    (y, _), run_b = _all_operators(seed=50, M=2050, N=200, K=133)
    want_a, want_b = run_a(), run_b()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(run_a(stream=s1), run_b(stream=s2)) for _ in range(10)]
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(p, q) for p, q in zip(want_a, a)) and all(torch.equal(p, q) for p, q in zip(want_b, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out_a, out_b = run_a(), run_b()
    for seed in (7, 8):
        x.copy_(_randn(seed, x.shape, "f16"))
        dh.copy_(_randn(seed + 10, dh.shape, "f16", 0.1))
        y.copy_(_randn(seed + 20, y.shape, "f16"))
        want_a, want_b = run_a(), run_b()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want_a, out_a))
        assert all(torch.equal(p, q) for p, q in zip(want_b, out_b))
    _ok()
    del graph


def test_given_workspace():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K = 20, 41, 33
    x, wg, wu, dh = (_randn(i, s, "f16") for i, s in enumerate(((M, K), (N, K), (N, K), (M, N))))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    h, g, u = tg.gated(x, wg, wu, save=True, workspace=ws)
    grads = tg.gated_backward(dh, x, wg, wu, g, u, workspace=ws)
    _ok()
    assert torch.equal(h, tg.gated(x, wg, wu))
    assert all(torch.equal(a, b) for a, b in zip(grads, tg.gated_backward(dh, x, wg, wu, g, u)))
    for bad in (None, torch.empty(256, dtype=torch.uint8, device="cuda")):
        with pytest.raises(tg.TGError):
            tg.gated(x, wg, wu, workspace=bad)
        with pytest.raises(tg.TGError):
            tg.gated_backward(dh, x, wg, wu, g, u, workspace=bad)
    for bad in ("none", torch.empty(1 << 20, dtype=torch.int8, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            tg.gated(x, wg, wu, workspace=bad)


# ---------------------------------------------------------------------------
# Refusals of the torch calls
# ---------------------------------------------------------------------------

def test_refusals():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    f, dev = torch.float16, "cuda"
    x, w, h = torch.zeros((4, 16), dtype=f, device=dev), torch.zeros((8, 16), dtype=f, device=dev), torch.zeros((4, 8), dtype=f, device=dev)
    cases = [
        (TypeError, lambda: tg.gated(x.float(), w.float(), w.float())),
        (TypeError, lambda: tg.gated(x, w.bfloat16(), w)),
        (ValueError, lambda: tg.gated(x, w, w[:7])),
        (ValueError, lambda: tg.gated(x, w[:, :8], w)),
        (ValueError, lambda: tg.gated(x, w, w.cpu())),
        (ValueError, lambda: tg.gated(x, w, w, act="swish")),
        (ValueError, lambda: tg.gated(x.t(), w[:, :4], w[:, :4])),
        (ValueError, lambda: tg.gated(x[:1].expand(4, 16), w, w)),        # rows on top of each other
        (ValueError, lambda: tg.gated(x.view(2, 2, 16).transpose(0, 1), w, w)),
        (ValueError, lambda: tg.gated(x, w, w, out=h[:3])),
        (TypeError, lambda: tg.gated(x, w, w, out=h.bfloat16())),
        (tg.TGError, lambda: tg.gated(x, w, w, out=x[:, :8])),            # the result on its input
        (ValueError, lambda: tg.gated_backward(h[:3], x, w, w, h, h)),
        (TypeError, lambda: tg.gated_backward(h, x, w, w, h.bfloat16(), h)),
        (ValueError, lambda: tg.gated_backward(h, x, w, w, h.cpu(), h)),
        (TypeError, lambda: tg.quantize_i8(x.float())),
        (TypeError, lambda: tg.quantize_i8(x, out=torch.zeros((4, 16), dtype=torch.uint8, device=dev))),
        (ValueError, lambda: tg.quantize_i8(x, scales=torch.zeros(3, device=dev))),
        (ValueError, lambda: tg.quantize_i8(torch.zeros((), dtype=f, device=dev))),
    ]
    q, s = tg.quantize_i8(x)
    qw, sw = tg.quantize_i8(w)
    cases += [
        (TypeError, lambda: tg.gemm_i8(x, s, qw, sw)),
        (TypeError, lambda: tg.gemm_i8(q, s.double(), qw, sw)),
        (ValueError, lambda: tg.gemm_i8(q, s[:3], qw, sw)),
        (TypeError, lambda: tg.gemm_i8(q, s, qw, sw, dtype=torch.float32)),
        (TypeError, lambda: tg.gemm_i8(q, s, qw, sw, bias=torch.zeros(8, device=dev))),
        (ValueError, lambda: tg.gemm_i8(q, s, qw, sw, bias=torch.zeros(7, dtype=f, device=dev))),
        (tg.TGError, lambda: tg.gemm_i8(q[:, :15].contiguous(), s, qw[:, :15].contiguous(), sw)),  # rows off 16 bytes
        (ValueError, lambda: tg.gated_i8(q, s, qw, sw, qw[:4], sw)),
        (ValueError, lambda: tg.gated_i8(q, s, qw, sw, qw, sw, act="tanh")),
        (TypeError, lambda: tg.gated_i8(q, s, qw, sw, qw, sw, dtype=torch.bfloat16, out=h)),
    ]
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            pytest.fail(f"case {i} was taken")
    _ok()


def test_one_dimension():
    """A single row without a row dimension."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, wg, wu, dh = _randn(1, (40,), "f16"), _randn(2, (24, 40), "f16"), _randn(3, (24, 40), "f16"), _randn(4, (24,), "f16")
    h, g, u = tg.gated(x, wg, wu, save=True)
    dx, dwg, dwu = tg.gated_backward(dh, x, wg, wu, g, u)
    q, s = tg.quantize_i8(x)
    qw, sw = tg.quantize_i8(wg)
    y = tg.gemm_i8(q, s, qw, sw)
    z = tg.gated_i8(q, s, qw, sw, qw, sw)
    _ok()
    assert h.shape == g.shape == u.shape == y.shape == z.shape == (24,) and dx.shape == q.shape == (40,) and s.shape == ()
    two = tg.gated(x[None], wg, wu, save=True)
    assert all(torch.equal(a, b[0]) for a, b in zip((h, g, u), two))
    grads = tg.gated_backward(dh[None], x[None], wg, wu, two[1], two[2])
    assert torch.equal(dx, grads[0][0]) and torch.equal(dwg, grads[1]) and torch.equal(dwu, grads[2])
    q2, s2 = tg.quantize_i8(x[None])
    assert torch.equal(q, q2[0]) and s == s2[0] and torch.equal(y, tg.gemm_i8(q2, s2, qw, sw)[0])


FIRST_CALL = """
import torch
x, w, dh = (torch.randn(s, device="cuda").half() for s in ((20, 40), (24, 40), (20, 24)))
a = torch.randint(-127, 128, (200, 48), device="cuda", dtype=torch.int8)
s = torch.rand(200, device="cuda")
torch.cuda.synchronize()
import tiled_dense_gemm_fp16_b200 as tg
graph = torch.cuda.CUDAGraph()

def run():
    h, g, u = tg.gated(x, w, w, save=True)
    q, qs = tg.quantize_i8(x)
    return (h, *tg.gated_backward(dh, x, w, w, g, u), q, qs, tg.gemm_i8(a, s, a, s), tg.gated_i8(a, s, a, s, a, s))

with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(out, run()))
assert tg.device_status()[0] == tg.Status.OK
del graph
print("same")
"""


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: nothing they set up is refused during a capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and "same" in done.stdout, done.stderr[-2000:]


def test_far_gates_in_the_gradient():
    """Gates past the type's range, stored as infinities, give the limits' gradients; a closed gate gives 0 whatever U is."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    inf = float("inf")
    g = torch.tensor([[-inf, inf, -60000.0, 60000.0, -inf, 0.0, -200.0, 300.0]] * 3, device="cuda").half()
    u = torch.tensor([[2.0, 3.0, inf, 4.0, inf, 1.0, -inf, 5.0]] * 3, device="cuda").half()
    dh = torch.full((3, 8), 0.5, device="cuda").half()
    x, w = torch.eye(3, 8, device="cuda").half(), torch.eye(8, device="cuda").half()
    half = {"silu": 0.5, "gelu": 0.5, "relu": 0.0}
    for act in ("silu", "gelu", "relu"):
        dx, dwg, dwu = tg.gated_backward(dh, x, w, torch.zeros_like(w), g, u, act=act)
        _ok()
        want_dg = torch.tensor([0.0, 1.5, 0.0, 2.0, 0.0, 0.5 * half[act], 0.0, 2.5])
        assert torch.equal(dwg[:, 0].float().cpu(), want_dg), act           # x is the identity: dWg holds dG
        # dU of the infinite gate is an infinity, and dWu's sum holds it times the identity's zeros.
        want_du = torch.tensor([0.0, float("nan"), 0.0, 30000.0, 0.0, 0.0, 0.0, 150.0])
        assert torch.equal(dwu[:, 0].float().cpu().nan_to_num(-1), want_du.nan_to_num(-1)), act


def test_gaps_between_rows_are_not_read():
    """NaN between the rows of every operand reaches no result."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K = 70, 72, 40

    def spaced(t):
        wide = torch.full((t.shape[0], t.shape[1] + 24), float("nan"), dtype=t.dtype, device="cuda")
        wide[:, :t.shape[1]] = t
        return wide[:, :t.shape[1]]

    for m in (M, 400):
        x, wg, wu, dh = (_randn(i, s, "bf16") for i, s in enumerate(((m, K), (N, K), (N, K), (m, N))))
        want = tg.gated(x, wg, wu, save=True)
        got = tg.gated(spaced(x), spaced(wg), spaced(wu), save=True)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        want_g = tg.gated_backward(dh, x, wg, wu, *want[1:])
        got_g = tg.gated_backward(spaced(dh), spaced(x), spaced(wg), spaced(wu), spaced(want[1]), spaced(want[2]))
        assert all(torch.equal(a, b) for a, b in zip(want_g, got_g))
        assert all(torch.equal(a, b) for a, b in zip(tg.quantize_i8(x), tg.quantize_i8(spaced(x))))
    _ok()


def test_one_weight_twice():
    """The same leaf as gate and up: its gradient is the sum of both."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, dh = _randn(1, (50, 40), "bf16"), _randn(2, (24, 40), "bf16", 0.2).requires_grad_(), _randn(3, (50, 24), "bf16")
    tg.gated_block(x, w, w).backward(dh)
    _ok()
    d = w.detach()
    _, g, u = tg.gated(x, d, d, save=True)
    _, dwg, dwu = tg.gated_backward(dh, x, d, d, g, u)
    assert torch.equal(w.grad, dwg + dwu)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (2, 1, 1), (1, 2, 3), (129, 1, 1), (300, 1, 2), (2, 3, 100000), (260, 8, 70000),
                                   (1, 4300001, 8), (2000003, 9, 8), (300, 600000, 8)])
def test_smallest_and_longest(M, N, K):
    """One element, one row, very long sums, more panels than a grid holds, very many rows or columns."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    dt = "bf16"
    x, wg, wu = _randn(1, (M, K), dt), _randn(2, (N, K), dt, K ** -0.5), _randn(3, (N, K), dt, K ** -0.5)
    h, g, u = tg.gated(x, wg, wu, save=True)
    dh = _randn(4, (M, N), dt)
    dx, dwg, dwu = tg.gated_backward(dh, x, wg, wu, g, u)
    q, s = tg.quantize_i8(x)
    (qg, sg), (qu, su) = tg.quantize_i8(wg), tg.quantize_i8(wu)
    h8, c8 = tg.gated_i8(q, s, qg, sg, qu, su), tg.gemm_i8(q, s, qg, sg)
    _ok()
    ri, ci, ki = (torch.from_numpy(_some(n, n)).cuda() for n in (M, N, K))
    outs, tols = ref.gated(ref.f64(x[ri]), ref.f64(wg[ci]), ref.f64(wu[ci]), "silu", dt)
    for t, o, tol in zip((h, g, u), outs, tols):
        ref.check(ref.f64(t[ri][:, ci]), o, tol, "gated")
    args = [ref.f64(t) for t in (dh[ri], x[ri][:, ki], wg[:, ki], wu[:, ki], g[ri], u[ri])]
    outs, tols = ref.gated_backward(*args, "silu", dt)
    ref.check(ref.f64(dx[ri][:, ki]), outs[0], tols[0], "dX")
    args = [ref.f64(t) for t in (dh[:, ci], x[:, ki], wg[ci][:, ki], wu[ci][:, ki], g[:, ci], u[:, ci])]
    outs, tols = ref.gated_backward(*args, "silu", dt)
    ref.check(ref.f64(dwg[ci][:, ki]), outs[1], tols[1], "dWg")
    ref.check(ref.f64(dwu[ci][:, ki]), outs[2], tols[2], "dWu")
    want_q, want_s = ref.quantize(ref.f64(x[ri]))
    assert np.array_equal(q[ri].cpu().numpy(), want_q) and np.array_equal(s[ri].cpu().numpy(), want_s)
    c, err = ref.i8_product(want_q, want_s, qg[ci].cpu().numpy(), sg[ci].cpu().numpy())
    v, verr = ref.i8_product(want_q, want_s, qu[ci].cpu().numpy(), su[ci].cpu().numpy())
    ref.check(ref.f64(c8[ri][:, ci]), c, err + ref.round_error(c, "f16"), "C")
    outs, tols = ref.gate(c, v, err, verr, "silu", "f16")
    ref.check(ref.f64(h8[ri][:, ci]), outs[0], tols[0], "H")


def test_two_host_threads():
    """Calls from two host threads, each on a stream of its own."""
    import threading

    import torch
    pairs = [_all_operators(seed=1), _all_operators(seed=50, M=301)]
    want = [run() for _, run in pairs]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[i] = pairs[i][1]()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _ok()
    assert not errors
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_results_given_count_as_written():
    """A given result that another operator saved for its backward pass: that pass refuses the changed values."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w = (torch.randn((n, 64), device="cuda").half() for n in (4, 32))
    out = torch.ones((4, 32), dtype=torch.float16, device="cuda")
    leaf = torch.ones((4, 32), dtype=torch.float16, device="cuda", requires_grad=True)
    loss = (leaf * out).sum()
    assert tg.gated(x, w, w, out=out) is out
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    codes, scales = torch.empty((4, 64), dtype=torch.int8, device="cuda"), torch.empty(4, device="cuda")
    before = codes._version, scales._version
    q, s = tg.quantize_i8(x, out=codes, scales=scales)
    assert q is codes and s is scales and codes._version > before[0] and scales._version > before[1]
    qw, sw = tg.quantize_i8(w)
    before = out._version
    tg.gemm_i8(q, s, qw, sw, out=out)
    tg.gated_i8(q, s, qw, sw, qw, sw, out=out)
    assert out._version == before + 2
    with torch.inference_mode():
        mine = torch.empty((4, 32), dtype=torch.float16, device="cuda")
    assert tg.gated(x, w, w, out=mine) is mine
    _ok()


def test_another_device():
    """Tensors of a device that is not the current one: the call runs there, on that device's stream."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    if torch.cuda.device_count() < 2:
        pytest.skip("needs two GPUs")
    x, wg, wu, dh = (_randn(i, s, "f16", 0.1) for i, s in enumerate(((40, 72), (24, 72), (24, 72), (40, 24))))

    def run(*ts):
        h, g, u = tg.gated(*ts[:3], save=True)
        q, s = tg.quantize_i8(ts[0])
        qw, sw = tg.quantize_i8(ts[1])
        return (h, g, u, *tg.gated_backward(ts[3], *ts[:3], g, u), q, s, tg.gemm_i8(q, s, qw, sw),
                tg.gated_i8(q, s, qw, sw, qw, sw))

    want = run(x, wg, wu, dh)
    with torch.cuda.device(0):
        got = run(*(t.to("cuda:1") for t in (x, wg, wu, dh)))
        assert torch.cuda.current_device() == 0
    torch.cuda.synchronize(1)
    assert all(b.device.index == 1 and torch.equal(a, b.to(a.device)) for a, b in zip(want, got))
    with pytest.raises(ValueError):
        tg.gated(x, wg.to("cuda:1"), wu)
