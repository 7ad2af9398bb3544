"""The feed-forward operators at the edges of their ranges and in uses that cross: overflowed projections, far gates,
results between the rows of other matrices, row blocks of every height, captured training steps.  Tolerances: ff_ref.py."""
import numpy as np
import pytest

import ff_ref as ref

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


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


# ---------------------------------------------------------------------------
# Gradients at projections that overflowed when they were stored
# ---------------------------------------------------------------------------

def _row_gradients(dh, g, u, act, dt):
    """dG and dU of one row: with X = 1 they are the columns of dWg and dWu."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    t = ref.torch_type(dt)
    dh, g, u = (torch.tensor([v], device="cuda").to(t) for v in (dh, g, u))
    n = g.shape[1]
    x, w = torch.ones((1, 1), dtype=t, device="cuda"), torch.ones((n, 1), dtype=t, device="cuda")
    dx, dwg, dwu = tg.gated_backward(dh, x, w, w, g, u, act=act)
    _ok()
    return dx.item(), dwg[:, 0].tolist(), dwu[:, 0].tolist()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_no_gradient_at_overflowed_projections(act, dt):
    """A token without a gradient (padded, masked) has none through stored infinities either; a NaN stays one."""
    for zero in (0.0, -0.0):
        g, u = [INF, 1.0, -INF, INF, 2.0, -INF], [2.0, INF, 3.0, -INF, -INF, INF]
        dx, dg, du = _row_gradients([zero] * 6, g, u, act, dt)
        assert dx == 0 and not any(dg) and not any(du), (dx, dg, du)
        _, dg, du = _row_gradients([zero] * 2, [2.0, NAN], [NAN, 1.0], act, dt)
        assert np.isnan(dg[0]) and du[0] == 0
        assert act == "relu" or (np.isnan(dg[1]) and np.isnan(du[1]))  # relu: a gate that is not > 0 is closed


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_closed_gates_hide_no_gradient(act, dt):
    """A closed gate gives dG = 0 whatever U is; dH that is not finite shows in dG and in dU."""
    closed = [-INF] * 6
    dh, u = [NAN, INF, -INF, 0.5, 0.5, 0.5], [1.0, 1.0, 0.0, INF, NAN, 7.0]
    _, dg, du = _row_gradients(dh, closed, u, act, dt)
    assert np.isnan(dg[:3]).all() and np.isnan(du[:3]).all(), (dg, du)
    assert not any(dg[3:]) and not any(du[3:]), (dg, du)


# ---------------------------------------------------------------------------
# Far gates: logistic values down to fp32's last normal reciprocals
# ---------------------------------------------------------------------------

# silu's logistic value falls to 2^-128 at g = -88.7, gelu's at g = -10.06: bf16 results times a large U are far from zero.
FAR = {"silu": [-60.0, -80.0, -86.5, -87.0, -87.5, -88.0, -88.5, -40.0], "gelu": [-8.0, -9.0, -9.5, -9.75, -10.0, -10.0625, -5.0, -7.0]}
# The exponent z log2 e, up to 128, carries at most 3.5 roundings of 2^-24 relative (gelu: the square, the constants, the
# polynomial, and half a one of the last step): 3.5 * 2^-24 * 128 ln 2 = 2^-15.7 relative to the logistic value.
FAR_ERROR = 2.0 ** -15


@pytest.mark.parametrize("M", [2, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_gates(act, M):
    """H, dWg and dWu where the gate's logistic value is next to fp32's end but what it multiplies is large."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x = torch.zeros((M, 8), dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1
    wg, wu = torch.zeros((2, 8, 8), dtype=torch.bfloat16, device="cuda")
    wg[:, 0] = torch.tensor(FAR[act], device="cuda")
    wu[:, 0] = 2.0 ** 90
    h, g, u = tg.gated(x, wg, wu, act=act, save=True)
    dh = torch.zeros((M, 8), dtype=torch.bfloat16, device="cuda")
    dh[1] = 2.0 ** 20
    dx, dwg, dwu = tg.gated_backward(dh, x, wg, wu, g, u, act=act)
    _ok()
    g64, u64 = ref.f64(g), ref.f64(u)
    assert np.array_equal(g64[0], np.array(FAR[act])) and np.all(u64 == 2.0 ** 90)
    a, s = ref.act(g64, act)
    tol = FAR_ERROR + ref.HALF["bf16"]
    ref.check(ref.f64(h), a * u64, tol * np.abs(a * u64), "H")
    # The slope p + g p (1 - p) z' loses up to the size of its larger term.
    p = np.abs(a / g64)
    dg, du = ref.f64(dh) * u64 * s, ref.f64(dh) * a
    err_g = np.abs(ref.f64(dh) * u64) * (np.abs(s) + 2 * p) * FAR_ERROR + ref.HALF["bf16"] * np.abs(dg)
    ref.check(ref.f64(dwg)[:, 0], dg[1], 1.01 * err_g[1] + ref.round_error(dg[1], "bf16"), "dWg")
    ref.check(ref.f64(dwu)[:, 0], du[1], (tol + 2 * ref.HALF["bf16"]) * np.abs(du[1]) + ref.TINY["bf16"], "dWu")


@pytest.mark.parametrize("M", [2, 300])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_gates_i8(act, M):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    a = torch.zeros((M, 16), dtype=torch.int8, device="cuda")
    a[:, 0] = 1
    wg, wu = torch.zeros((2, 8, 16), dtype=torch.int8, device="cuda")
    wg[:, 0], wu[:, 0] = -1, 1
    sa, sg = torch.ones(M, device="cuda"), -torch.tensor(FAR[act], device="cuda")
    su = torch.full((8,), 2.0 ** 90, device="cuda")
    h = tg.gated_i8(a, sa, wg, sg, wu, su, act=act, dtype=torch.bfloat16)
    _ok()
    want = np.broadcast_to(ref.act(np.array(FAR[act]), act)[0] * 2.0 ** 90, (M, 8))
    ref.check(ref.f64(h), want, (FAR_ERROR + ref.HALF["bf16"]) * np.abs(want), "H")


# ---------------------------------------------------------------------------
# Results in the gaps between the rows of other matrices
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(20, 136, 72), (20, 41, 33), (300, 136, 72), (300, 261, 129), (700, 264, 130)])
def test_results_beside_inputs(M, N, K):
    """X, H, G and U as column ranges of one buffer, and dX, dWg and dWu beside X, Wg and Wu: equal to results of their
    own, the inputs unchanged."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    wide = K + 3 * N
    buf = _randn(1, (M, wide), "f16")
    weights = _randn(2, (N, 4 * K), "f16", K ** -0.5)  # Wg, dWg, Wu, dWu
    dx_wide = torch.zeros((M, 2 * K), dtype=torch.float16, device="cuda")
    x, h, g, u = buf[:, :K], *(buf[:, K + i * N:K + (i + 1) * N] for i in range(3))
    wg, dwg, wu, dwu = (weights[:, i * K:(i + 1) * K] for i in range(4))
    keep = [t.clone() for t in (x, wg, wu)]
    dh = _randn(3, (M, N), "f16", 0.1)
    want = tg.gated(x, wg, wu, act="gelu", save=True)
    want_grads = tg.gated_backward(dh, x, wg, wu, *want[1:], act="gelu")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    opts = tg.gated_options(act=tg.ACT_GELU, ldx=wide, ldwg=4 * K, ldwu=4 * K, ldh=wide, ldg=wide, ldu=wide)
    ptr = [t.data_ptr() for t in (x, wg, wu, h, g, u)]
    assert tg.gated_raw(*ptr, M, N, K, opts, stream, ws.data_ptr(), ws.numel()) == tg.Status.OK
    _ok()
    for name, got, t in zip("HGU", (h, g, u), want):
        assert torch.equal(got, t), name

    # dX beside a copy of X with the same pitch.
    x2, dx = dx_wide[:, :K], dx_wide[:, K:]
    x2.copy_(keep[0])
    opts = tg.gated_options(act=tg.ACT_GELU, ldx=2 * K, ldwg=4 * K, ldwu=4 * K, ldg=wide, ldu=wide, lddx=2 * K, lddwg=4 * K,
                            lddwu=4 * K)
    ptr = [t.data_ptr() for t in (dh, x2, wg, wu, g, u, dx, dwg, dwu)]
    assert tg.gated_backward_raw(*ptr, M, N, K, opts, stream, ws.data_ptr(), ws.numel()) == tg.Status.OK
    _ok()
    for name, got, t in zip(("dX", "dWg", "dWu"), (dx, dwg, dwu), want_grads):
        assert torch.equal(got, t), name
    assert all(torch.equal(a, b) for a, b in zip((x, wg, wu), keep)) and torch.equal(x2, keep[0])


def test_out_beside_x():
    """The torch call with H beside X in one buffer."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for M in (5, 300):
        buf = _randn(1, (M, 72 + 40), "bf16")
        w = _randn(2, (40, 72), "bf16", 0.1)
        want = tg.gated(buf[:, :72].contiguous(), w, w)
        got = tg.gated(buf[:, :72], w, w, out=buf[:, 72:])
        _ok()
        assert torch.equal(got, want) and torch.equal(buf[:, 72:], want)


@pytest.mark.parametrize("M,K", [(9, 64), (200, 1000), (3, 20000), (400, 8200)])
def test_codes_beside_values(M, K):
    """Codes in the gaps between the rows they are made from."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for shift in (0, 1):  # rows of X on 16-byte boundaries or off them
        pitch = (3 * K + 2 * shift + 15) // 16 * 16 + 2 * shift
        buf = torch.zeros(M * pitch + 64, dtype=torch.int8, device="cuda")
        x = buf[2 * shift:].view(torch.float16).as_strided((M, K), (pitch // 2, 1), shift)
        q = buf.as_strided((M, K), (pitch, 1), 2 * K + 2 * shift)
        src = _randn(K, (M, K), "f16")
        x.copy_(src)
        want = tg.quantize_i8(src)
        got = tg.quantize_i8(x, out=q)
        _ok()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(x, src)


# ---------------------------------------------------------------------------
# Blocks of every height of the small-M kernel
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [15, 32, 47, 64, 79, 81, 96, 112, 113, 128, 144, 190, 192, 240, 288])
def test_heights_of_row_blocks(M):
    """One block of 16 to 128 rows, and blocks of 64 to 96: rings of every size, K long enough to go round them."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    N, K, dt = 136, 2600, "bf16"
    x, wg, wu = _randn(M, (M, K), dt), _randn(2, (N, K), dt, K ** -0.5), _randn(3, (N, K), dt, K ** -0.5)
    got = tg.gated(x, wg, wu, save=True)
    (q, s), (qg, sg), (qu, su) = (tg.quantize_i8(t) for t in (x, wg, wu))
    c8, h8 = tg.gemm_i8(q, s, qg, sg, dtype=torch.bfloat16), tg.gated_i8(q, s, qg, sg, qu, su, dtype=torch.bfloat16)
    _ok()
    outs, tols = ref.gated(ref.f64(x), ref.f64(wg), ref.f64(wu), "silu", dt)
    for name, t, o, tol in zip("HGU", got, outs, tols):
        ref.check(ref.f64(t), o, tol, name)
    rows = (q.cpu().numpy(), s.cpu().numpy())
    g, dg = ref.i8_product(*rows, qg.cpu().numpy(), sg.cpu().numpy())
    u, du = ref.i8_product(*rows, qu.cpu().numpy(), su.cpu().numpy())
    ref.check(ref.f64(c8), g, dg + ref.round_error(g, dt), "C")
    outs, tols = ref.gate(g, u, dg, du, "silu", dt)
    ref.check(ref.f64(h8), outs[0], tols[0], "H, 8-bit")


# ---------------------------------------------------------------------------
# gated_block inside other machinery of torch
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("M", [40, 300])
def test_captured_training_step(M):
    """Forward and backward of gated_block captured after a warm-up on a side stream, replayed on new inputs."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    N, K, dt = 131, 72, "bf16"
    x, dh = _randn(1, (M, K), dt).requires_grad_(), _randn(4, (M, N), dt, 0.5)
    wg, wu = (_randn(i, (N, K), dt, 0.1).requires_grad_() for i in (2, 3))
    leaves = (x, wg, wu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            tg.gated_block(*leaves).backward(dh)
            for t in leaves:
                t.grad = None
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = tg.gated_block(*leaves)
        h.backward(dh)
    for seed in (7, 8):
        with torch.no_grad():
            x.copy_(_randn(seed, (M, K), dt))
            wu.copy_(_randn(seed + 1, (N, K), dt, 0.1))
        dh.copy_(_randn(seed + 2, (M, N), dt, 0.5))
        for t in leaves:
            t.grad.fill_(NAN)  # a replay writes the gradients, it does not add to them
        graph.replay()
        _ok()
        plain = [t.detach() for t in leaves]
        want_h, g, u = tg.gated(*plain, save=True)
        want = tg.gated_backward(dh, *plain, g, u)
        _ok()
        assert torch.equal(h, want_h) and all(torch.equal(t.grad, w) for t, w in zip(leaves, want))
    del graph


def test_checkpointed_and_compiled():
    """Recomputed in the backward pass, and between the parts of a compiled function: the same values."""
    import torch
    from torch.utils.checkpoint import checkpoint
    import tiled_dense_gemm_fp16_b200 as tg
    x, w = _randn(1, (40, 72), "f16"), _randn(2, (24, 72), "f16", 0.1).requires_grad_()

    def loss(a):
        return (tg.gated_block(a, w, w) * 2).float().sum()

    loss(x).backward()
    want, w.grad = w.grad, None
    for form in (lambda: checkpoint(loss, x, use_reentrant=False), lambda: torch.compile(loss, backend="eager")(x)):
        form().backward()
        _ok()
        assert torch.equal(w.grad, want)
        w.grad = None


def test_transforms_are_refused():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w = _randn(1, (40, 72), "f16"), _randn(2, (24, 72), "f16", 0.1)
    for call in (lambda: torch.func.vmap(lambda a: tg.gated_block(a, w, w))(x[None].expand(2, 40, 72)),
                 lambda: torch.func.grad(lambda a: tg.gated_block(a, w, w).float().sum())(x),
                 lambda: torch.func.jvp(lambda a: tg.gated_block(a, w, w), (x,), (x,))):
        with pytest.raises(RuntimeError):
            call()
    w.requires_grad_()
    first = torch.autograd.grad(tg.gated_block(x, w, w).float().sum(), w, create_graph=True)[0]
    with pytest.raises(RuntimeError):
        first.float().sum().backward()
    _ok()


def test_negated_views_under_autograd():
    """Values and gradients that are negated views count with their sign."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, w, dh = _randn(1, (40, 72), "f16"), _randn(2, (24, 72), "f16", 0.1).requires_grad_(), _randn(3, (40, 24), "f16")
    h = tg.gated_block(torch._neg_view(x), w, w)
    h.backward(torch._neg_view(dh))
    got, w.grad = w.grad, None
    want = tg.gated_block(-x, w, w)
    want.backward(-dh)
    _ok()
    assert torch.equal(h, want) and torch.equal(got, w.grad)


@pytest.mark.parametrize("M", [20, 128, 300, 2000])
@pytest.mark.parametrize("N,ld", [(41, 48), (129, 136), (263, 264), (7, 8)])
def test_bytes_behind_rows_on_16_byte_boundaries(M, N, ld):
    """Rows that start on 16-byte boundaries and end inside one: the bytes up to the next row stay."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    K, guard = 96, 0x5A5A
    x, wg, wu = _randn(1, (M, K), "f16"), _randn(2, (N, K), "f16", 0.1), _randn(3, (N, K), "f16", 0.1)
    dh = _randn(4, (M, N), "f16", 0.5)

    def framed(rows, cols, pitch):
        whole = torch.full((rows, pitch), guard, dtype=torch.int16, device="cuda")
        return whole, whole.view(torch.float16)[:, :cols]

    stream = torch.cuda.current_stream().cuda_stream
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    results = [framed(M, N, ld) for _ in range(3)]
    opts = tg.gated_options(act=tg.ACT_SILU, ldh=ld, ldg=ld, ldu=ld)
    ptr = [t.data_ptr() for t in (x, wg, wu, *(r[1] for r in results))]
    assert tg.gated_raw(*ptr, M, N, K, opts, stream, ws.data_ptr(), ws.numel()) == tg.Status.OK
    grads = [framed(rows, K - 1, K) for rows in (M, N, N)]  # of a block that is K - 1 wide
    opts = tg.gated_options(act=tg.ACT_SILU, ldx=K, ldwg=K, ldwu=K, ldg=ld, ldu=ld, lddx=K, lddwg=K, lddwu=K)
    ptr = [t.data_ptr() for t in (dh, x, wg, wu, *(r[1] for r in results[1:]), *(r[1] for r in grads))]
    assert tg.gated_backward_raw(*ptr, M, N, K - 1, opts, stream, ws.data_ptr(), ws.numel()) == tg.Status.OK
    (q, s), (qw, sw) = tg.quantize_i8(x), tg.quantize_i8(wg)
    products = [framed(M, N, ld) for _ in range(2)]
    tg.gemm_i8(q, s, qw, sw, out=products[0][1])
    tg.gated_i8(q, s, qw, sw, qw, sw, out=products[1][1])
    _ok()
    for (whole, view), cols in [(r, N) for r in (*results, *products)] + [(r, K - 1) for r in grads]:
        assert torch.all(whole[:, cols:] == guard)
    want = tg.gated(x, wg, wu, save=True)
    assert all(torch.equal(r[1], w) for r, w in zip(results, want))
    xk, gk, uk = (t[:, :K - 1].contiguous() for t in (x, wg, wu))
    for r, w in zip(grads, tg.gated_backward(dh, xk, gk, uk, *want[1:])):
        assert torch.equal(r[1], w)
    assert torch.equal(products[0][1], tg.gemm_i8(q, s, qw, sw)) and torch.equal(products[1][1], tg.gated_i8(q, s, qw, sw, qw, sw))


@pytest.mark.parametrize("M", [5, 70, 300, 700])
@pytest.mark.parametrize("N,K", [(41, 33), (137, 65), (264, 127), (40, 7)])
def test_short_gaps_are_not_read(M, N, K):
    """NaN behind rows that start on 16-byte boundaries and end inside one (TMA reads such operands in place)."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg

    def spaced(t):
        wide = torch.full((t.shape[0], (t.shape[1] + 7) // 8 * 8), NAN, dtype=t.dtype, device="cuda")
        wide[:, :t.shape[1]] = t
        return wide[:, :t.shape[1]]

    x, wg, wu, dh = (_randn(i, s, "bf16", 0.2) for i, s in enumerate(((M, K), (N, K), (N, K), (M, N))))
    want = tg.gated(x, wg, wu, save=True)
    got = tg.gated(spaced(x), spaced(wg), spaced(wu), save=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    want_g = tg.gated_backward(dh, x, wg, wu, *want[1:])
    got_g = tg.gated_backward(spaced(dh), spaced(x), spaced(wg), spaced(wu), spaced(want[1]), spaced(want[2]))
    assert all(torch.equal(a, b) for a, b in zip(want_g, got_g))
    assert all(torch.equal(a, b) for a, b in zip(tg.quantize_i8(x), tg.quantize_i8(spaced(x))))
    _ok()
