"""The feed-forward operators against their definitions in 64 bits: the gated block, its gradients, row
quantization and the 8-bit products.  Tolerances: ff_ref.py."""
import numpy as np
import pytest

import ff_ref as ref

pytestmark = pytest.mark.gpu

GUARD = 0x5A5A


def _rng_tensor(seed, shape, dt, scale=1.0):
    import torch
    v = np.random.default_rng(seed).standard_normal(shape) * scale
    return torch.from_numpy(v).cuda().to(ref.torch_type(dt))


def _ok():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    torch.cuda.synchronize()
    st, word = tg.device_status()
    assert st == tg.Status.OK, hex(word)


def _framed(rows, cols, ld, offset, dtype):
    """A (rows, cols) view with row stride ld at an element offset inside a guarded buffer."""
    import torch
    width = torch.empty(0, dtype=dtype).element_size()
    bits = torch.int8 if width == 1 else torch.int16
    buf = torch.full((64 + offset + max(rows, 1) * ld + 64,), 0x5A if width == 1 else GUARD, dtype=bits, device="cuda").view(dtype)
    return buf, buf[64 + offset:].as_strided((rows, cols), (ld, 1))


def _guards_ok(buf, view, ld, offset):
    import torch
    width = view.element_size()
    host = buf.view(torch.int8 if width == 1 else torch.int16).cpu().numpy().copy()
    rows, cols = view.shape
    for r in range(rows):
        host[64 + offset + r * ld:64 + offset + r * ld + cols] = 0x5A if width == 1 else GUARD
    assert np.all(host == (0x5A if width == 1 else GUARD)), "bytes outside the result were written"


def _gated_inputs(M, N, K, dt, seed):
    return (_rng_tensor(seed, (M, K), dt), _rng_tensor(seed + 1, (N, K), dt, K ** -0.5),
            _rng_tensor(seed + 2, (N, K), dt, K ** -0.5))


SIZES = [(1, 8, 8), (1, 1, 64), (2, 64, 72), (16, 136, 520), (127, 70, 264), (129, 130, 64), (130, 1000, 264),
         (257, 129, 72), (300, 520, 1032), (513, 257, 200)]


# ---------------------------------------------------------------------------
# Gated forward
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated(M, N, K, act, dt):
    import tiled_dense_gemm_fp16_b200 as tg
    x, wg, wu = _gated_inputs(M, N, K, dt, seed=M + N + K)
    got = tg.gated(x, wg, wu, act=act)
    saved = tg.gated(x, wg, wu, act=act, save=True)
    _ok()
    outs, tols = ref.gated(ref.f64(x), ref.f64(wg), ref.f64(wu), act, dt)
    ref.check(ref.f64(got), outs[0], tols[0], "H")
    for name, t, o, tol in zip(("H saved", "G", "U"), saved, outs, tols):
        ref.check(ref.f64(t), o, tol, name)
    assert np.array_equal(ref.f64(got), ref.f64(saved[0])), "storing G and U changed H"


@pytest.mark.parametrize("M,N,K,dx,dw,dh", [
    (5, 40, 33, 0, 0, 0), (1, 24, 21, 1, 1, 1), (200, 72, 65, 3, 0, 5), (300, 261, 136, 0, 5, 1), (300, 264, 129, 8, 3, 0),
])
def test_gated_strides_and_offsets(M, N, K, dx, dw, dh):
    """Row strides and bases on any 2-byte boundary; bytes around and between the rows of the results stay."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    dt = torch.float16
    x0, wg0, wu0 = _gated_inputs(M, N, K, "f16", seed=K)
    _, x = _framed(M, K, K + dx, dx, dt)
    _, wg = _framed(N, K, K + dw, dw, dt)
    _, wu = _framed(N, K, K + 2 * dw + 1, 0, dt)
    for view, src in ((x, x0), (wg, wg0), (wu, wu0)):
        view.copy_(src)
    ldh = N + dh
    frames = [_framed(M, N, ldh, dh, dt) for _ in range(3)]
    H, G, U = (f[1] for f in frames)
    opts = tg.gated_options(act=tg.ACT_SILU, ldx=K + dx, ldwg=K + dw, ldwu=K + 2 * dw + 1, ldh=ldh, ldg=ldh, ldu=ldh)
    need = tg.gated_workspace_size(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), M, N, K, opts)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    st = tg.gated_raw(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), H.data_ptr(), G.data_ptr(), U.data_ptr(), M, N, K, opts,
                      torch.cuda.current_stream().cuda_stream, ws.data_ptr(), need)
    assert st == tg.Status.OK
    _ok()
    outs, tols = ref.gated(ref.f64(x0), ref.f64(wg0), ref.f64(wu0), "silu", "f16")
    for name, f, o, tol in zip("HGU", frames, outs, tols):
        ref.check(ref.f64(f[1]), o, tol, name)
        _guards_ok(f[0], f[1], ldh, dh)


def test_gated_merged_weight_leading_dims_and_out():
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    w = _rng_tensor(3, (2 * 136, 72), "bf16", 0.1)
    x = _rng_tensor(4, (3, 50, 72), "bf16")
    out = torch.empty((3, 50, 136), dtype=torch.bfloat16, device="cuda")
    got = tg.gated(x, w[:136], w[136:], act="gelu", out=out)
    assert got is out
    _ok()
    outs, tols = ref.gated(ref.f64(x).reshape(150, 72), ref.f64(w[:136]), ref.f64(w[136:]), "gelu", "bf16")
    ref.check(ref.f64(got).reshape(150, 136), outs[0], tols[0], "H")


@pytest.mark.parametrize("M,N,K", [(0, 8, 8), (8, 0, 8), (0, 0, 0), (3, 5, 0), (300, 9, 0)])
def test_gated_empty(M, N, K):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    x, wg, wu = (torch.zeros(s, dtype=torch.float16, device="cuda") for s in ((M, K), (N, K), (N, K)))
    h, g, u = tg.gated(x, wg, wu, act="gelu", save=True)
    grads = tg.gated_backward(torch.ones_like(h), x, wg, wu, g, u, act="gelu")
    _ok()
    assert h.shape == (M, N) and not h.any() and not g.any() and not u.any()
    for t, like in zip(grads, (x, wg, wu)):
        assert t.shape == like.shape and not t.any()


def test_gated_special_values():
    """Overflow gives infinities, a row that is not finite reaches no other row, and far gates are exact zeros or the identity."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for M in (7, 300):
        x = torch.zeros((M, 64), dtype=torch.float16, device="cuda")
        x[:, 0] = torch.linspace(-60000, 60000, M).to(torch.float16)
        x[3, 1] = float("inf")
        x[5, 2] = float("nan")
        w = torch.zeros((16, 64), dtype=torch.float16, device="cuda")
        w[:, 0] = 1
        w[:, 1] = 1
        w[:, 2] = 1
        wu = torch.zeros_like(w)
        wu[:, 0] = 1
        for act in ("silu", "gelu", "relu"):
            h = tg.gated(x, w, wu, act=act).float().cpu()
            _ok()
            for m in range(M):
                v = float(x[m, 0])
                if m in (3, 5):  # U holds 0 * inf or NaN: NaN whatever the gate is
                    assert torch.all(torch.isnan(h[m]))
                else:
                    want = v * v if v > 0 else 0.0
                    want = float("inf") if want >= 65520 else float(np.float16(want))
                    assert torch.all(h[m] == want), (act, m, v, h[m, 0])


# ---------------------------------------------------------------------------
# Gated backward
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_gated_backward(M, N, K, act, dt):
    import tiled_dense_gemm_fp16_b200 as tg
    x, wg, wu = _gated_inputs(M, N, K, dt, seed=M * 3 + N + K)
    dh = _rng_tensor(9, (M, N), dt, 0.5)
    _, g, u = tg.gated(x, wg, wu, act=act, save=True)
    grads = tg.gated_backward(dh, x, wg, wu, g, u, act=act)
    _ok()
    outs, tols = ref.gated_backward(*(ref.f64(t) for t in (dh, x, wg, wu, g, u)), act, dt)
    for name, t, o, tol in zip(("dX", "dWg", "dWu"), grads, outs, tols):
        ref.check(ref.f64(t), o, tol, name)


@pytest.mark.parametrize("needs", [(True, False, False), (False, True, False), (False, False, True), (True, False, True),
                                   (False, False, False)])
def test_gated_backward_needs(needs):
    import tiled_dense_gemm_fp16_b200 as tg
    x, wg, wu = _gated_inputs(70, 136, 72, "f16", seed=5)
    dh = _rng_tensor(6, (70, 136), "f16")
    _, g, u = tg.gated(x, wg, wu, save=True)
    full = tg.gated_backward(dh, x, wg, wu, g, u)
    part = tg.gated_backward(dh, x, wg, wu, g, u, needs=needs)
    _ok()
    for n, f, p in zip(needs, full, part):
        assert (p is not None) == n
        if n:
            assert np.array_equal(ref.f64(f), ref.f64(p))


@pytest.mark.parametrize("M,N,K,pad", [(5, 41, 33, 1), (200, 72, 65, 3), (300, 263, 129, 0), (300, 136, 72, 5)])
def test_gated_backward_strides(M, N, K, pad):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    dt = torch.float16
    x0, wg0, wu0 = _gated_inputs(M, N, K, "f16", seed=K)
    dh0 = _rng_tensor(8, (M, N), "f16")
    _, g0, u0 = tg.gated(x0, wg0, wu0, act="gelu", save=True)
    views = []
    for src in (dh0, x0, wg0, wu0, g0, u0):
        _, v = _framed(*src.shape, src.shape[1] + pad, pad, dt)
        v.copy_(src)
        views.append(v)
    outs = [_framed(*s, s[1] + pad, pad, dt) for s in ((M, K), (N, K), (N, K))]
    opts = tg.gated_options(act=tg.ACT_GELU, ldx=K + pad, ldwg=K + pad, ldwu=K + pad, ldh=N + pad, ldg=N + pad, ldu=N + pad,
                            lddx=K + pad, lddwg=K + pad, lddwu=K + pad)
    ptr = [v.data_ptr() for v in views]
    optr = [o[1].data_ptr() for o in outs]
    need = tg.gated_backward_workspace_size(*ptr[1:4], *optr, M, N, K, opts)
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    st = tg.gated_backward_raw(*ptr, *optr, M, N, K, opts, torch.cuda.current_stream().cuda_stream, buf.data_ptr(), need)
    assert st == tg.Status.OK
    _ok()
    assert torch.all(buf[need:] == 0x5A)
    want, tols = ref.gated_backward(*(ref.f64(t) for t in (dh0, x0, wg0, wu0, g0, u0)), "gelu", "f16")
    for name, o, w, tol in zip(("dX", "dWg", "dWu"), outs, want, tols):
        ref.check(ref.f64(o[1]), w, tol, name)
        _guards_ok(o[0], o[1], K + pad, pad)


# ---------------------------------------------------------------------------
# Row quantization
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 8), (3, 7), (9, 64), (17, 1000), (5, 1024), (4, 1025), (3, 4096), (7, 8192),
                                 (2, 8200), (3, 20001), (2000, 40)])
def test_quantize(M, K, dt):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    rng = np.random.default_rng(M + K)
    v = rng.standard_normal((M, K)) * 10.0 ** rng.uniform(-3, 3, size=(M, 1))
    if M > 2:
        v[1] = 0.0
    if K > 5:  # exact ties: multiples of half a scale of 1
        v[0, 0] = 127.0
        v[0, 1:] = rng.integers(-253, 254, size=K - 1) / 2
    x = torch.from_numpy(v).cuda().to(ref.torch_type(dt))
    q, s = tg.quantize_i8(x)
    _ok()
    want_q, want_s = ref.quantize(ref.f64(x))
    assert q.shape == x.shape and q.stride(0) % 16 == 0
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.cpu().numpy(), want_q)


def test_quantize_every_pattern():
    """Every bit pattern of either type, in rows whose largest value sweeps the whole range."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    bits = np.arange(1 << 15, dtype=np.uint16)
    for dt, top in (("f16", 0x7C00), ("bf16", 0x7F80)):
        rows = []
        for hi in list(range(1, 40)) + list(range(40, top, 977)) + [top - 1]:
            lo = max(0, hi - 2000)
            row = np.resize(bits[lo:hi + 1], 2048).copy()
            row[0] = hi
            row[1::2] |= 0x8000
            rows.append(row)
        x = torch.from_numpy(np.stack(rows).view(np.int16)).cuda().view(ref.torch_type(dt))
        q, s = tg.quantize_i8(x)
        _ok()
        want_q, want_s = ref.quantize(ref.f64(x))
        assert np.array_equal(s.cpu().numpy(), want_s)
        assert np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_quantize_not_finite(dt):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    for K in (65, 5000):
        x = _rng_tensor(1, (6, K), dt)
        x[1, K - 1] = float("inf")
        x[2, 0] = float("-inf")
        x[4, K // 2] = float("nan")
        q, s = tg.quantize_i8(x)
        _ok()
        want_q, want_s = ref.quantize(ref.f64(x))
        assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True) and np.array_equal(q.cpu().numpy(), want_q)


@pytest.mark.parametrize("M,K,ldx,ldq,off", [(9, 33, 33, 33, 0), (9, 33, 40, 48, 0), (5, 1031, 1033, 1031, 1), (6, 4096, 4104, 4100, 8)])
def test_quantize_strides(M, K, ldx, ldq, off):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    src = _rng_tensor(2, (M, K), "bf16")
    _, x = _framed(M, K, ldx, off, torch.bfloat16)
    x.copy_(src)
    buf, q = _framed(M, K, ldq, off, torch.int8)
    s = torch.empty(M, dtype=torch.float32, device="cuda")
    st = tg.quantize_rows_i8_raw(x.data_ptr(), q.data_ptr(), s.data_ptr(), M, K, ldx, ldq, tg.TYPE_BF16,
                                 torch.cuda.current_stream().cuda_stream)
    assert st == tg.Status.OK
    _ok()
    want_q, want_s = ref.quantize(ref.f64(src))
    assert np.array_equal(q.cpu().numpy(), want_q) and np.array_equal(s.cpu().numpy(), want_s)
    _guards_ok(buf, q, ldq, off)


# ---------------------------------------------------------------------------
# 8-bit products
# ---------------------------------------------------------------------------

def _codes(seed, rows, K, ld=None):
    """Codes over the whole signed byte, -128 included, rows on 16-byte boundaries; and scales."""
    import torch
    rng = np.random.default_rng(seed)
    ld = ld or (K + 15) // 16 * 16
    full = torch.from_numpy(rng.integers(-128, 128, size=(rows, ld)).astype(np.int8)).cuda()
    scale = torch.from_numpy((rng.uniform(0.5, 2.0, size=rows) * 0.01).astype(np.float32)).cuda()
    return full[:, :K], scale  # bytes past K are not zero


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("relu,bias", [(False, False), (True, True)])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 130, 40), (16, 264, 1000), (65, 129, 513), (130, 72, 200), (257, 300, 72),
                                   (300, 520, 1032), (600, 515, 333)])
def test_gemm_i8(M, N, K, relu, bias, dt):
    import tiled_dense_gemm_fp16_b200 as tg
    a, sa = _codes(M, M, K)
    w, sw = _codes(N + 1, N, K)
    b = _rng_tensor(3, (N,), dt) if bias else None
    got = tg.gemm_i8(a, sa, w, sw, bias=b, relu=relu, dtype=ref.torch_type(dt))
    _ok()
    c, err = ref.i8_product(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy())
    if bias:
        c = c + ref.f64(b)
        err = err + np.abs(c) * 2.0 ** -24
    if relu:
        c = np.maximum(c, 0)
    ref.check(ref.f64(got), c, err + ref.round_error(c, dt), "C")


@pytest.mark.parametrize("M", [1, 64, 300])
def test_gemm_i8_sums_are_exact(M):
    """The largest K and codes of one sign: sums next to 2^31, exact before their one rounding."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    K, N = 131071, 24
    a = torch.full((M, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    w = torch.full((N, 131072), -128, dtype=torch.int8, device="cuda")[:, :K]
    w[1::2] = 127
    one = torch.ones(M, device="cuda")
    sw = torch.full((N,), 2.0 ** -20, device="cuda")
    got = tg.gemm_i8(a, one, w, sw, dtype=torch.bfloat16).double().cpu()
    _ok()
    want = torch.where(torch.arange(N) % 2 == 0, 16384.0 * K, -16256.0 * K).float() * 2.0 ** -20
    assert torch.equal(got, want.to(torch.bfloat16).double().expand(M, N))


@pytest.mark.parametrize("M,N,bias,relu", [(5, 9, True, True), (5, 9, True, False), (300, 7, False, False)])
def test_gemm_i8_without_k(M, N, bias, relu):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    a, w = (torch.empty((r, 0), dtype=torch.int8, device="cuda") for r in (M, N))
    b = _rng_tensor(3, (N,), "f16") if bias else None
    got = tg.gemm_i8(a, torch.ones(M, device="cuda"), w, torch.ones(N, device="cuda"), bias=b, relu=relu)
    _ok()
    want = torch.zeros((M, N), dtype=torch.float16, device="cuda") + (b if bias else 0)
    assert torch.equal(got, want.relu() if relu else want)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (16, 136, 1000), (129, 130, 200), (257, 129, 72), (520, 520, 1040)])
def test_gated_i8(M, N, K, act, dt):
    import tiled_dense_gemm_fp16_b200 as tg
    a, sa = _codes(M, M, K)
    wg, sg = _codes(N + 1, N, K)
    wu, su = _codes(N + 2, N, K)
    got = tg.gated_i8(a, sa, wg, sg, wu, su, act=act, dtype=ref.torch_type(dt))
    _ok()
    host = [t.cpu().numpy() for t in (a, sa, wg, sg, wu, su)]
    g, dg = ref.i8_product(host[0], host[1], host[2], host[3])
    u, du = ref.i8_product(host[0], host[1], host[4], host[5])
    outs, tols = ref.gate(g, u, dg, du, act, dt)
    ref.check(ref.f64(got), outs[0], tols[0], "H")


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,pad,off", [(300, 700, 0, 1), (300, 700, 1, 0), (300, 701, 0, 0), (290, 1025, 1, 1), (257, 95, 2, 3),
                                         (130, 64, 1, 0), (1000, 5003, 0, 0), (20, 77, 3, 1)])
def test_i8_results_on_any_boundary(M, N, pad, off, gated):
    """Rows of the result on every 2-byte boundary; bytes around and between them stay."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    K = 48
    a, sa = _codes(M, M, K)
    w, sw = _codes(N + 1, N, K)
    u, su = _codes(N + 2, N, K)
    frame, c = _framed(M, N, N + pad, off, torch.bfloat16)
    if gated:
        got = tg.gated_i8(a, sa, w, sw, u, su, act="relu", out=c)
    else:
        got = tg.gemm_i8(a, sa, w, sw, out=c)
    _ok()
    assert got is c
    host = [t.cpu().numpy() for t in (a, sa, w, sw, u, su)]
    g, dg = ref.i8_product(*host[:4])
    if gated:
        v, dv = ref.i8_product(host[0], host[1], host[4], host[5])
        outs, tols = ref.gate(g, v, dg, dv, "relu", "bf16")
        g, tol = outs[0], tols[0]
    else:
        tol = dg + ref.round_error(g, "bf16")
    ref.check(ref.f64(c), g, tol, "C")
    _guards_ok(frame, c, N + pad, off)


# ---------------------------------------------------------------------------
# Few tiles and long sums: K split over a cluster, in blocks of rows
# ---------------------------------------------------------------------------

# Blocks that end inside their rows, panels that end inside their columns, K that ends inside a k-block; sums over
# the columns of X (forward), of G and U (dX) and over the rows (dWg, dWu).
LONG = [(129, 64, 1536), (131, 70, 1501), (300, 136, 2104), (640, 40, 3001), (700, 1040, 72), (515, 1501, 129),
        (1500, 89, 93), (2050, 200, 136), (2304, 320, 64), (4099, 65, 7)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,N,K", LONG)
def test_gated_long_sums(M, N, K, dt):
    import tiled_dense_gemm_fp16_b200 as tg
    x, wg, wu = _gated_inputs(M, N, K, dt, seed=M + N + K)
    dh = _rng_tensor(9, (M, N), dt, 0.5)
    h, g, u = tg.gated(x, wg, wu, act="gelu", save=True)
    again = tg.gated(x, wg, wu, act="gelu")
    grads = tg.gated_backward(dh, x, wg, wu, g, u, act="gelu")
    _ok()
    outs, tols = ref.gated(ref.f64(x), ref.f64(wg), ref.f64(wu), "gelu", dt)
    for name, t, o, tol in zip("HGU", (h, g, u), outs, tols):
        ref.check(ref.f64(t), o, tol, name)
    assert np.array_equal(ref.f64(h), ref.f64(again))
    outs, tols = ref.gated_backward(*(ref.f64(t) for t in (dh, x, wg, wu, g, u)), "gelu", dt)
    for name, t, o, tol in zip(("dX", "dWg", "dWu"), grads, outs, tols):
        ref.check(ref.f64(t), o, tol, name)


@pytest.mark.parametrize("needs", [(False, True, False), (False, False, True), (True, False, True)])
def test_gated_backward_long_sums_needs(needs):
    """One weight's gradient alone is the same as beside the other's, whatever K is split into."""
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K = 2050, 200, 136
    x, wg, wu = _gated_inputs(M, N, K, "f16", seed=5)
    dh = _rng_tensor(6, (M, N), "f16")
    _, g, u = tg.gated(x, wg, wu, save=True)
    part = tg.gated_backward(dh, x, wg, wu, g, u, needs=needs)
    again = tg.gated_backward(dh, x, wg, wu, g, u, needs=needs)
    _ok()
    outs, tols = ref.gated_backward(*(ref.f64(t) for t in (dh, x, wg, wu, g, u)), "silu", "f16")
    for n, p, a, o, tol in zip(needs, part, again, outs, tols):
        assert (p is not None) == n
        if n:
            ref.check(ref.f64(p), o, tol, "gradient")
            assert np.array_equal(ref.f64(p), ref.f64(a))


@pytest.mark.parametrize("M,N,K,pad", [(300, 72, 1537, 1), (1301, 72, 65, 3), (259, 1101, 40, 0)])
def test_long_sums_on_any_boundary(M, N, K, pad):
    """Results with gaps between their rows, on every 2-byte boundary; bytes around and between the rows stay."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    dt = torch.float16
    x, wg, wu = _gated_inputs(M, N, K, "f16", seed=K)
    dh = _rng_tensor(8, (M, N), "f16")
    frames = [_framed(M, N, N + pad, pad, dt) for _ in range(3)]
    outs = [_framed(*s, s[1] + pad, pad, dt) for s in ((M, K), (N, K), (N, K))]
    opts = tg.gated_options(act=tg.ACT_GELU, ldh=N + pad, ldg=N + pad, ldu=N + pad)
    stream = torch.cuda.current_stream().cuda_stream
    px, pg, pu = (t.data_ptr() for t in (x, wg, wu))
    ptr = [f[1].data_ptr() for f in frames]
    need = tg.gated_workspace_size(px, pg, pu, M, N, K, opts)
    ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    assert tg.gated_raw(px, pg, pu, *ptr, M, N, K, opts, stream, ws.data_ptr(), need) == tg.Status.OK
    opts = tg.gated_options(act=tg.ACT_GELU, ldg=N + pad, ldu=N + pad, lddx=K + pad, lddwg=K + pad, lddwu=K + pad)
    optr = [o[1].data_ptr() for o in outs]
    need = tg.gated_backward_workspace_size(px, pg, pu, *optr, M, N, K, opts)
    buf = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    st = tg.gated_backward_raw(dh.data_ptr(), px, pg, pu, ptr[1], ptr[2], *optr, M, N, K, opts, stream, buf.data_ptr(), need)
    assert st == tg.Status.OK
    _ok()
    assert torch.all(buf[need:] == 0x5A)
    want, tols = ref.gated(ref.f64(x), ref.f64(wg), ref.f64(wu), "gelu", "f16")
    for name, f, w, tol in zip("HGU", frames, want, tols):
        ref.check(ref.f64(f[1]), w, tol, name)
        _guards_ok(f[0], f[1], N + pad, pad)
    want, tols = ref.gated_backward(*(ref.f64(t) for t in (dh, x, wg, wu, frames[1][1], frames[2][1])), "gelu", "f16")
    for name, o, w, tol in zip(("dX", "dWg", "dWu"), outs, want, tols):
        ref.check(ref.f64(o[1]), w, tol, name)
        _guards_ok(o[0], o[1], K + pad, pad)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(129, 64, 4096), (300, 520, 2064), (600, 71, 3333), (131, 700, 2500), (2000, 130, 4000)])
def test_i8_long_sums(M, N, K, gated):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    a, sa = _codes(M, M, K)
    w, sw = _codes(N + 1, N, K)
    u, su = _codes(N + 2, N, K)
    b = _rng_tensor(3, (N,), "bf16")
    host = [t.cpu().numpy() for t in (a, sa, w, sw, u, su)]
    c, err = ref.i8_product(*host[:4])
    if gated:
        got = tg.gated_i8(a, sa, w, sw, u, su, act="silu", dtype=torch.bfloat16)
        v, dv = ref.i8_product(*host[:2], *host[4:])
        outs, tols = ref.gate(c, v, err, dv, "silu", "bf16")
        c, tol = outs[0], tols[0]
    else:
        got = tg.gemm_i8(a, sa, w, sw, bias=b, relu=True, dtype=torch.bfloat16)
        c = c + ref.f64(b)
        err = err + np.abs(c) * 2.0 ** -24
        c = np.maximum(c, 0)
        tol = err + ref.round_error(c, "bf16")
    _ok()
    ref.check(ref.f64(got), c, tol, "C")


def test_long_sums_keep_rows_apart():
    """A row with an infinity or a NaN reaches its own row of H and of dX, and no other; a column of G does so in dWg."""
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    M, N, K = 260, 72, 1536
    x, wg, wu = _gated_inputs(M, N, K, "f16", seed=1)
    clean = tg.gated(x, wg, wu, act="relu")
    x[127, 3], x[259, K - 1] = float("nan"), float("inf")
    got = tg.gated(x, wg, wu, act="relu")
    _ok()
    rows = torch.ones(M, dtype=torch.bool, device="cuda")
    rows[127] = rows[259] = False
    assert torch.equal(got[rows], clean[rows])
    assert torch.isnan(got[127]).all()
    M, N, K = 2100, 130, 72
    x, wg, wu = _gated_inputs(M, N, K, "f16", seed=2)
    dh = _rng_tensor(3, (M, N), "f16")
    _, g, u = tg.gated(x, wg, wu, act="silu", save=True)
    dx0, dwg0, dwu0 = tg.gated_backward(dh, x, wg, wu, g, u)
    dh[2099, 63] = float("nan")
    dx, dwg, dwu = tg.gated_backward(dh, x, wg, wu, g, u)
    _ok()
    assert torch.equal(dx[:2099], dx0[:2099]) and torch.isnan(dx[2099]).all()
    cols = torch.ones(N, dtype=torch.bool, device="cuda")
    cols[63] = False
    for got, want in ((dwg, dwg0), (dwu, dwu0)):
        assert torch.equal(got[cols], want[cols]) and torch.isnan(got[63]).all()
