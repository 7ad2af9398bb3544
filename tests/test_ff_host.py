"""Host logic of the feed-forward operators: sizes, strides, alignment, overlap, workspaces.  No kernel is
launched: without a GPU a call that passes every check ends in UNSUPPORTED_DEVICE."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

import tiled_dense_gemm_fp16_b200 as tg
from tiled_dense_gemm_fp16_b200 import Status

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Well-separated fake device addresses (never dereferenced by host logic).
P = [0x10_0000_0000 * (i + 1) for i in range(12)]
BAD = Status.INVALID_ARG


def gated(M=8, N=8, K=8, opts=None, x=P[0], wg=P[1], wu=P[2], h=P[3], g=0, u=0, ws=0, ws_bytes=0):
    return tg.gated_raw(x, wg, wu, h, g, u, M, N, K, opts, 0, ws, ws_bytes)


def backward(M=8, N=8, K=8, opts=None, dh=P[0], x=P[1], wg=P[2], wu=P[3], g=P[4], u=P[5], dx=P[6], dwg=P[7], dwu=P[8],
             ws=P[9], ws_bytes=1 << 30):
    return tg.gated_backward_raw(dh, x, wg, wu, g, u, dx, dwg, dwu, M, N, K, opts, 0, ws, ws_bytes)


def gemm_i8(M=8, N=8, K=16, a=P[0], sa=P[1], w=P[2], sw=P[3], bias=0, c=P[4], **kw):
    return tg.gemm_i8_raw(a, sa, w, sw, bias, c, M, N, K, **kw)


def gated_i8(M=8, N=8, K=16, opts=None, a=P[0], sa=P[1], wg=P[2], sg=P[3], wu=P[4], su=P[5], h=P[6]):
    return tg.gated_i8_raw(a, sa, wg, sg, wu, su, h, M, N, K, opts)


def quantize(M=8, K=8, x=P[0], q=P[1], s=P[2], **kw):
    return tg.quantize_rows_i8_raw(x, q, s, M, K, **kw)


def test_options_struct_matches_the_header():
    text = open(os.path.join(ROOT, "include", "tg_gemm.h")).read()
    body = re.search(r"typedef struct tg_gated_options \{(.*?)\}", text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [n for t, ns in re.findall(r"(int32_t|int64_t)\s+([\w, ]+);", body) for n in ns.replace(" ", "").split(",")]
    assert names == [f[0] for f in tg.GatedOptions._fields_]
    assert ctypes.sizeof(tg.GatedOptions) == 2 * 4 + 10 * 8


@pytest.mark.parametrize("sizes", [(-1, 8, 8), (8, -1, 8), (8, 8, -1), ((1 << 30) + 1, 8, 8), (8, (1 << 30) + 1, 8),
                                   (8, 8, (1 << 30) + 1)])
def test_sizes(sizes):
    assert gated(*sizes) == BAD and backward(*sizes) == BAD
    assert gemm_i8(*sizes) == BAD and gated_i8(*sizes) == BAD
    assert tg.gated_workspace_size(*P[:3], *sizes) == -1
    assert tg.gated_backward_workspace_size(*P[:6], *sizes) == -1


def test_spans_stay_countable():
    """Sizes or strides whose byte counts would leave 64 bits are refused, not computed with."""
    big = 1 << 30
    assert tg.gated_workspace_size(*P[:3], big, big, 8) == -1 and tg.gated_workspace_size(*P[:3], big, 8, big) == -1
    assert tg.gated_backward_workspace_size(*P[:6], 8, big, big) == -1
    assert tg.gated_workspace_size(*P[:3], big, 1 << 20, 8) == 0
    assert gated(big, 8, 8, tg.gated_options(ldx=1 << 38)) == BAD and gated(big, 8, 8, tg.gated_options(ldh=1 << 38)) == BAD
    assert gemm_i8(big, 8, 16, lda=1 << 38) == BAD and quantize(big, 8, ldx=1 << 38) == BAD and quantize(big, 8, ldq=1 << 38) == BAD


def test_k_of_the_integer_sums():
    assert gemm_i8(K=131072) == BAD and gated_i8(K=131072) == BAD
    if not _gpu():
        assert gemm_i8(K=131071, lda=131072, ldw=131072) == Status.UNSUPPORTED_DEVICE


def _gpu():
    import torch
    return torch.cuda.is_available()


def test_enumerations():
    for o in (tg.gated_options(type=2), tg.gated_options(type=-1), tg.gated_options(act=3), tg.gated_options(act=-1),
              tg.gated_options(reserved=1)):
        assert gated(opts=o) == BAD and backward(opts=o) == BAD and gated_i8(opts=o) == BAD
    assert gemm_i8(type=2) == BAD and quantize(type=2) == BAD
    lib = tg.lib()
    assert lib.tg_gemm_i8(P[0], P[1], P[2], P[3], 0, P[4], 8, 8, 16, 0, 0, 0, 2, 0, 0) == BAD  # relu is 0 or 1


def test_null_and_odd_pointers():
    for name in ("x", "wg", "wu", "h"):
        assert gated(**{name: 0}) == BAD and gated(**{name: P[11] + 1}) == BAD
    assert gated(g=P[4]) == BAD and gated(u=P[4]) == BAD  # both or neither
    for name in ("dh", "x", "wg", "wu", "g", "u"):
        assert backward(**{name: 0}) == BAD and backward(**{name: P[11] + 1}) == BAD
    for name in ("dx", "dwg", "dwu"):
        assert backward(**{name: P[11] + 1}) == BAD
    for name in ("a", "sa", "w", "sw", "c"):
        assert gemm_i8(**{name: 0}) == BAD
    for name, off in (("a", 8), ("w", 8), ("sa", 2), ("sw", 2), ("c", 1), ("bias", 1)):
        assert gemm_i8(**{name: P[11] + off}) == BAD
    for name in ("a", "sa", "wg", "sg", "wu", "su", "h"):
        assert gated_i8(**{name: 0}) == BAD and gated_i8(**{name: P[11] + 1}) == BAD
    assert quantize(x=0) == BAD and quantize(q=0) == BAD and quantize(s=0) == BAD
    assert quantize(x=P[0] + 1) == BAD and quantize(s=P[2] + 2) == BAD


def test_strides():
    o = tg.gated_options
    for field in ("ldx", "ldwg", "ldwu", "ldh"):
        for bad in (7, -8, (1 << 38) + 8):
            assert gated(opts=o(**{field: bad})) == BAD, (field, bad)
    for field in ("ldg", "ldu"):
        assert gated(opts=o(**{field: 7}), g=P[4], u=P[5]) == BAD
    for field in ("ldx", "ldwg", "ldwu", "ldh", "ldg", "ldu", "lddx", "lddwg", "lddwu"):
        assert backward(opts=o(**{field: 7})) == BAD and backward(opts=o(**{field: -1})) == BAD
    for field in ("lda", "ldw"):
        assert gemm_i8(**{field: 15}) == BAD and gemm_i8(**{field: 24}) == BAD  # too short; off 16 bytes
    assert gemm_i8(K=15) == BAD  # dense rows of 15 bytes
    assert gemm_i8(ldc=7) == BAD and gated_i8(opts=o(ldh=7)) == BAD and gated_i8(opts=o(ldwu=24)) == BAD
    assert quantize(ldx=7) == BAD and quantize(ldq=7) == BAD


def test_overlaps():
    M = N = K = 64
    for src in (P[0], P[1], P[2]):
        assert gated(M, N, K, h=src + 2 * M * K - 2) == BAD
    assert gated(M, N, K, g=P[3] + 128, u=P[5]) == BAD           # G inside H
    assert gated(M, N, K, g=P[4], u=P[4] + 2 * M * N - 2) == BAD  # U on G's last element
    for src in P[:6]:
        assert backward(M, N, K, dx=src) == BAD
    assert backward(M, N, K, dwg=P[6]) == BAD and backward(M, N, K, dwu=P[7] + 2) == BAD
    assert backward(M, N, K, ws=P[0]) == BAD and backward(M, N, K, ws=P[8] - 256) == BAD
    assert gemm_i8(M, N, K, c=P[0]) == BAD and gemm_i8(M, N, K, c=P[1] + 4) == BAD and gemm_i8(M, N, K, bias=P[4]) == BAD
    assert gated_i8(M, N, K, h=P[5]) == BAD
    assert quantize(M, K, q=P[0] + 2) == BAD and quantize(M, K, s=P[1]) == BAD and quantize(M, K, s=P[0]) == BAD


def test_workspace_sizes():
    def up(n):
        return (n + 255) // 256 * 256
    M, N, K = 100, 41, 33
    # Rows of 33 elements are off 16 bytes: x and both weights are copied into rows of 40.
    assert tg.gated_workspace_size(*P[:3], M, N, K) == up(2 * M * 40) + 2 * up(2 * N * 40)
    assert tg.gated_workspace_size(*P[:3], M, N, 40) == 0
    assert tg.gated_workspace_size(P[0] + 2, *P[1:3], M, N, 40) == up(2 * M * 40)
    assert tg.gated_workspace_size(*P[:3], M, N, 40, tg.gated_options(ldwu=44)) == up(2 * N * 40)
    assert tg.gated_workspace_size(*P[:3], 1, N, 40, tg.gated_options(ldx=41)) == 0  # one row has no stride
    half = up(2 * M * 48)
    assert tg.gated_backward_workspace_size(*P[:6], M, N, 40) == 2 * half
    assert tg.gated_backward_workspace_size(*P[:6], M, N, K) == 2 * half + up(2 * M * 40) + 2 * up(2 * N * 40)
    assert tg.gated_backward_workspace_size(*P[:3], 0, *P[4:6], M, N, K) == 2 * half + up(2 * M * 40)
    assert tg.gated_backward_workspace_size(*P[:4], 0, 0, M, N, K) == 2 * half + 2 * up(2 * N * 40)
    for sizes in ((0, N, K), (M, 0, K), (M, N, 0)):
        assert tg.gated_workspace_size(*P[:3], *sizes) == 0
        assert tg.gated_backward_workspace_size(*P[:6], *sizes) == 0


def test_workspace_refusals():
    M, N, K = 100, 41, 33
    need = tg.gated_workspace_size(*P[:3], M, N, K)
    assert gated(M, N, K) == BAD                                      # none given
    assert gated(M, N, K, ws=P[9], ws_bytes=need - 1) == BAD          # too small
    assert gated(M, N, K, ws=P[9] + 128, ws_bytes=need) == BAD        # not 256-byte aligned
    assert gated(M, N, K, ws=P[3] - 256, ws_bytes=need) == BAD        # overlaps H
    assert gated(M, N, K, ws=0, ws_bytes=need) == BAD
    assert gated(ws=P[9], ws_bytes=-1) == BAD
    need = tg.gated_backward_workspace_size(*P[1:4], *P[6:9], M, N, K)
    assert backward(M, N, K, ws_bytes=need - 1) == BAD and backward(M, N, K, ws=P[9] + 64) == BAD
    assert backward(M, N, K, ws=0, ws_bytes=0) == BAD


def test_empty_calls_need_no_pointers():
    assert tg.gated_raw(0, 0, 0, 0, 0, 0, 0, 8, 8) == Status.OK
    assert tg.gated_raw(0, 0, 0, 0, 0, 0, 8, 0, 8) == Status.OK
    assert backward(dx=0, dwg=0, dwu=0) == Status.OK                   # nothing asked for
    assert tg.gemm_i8_raw(0, 0, 0, 0, 0, 0, 0, 8, 16) == Status.OK
    assert tg.gated_i8_raw(0, 0, 0, 0, 0, 0, 0, 8, 0, 16) == Status.OK
    assert tg.quantize_rows_i8_raw(0, 0, 0, 0, 8) == Status.OK


def test_valid_calls_reach_the_device():
    if _gpu():
        pytest.skip("fake addresses must not reach a device")
    want = Status.UNSUPPORTED_DEVICE
    assert gated() == want and gated(g=P[4], u=P[5]) == want and backward() == want
    assert gemm_i8() == want and gemm_i8(bias=P[5], relu=True, type=tg.TYPE_BF16) == want
    assert gated_i8() == want and quantize() == want and quantize(type=tg.TYPE_BF16, ldx=11, ldq=9) == want
    need = tg.gated_workspace_size(*P[:3], 100, 41, 33)
    assert gated(100, 41, 33, ws=P[9], ws_bytes=need) == want


def test_compiled_refusals():
    """The compiled calls raise and go on raising (in a process of their own: two C++ runtimes in one process
    end it at the third exception), and keep no reference to what they refused."""
    pytest.importorskip("torch")
    code = """
import sys, torch
from tiled_dense_gemm_fp16_b200 import feedforward
calls, x = feedforward._calls, torch.zeros(4, 16)
def refused(error, f, *args):
    try:
        f(*args)
    except error:
        return
    raise SystemExit(f"{f.__name__} took its arguments")
before = sys.getrefcount(x)
for i in range(100):
    refused(ValueError, calls.gated, x, x, x, "silu", None, False, "auto")
    refused(TypeError, calls.gated, None, x, x, "silu", None, False, "auto")
    refused(TypeError, calls.gated, x, x, x)
    refused(ValueError, calls.gated_backward, x, x, x, x, x, x, "silu", True, True, True, "auto")
    refused(TypeError, calls.gated_backward, x, 0, x, x, x, x, "silu", True, True, True, "auto")
    refused(ValueError, calls.quantize_i8, x, None, None)
    refused(ValueError, calls.gemm_i8, x, x, x, x, None, False, None, None)
    refused(ValueError, calls.gated_i8, x, x, x, x, x, x, "silu", None, None)
assert sys.getrefcount(x) == before
print("done")
"""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "done", p.stderr[-2000:]


def test_python_refusals():
    import torch
    x, w = torch.zeros(4, 8, dtype=torch.float16), torch.zeros(16, 8, dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        tg.gated(x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        tg.gated_block(x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        tg.gated_backward(x, x, w, w, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        tg.quantize_i8(x)
    with pytest.raises(ValueError, match="CUDA"):
        tg.gemm_i8(x.to(torch.int8), x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        tg.gated_i8(x.to(torch.int8), x, w, w, w, w)


# ---------------------------------------------------------------------------
# The 64-bit forms that the GPU tests compare with
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
def test_reference_gradients_against_differences(act):
    import numpy as np

    import ff_ref as ref
    rng = np.random.default_rng(3)
    M, N, K = 5, 4, 6
    x, wg, wu, dh = (rng.standard_normal(s) for s in ((M, K), (N, K), (N, K), (M, N)))
    g, u = x @ wg.T, x @ wu.T
    assert np.abs(g).min() > 1e-4  # relu: no kink within a step
    grads, _ = ref.gated_backward(dh, x, wg, wu, g, u, act, "f16")

    def loss(*args):
        return float((ref.gated(*args, act, "f16")[0][0] * dh).sum())

    for i, (t, grad) in enumerate(zip((x, wg, wu), grads)):
        for at in np.ndindex(*t.shape):
            ends = []
            for d in (1e-5, -1e-5):
                args = [x.copy(), wg.copy(), wu.copy()]
                args[i][at] += d
                ends.append(loss(*args))
            assert abs((ends[0] - ends[1]) / 2e-5 - grad[at]) <= 1e-7 * (1 + abs(grad[at])), (i, at)


def test_reference_quantization():
    import numpy as np

    import ff_ref as ref
    x = np.array([[127.0, 0.5, 1.5, -2.5, -63.5], [0.0] * 5, [1.0, np.inf, 0, 0, 0], [-4.0, 1.0, 2.0, 0.0157, -0.0158]])
    q, s = ref.quantize(x)
    assert s[0] == 1.0 and list(q[0]) == [127, 0, 2, -2, -64]      # ties to even
    assert s[1] == 0.0 and not q[1].any()
    assert np.isnan(s[2]) and not q[2].any()
    assert list(q[3]) == [-127, 32, 64, 0, -1]                     # 0.0157 / (4 / 127) = 0.498..., 0.0158: 0.502
