"""Host logic of the grouped products and the adapters: sizes, strides, alignment, overlap, workspaces, refusals.  No
kernel is launched: without a GPU a call that passes every check ends in UNSUPPORTED_DEVICE."""
import ctypes
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest

import tiled_dense_gemm_fp16_b200 as tg
from tiled_dense_gemm_fp16_b200 import Status, build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x10_0000_0000 * (i + 1) for i in range(12)]  # well-separated fake device addresses (never dereferenced)
BAD = Status.INVALID_ARG
BIG = 1 << 30


def grouped(G=4, M=8, N=8, K=8, opts=None, x=P[0], w=P[1], ends=P[2], y=P[3], ws=0, ws_bytes=0):
    return tg.grouped_raw(x, w, ends, y, G, M, N, K, opts, 0, ws, ws_bytes)


def backward(G=4, M=8, N=8, K=8, opts=None, dy=P[0], x=P[1], w=P[2], ends=P[3], dx=P[4], dw=P[5], ws=0, ws_bytes=0):
    return tg.grouped_backward_raw(dy, x, w, ends, dx, dw, G, M, N, K, opts, 0, ws, ws_bytes)


def lora(M=8, N=8, K=8, rank=8, adapters=3, opts=None, x=P[0], w=P[1], a=P[2], b=P[3], scale=P[4], index=P[5], bias=P[6],
         y=P[7], ws=P[8], ws_bytes=1 << 20):
    return tg.lora_raw(x, w, a, b, scale, index, bias, y, M, N, K, rank, adapters, opts, 0, ws, ws_bytes)


def _gpu():
    import torch
    return torch.cuda.is_available()


def up(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("struct,mirror", [("tg_grouped_options", tg.GroupedOptions), ("tg_lora_options", tg.LoraOptions)])
def test_options_structs_match_the_header(struct, mirror):
    text = open(os.path.join(ROOT, "include", "tg_gemm.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\}" % struct, text, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    names = [(n, t) for t, ns in re.findall(r"(int32_t|int64_t)\s+([\w, ]+);", body) for n in ns.replace(" ", "").split(",")]
    assert [n for n, _ in names] == [f[0] for f in mirror._fields_]
    assert ctypes.sizeof(mirror) == sum(4 if t == "int32_t" else 8 for _, t in names)


@pytest.mark.parametrize("sizes", [(-1, 8, 8), (8, -1, 8), (8, 8, -1), (BIG + 1, 8, 8), (8, BIG + 1, 8), (8, 8, BIG + 1),
                                   (8, BIG, BIG), (BIG, BIG, 8)])
def test_sizes(sizes):
    M, N, K = sizes
    assert grouped(4, M, N, K) == BAD and backward(4, M, N, K) == BAD and lora(M, N, K) == BAD
    assert tg.grouped_workspace_size(P[0], P[1], 4, M, N, K) == -1 and tg.lora_workspace_size(P[0], P[1], M, N, K, 8, 3) == -1
    assert tg.grouped_backward_workspace_size(*P[:5], 4, M, N, K) == -1


def test_groups_and_ranks():
    assert grouped(-1) == BAD and grouped(1025) == BAD and backward(-1) == BAD and backward(1025) == BAD
    assert grouped(1024, 8, 1 << 25, 1 << 20) == BAD  # more elements than are counted
    for kw in ({"rank": -8}, {"rank": 12}, {"rank": 520}, {"adapters": -1}, {"adapters": (1 << 20) + 1}):
        assert lora(**kw) == BAD, kw


def test_enumerations():
    for bad in ({"type": 2}, {"type": -1}, {"reserved": 1}):
        assert grouped(opts=tg.grouped_options(**bad)) == BAD and backward(opts=tg.grouped_options(**bad)) == BAD
        assert lora(opts=tg.lora_options(**bad)) == BAD
    assert grouped(opts=tg.grouped_options(rest=2)) == BAD and grouped(opts=tg.grouped_options(rest=-1)) == BAD


def test_null_and_odd_pointers():
    for name in ("x", "w", "ends", "y"):
        assert grouped(**{name: 0}) == BAD and grouped(**{name: P[11] + 1}) == BAD, name
    for name in ("dy", "x", "w", "ends"):
        assert backward(**{name: 0}) == BAD and backward(**{name: P[11] + 1}) == BAD, name
    for name in ("dx", "dw"):
        assert backward(**{name: P[11] + 1}) == BAD, name
    for name in ("x", "w", "a", "b", "index", "y"):
        assert lora(**{name: 0}) == BAD and lora(**{name: P[11] + 1}) == BAD, name
    for name, off in (("a", 8), ("b", 8), ("scale", 2), ("index", 2), ("bias", 1)):
        assert lora(**{name: P[11] + off}) == BAD, name
    assert grouped(ends=P[2] + 2) == BAD


def test_strides():
    o = tg.grouped_options
    for field in ("ldx", "ldw", "ldy"):
        for bad in (7, -8, (1 << 38) + 8):
            assert grouped(opts=o(**{field: bad})) == BAD, (field, bad)
    for field in ("ldx", "ldw", "ldy", "lddx", "lddw"):
        assert backward(opts=o(**{field: 7})) == BAD and backward(opts=o(**{field: -1})) == BAD, field
    for bad in (7, -8, (1 << 38) + 8):
        assert grouped(opts=o(stride_w=bad)) == BAD, bad
    assert backward(opts=o(stride_dw=63)) == BAD and backward(opts=o(stride_dw=-64)) == BAD  # matrices of 8 x 8 would overlap
    for field in ("ldx", "ldw", "ldy", "lda", "ldb", "stride_a", "stride_b"):
        assert lora(opts=tg.lora_options(**{field: 7})) == BAD and lora(opts=tg.lora_options(**{field: -8})) == BAD, field
    for field in ("lda", "ldb", "stride_a", "stride_b"):
        assert lora(opts=tg.lora_options(**{field: 68})) == BAD, field  # off 16 bytes
    assert lora(K=12) == BAD and lora(K=12, opts=tg.lora_options(lda=12)) == BAD  # rows of A of 24 bytes


def test_overlaps():
    G, M, N, K = 4, 64, 64, 64
    for src in (P[0], P[1], P[2]):
        assert grouped(G, M, N, K, y=src) == BAD
    assert grouped(G, M, N, K, y=P[1] + 2 * G * N * K - 2) == BAD        # the last weight's last element
    for src in (P[0], P[1], P[2], P[3]):
        assert backward(G, M, N, K, dx=src) == BAD and backward(G, M, N, K, dw=src) == BAD
    assert backward(G, M, N, K, dw=P[4]) == BAD
    for src in (P[0], P[1], P[2], P[3], P[4], P[5], P[6]):
        assert lora(M, N, K, y=src) == BAD
    assert lora(M, N, K, ws=P[7]) == BAD and lora(M, N, K, ws=P[2]) == BAD


def test_workspace_sizes():
    G, M, N, K = 5, 100, 41, 33
    size = tg.grouped_workspace_size
    assert size(*P[:2], G, M, N, K) == up(2 * M * 40) + up(2 * G * N * 40)
    assert size(*P[:2], G, M, N, 40) == 0 and size(P[0] + 2, P[1], G, M, N, 40) == up(2 * M * 40)
    assert size(*P[:2], G, M, N, 40, tg.grouped_options(ldw=44)) == up(2 * G * N * 40)
    assert size(*P[:2], G, M, N, 40, tg.grouped_options(stride_w=44 * 40)) == 0
    assert size(*P[:2], G, M, N, 40, tg.grouped_options(stride_w=44 * 40 + 1)) == -1  # uneven rows that TMA cannot take
    grad = tg.grouped_backward_workspace_size
    dy, x, w = up(2 * M * 48), up(2 * M * 40), up(2 * G * N * 40)
    assert grad(*P[:5], G, M, N, K) == dy + x + w
    assert grad(*P[:3], 0, P[4], G, M, N, K) == dy + x and grad(*P[:4], 0, G, M, N, K) == dy + w
    assert grad(*P[:5], G, M, 48, 40) == 0
    inner = up(2 * M * 16) + up(4 * 4)
    assert tg.lora_workspace_size(*P[:2], M, N, 40, 16, 3) == inner
    assert tg.lora_workspace_size(*P[:2], M, N, K, 16, 3) == inner + up(2 * M * 40) + up(2 * N * 40)
    assert tg.lora_workspace_size(*P[:2], M, N, 40, 0, 3) == 0 and tg.lora_workspace_size(*P[:2], M, N, 40, 16, 0) == 0
    for sizes in ((0, N, K), (M, 0, K), (M, N, 0)):
        assert size(*P[:2], G, *sizes) == 0 and grad(*P[:5], G, *sizes) == 0 and tg.lora_workspace_size(*P[:2], *sizes, 8, 3) == 0
    assert size(*P[:2], 0, M, N, K) == 0


def test_weights_of_one_row():
    """The row of each weight may lie anywhere: the distance between the weights is all that TMA or a copy needs."""
    size = tg.grouped_workspace_size
    assert size(*P[:2], 3, 16, 1, 5, tg.grouped_options(ldx=8, stride_w=8)) == 0
    assert size(*P[:2], 3, 16, 1, 5, tg.grouped_options(ldx=8, stride_w=7)) == up(2 * 3 * 8)
    assert size(*P[:2], 3, 16, 1, 5, tg.grouped_options(ldx=8, ldw=16)) == 0
    assert size(*P[:2], 3, 16, 1, 8, tg.grouped_options(stride_w=9)) == up(2 * 3 * 8)


def test_copies_of_many_rows():
    """Rows of all weights are counted in 32 bits, and so are the steps over them."""
    size = tg.grouped_workspace_size
    assert size(*P[:2], 1000, 8, 2147000, 1) == up(2 * 8 * 8) + up(2 * 8 * 2147000000)
    assert size(*P[:2], 1024, 8, 2097151, 1) == -1 and size(*P[:2], 1024, 8, 1 << 22, 1) == -1
    assert size(*P[:2], 1024, 8, 2097151, 8) == 0  # no copy


def test_workspace_refusals():
    G, M, N, K = 5, 100, 41, 33
    need = tg.grouped_workspace_size(*P[:2], G, M, N, K)
    assert grouped(G, M, N, K) == BAD and grouped(G, M, N, K, ws=P[9], ws_bytes=need - 1) == BAD
    assert grouped(G, M, N, K, ws=P[9] + 128, ws_bytes=need) == BAD and grouped(G, M, N, K, ws=P[3] - 256, ws_bytes=need) == BAD
    assert grouped(ws=P[9], ws_bytes=-1) == BAD
    need = tg.grouped_backward_workspace_size(*P[:3], *P[4:6], G, M, N, K)
    assert backward(G, M, N, K, ws=P[9], ws_bytes=need - 1) == BAD
    need = tg.lora_workspace_size(*P[:2], M, N, 40, 16, 3)
    assert lora(M, N, 40, 16, ws_bytes=need - 1) == BAD and lora(M, N, 40, 16, ws=P[8] + 64) == BAD and lora(M, N, 40, 16, ws=0, ws_bytes=0) == BAD


def test_empty_calls_need_no_pointers():
    assert tg.grouped_raw(0, 0, 0, 0, 4, 0, 8, 8) == Status.OK and tg.grouped_raw(0, 0, 0, 0, 4, 8, 0, 8) == Status.OK
    assert backward(dx=0, dw=0) == Status.OK and backward(0, 8, 8, 8, dx=0) == Status.OK
    assert tg.lora_raw(0, 0, 0, 0, 0, 0, 0, 0, 0, 8, 8, 8, 3) == Status.OK
    assert tg.lora_raw(0, 0, 0, 0, 0, 0, 0, 0, 8, 0, 8, 8, 3) == Status.OK


def test_valid_calls_reach_the_device():
    if _gpu():
        pytest.skip("fake addresses must not reach a device")
    want = Status.UNSUPPORTED_DEVICE
    assert grouped() == want and backward() == want and backward(dx=0) == want and backward(dw=0) == want
    assert grouped(opts=tg.grouped_options(type=tg.TYPE_BF16, rest=1, ldx=16, ldw=24, ldy=11, stride_w=1000)) == want
    assert grouped(G=0) == want and grouped(K=0, opts=tg.grouped_options(rest=1)) == want
    assert lora() == want and lora(scale=0, bias=0) == want and lora(adapters=0, a=0, b=0, index=0, ws=0, ws_bytes=0) == want
    assert lora(rank=512, ws_bytes=1 << 24) == want and lora(K=12, opts=tg.lora_options(lda=16), ws_bytes=1 << 24) == want
    need = tg.grouped_workspace_size(*P[:2], 5, 100, 41, 33)
    assert grouped(5, 100, 41, 33, ws=P[9], ws_bytes=need) == want


def test_python_refusals():
    import torch
    x, w, ends = torch.zeros(4, 8).half(), torch.zeros(3, 16, 8).half(), torch.tensor([1, 2, 4], dtype=torch.int32)
    a, b = torch.zeros(2, 8, 8).half(), torch.zeros(2, 16, 8).half()
    for call in (lambda: tg.grouped(x, w, ends), lambda: tg.grouped_linear(x, w, ends), lambda: tg.grouped_backward(x, x, w, ends),
                 lambda: tg.lora(x, w[0], a, b, torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_forward_mode_is_refused():
    import torch
    from torch.autograd import forward_ad
    x, w, ends = torch.ones(4, 8).half(), torch.ones(3, 16, 8).half(), torch.tensor([1, 2, 4], dtype=torch.int32)
    with forward_ad.dual_level():
        for i in range(2):
            args = [x, w]
            args[i] = forward_ad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(NotImplementedError, match="forward-mode"):
                tg.grouped_linear(*args, ends)


def test_compiled_refusals():
    """The compiled calls raise and go on raising (in a process of their own), and keep no reference to what they refused."""
    pytest.importorskip("torch")
    code = """
import sys, torch
from tiled_dense_gemm_fp16_b200 import experts
calls, x = experts._calls, torch.zeros(4, 16)
def refused(error, f, *args):
    try:
        f(*args)
    except error:
        return
    raise SystemExit(f"{f.__name__} took its arguments")
before = sys.getrefcount(x)
for i in range(100):
    refused(ValueError, calls.grouped, x, x, x, None, "auto")
    refused(TypeError, calls.grouped, None, x, x, None, "auto")
    refused(TypeError, calls.grouped, x, x)
    refused(ValueError, calls.grouped_backward, x, x, x, x, True, True, "auto")
    refused(ValueError, calls.lora, x, x, x, x, x, None, None, None, "auto")
    refused(TypeError, calls.lora, 0, x, x, x, x, None, None, None, "auto")
assert sys.getrefcount(x) == before
print("done")
"""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0 and p.stdout.strip() == "done", p.stderr[-2000:]


# ---------------------------------------------------------------------------
# How a group is cut into tiles: the kernels' own function in a small host program
# ---------------------------------------------------------------------------

PROGRAM = """
#include <cstdio>
#include "grp_ops.cuh"
int main() {
  const int most[][2] = {{256, 32}, {224, 32}, {192, 32}, {160, 32}, {128, 32}, {96, 32}, {128, 16}, {64, 16}, {32, 16}, {16, 16}};
  for (auto& m : most)
    for (int rows = 1; rows <= 1200; ++rows) {
      const tg::GrpCut c = tg::grp_cut(rows, m[0], m[1]);
      int at = 0;
      for (int i = 0; i < c.tiles; ++i) {
        int first, count;
        tg::grp_cut_tile(c, rows, m[0], i, first, count);
        if (first != at || count < 1 || count > m[0] || first % m[1] != 0) return std::printf("%d %d: tile %d\\n", m[0], rows, i), 1;
        at += count;
      }
      if (at != rows || c.tiles != (rows + m[0] - 1) / m[0]) return std::printf("%d %d\\n", m[0], rows), 1;
    }
  std::printf("ok\\n");
}
"""


def test_tiles_cover_their_group(tmp_path):
    nvcc = build._nvcc()
    if not (os.path.exists(nvcc) or shutil.which(nvcc)):
        pytest.skip("no nvcc")
    source, program = tmp_path / "cut.cu", tmp_path / "cut"
    source.write_text(PROGRAM)
    subprocess.run([nvcc, *build.ARCH, "-std=c++17", f"-I{build.CSRC}", f"-I{os.path.join(build.ROOT, 'include')}", str(source),
                    "-o", str(program)], check=True, timeout=600)
    p = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert p.returncode == 0 and p.stdout.strip() == "ok", p.stdout


# ---------------------------------------------------------------------------
# The 64-bit forms that the GPU tests compare with
# ---------------------------------------------------------------------------

def test_reference_gradients_against_differences():
    import grp_ref as ref
    rng = np.random.default_rng(3)
    sizes, N, K = [2, 0, 3], 4, 3
    x, w, dy = rng.standard_normal((6, K)), rng.standard_normal((3, N, K)), rng.standard_normal((6, N))
    grads, _ = ref.grouped_backward(dy, x, w, sizes, "f16")
    for i, (t, grad) in enumerate(zip((x, w), grads)):
        for at in np.ndindex(*t.shape):
            ends = []
            for d in (1e-5, -1e-5):
                args = [x.copy(), w.copy()]
                args[i][at] += d
                ends.append(float((ref.grouped(*args, sizes, "f16")[0] * dy).sum()))
            assert abs((ends[0] - ends[1]) / 2e-5 - grad[at]) <= 1e-8 * (1 + abs(grad[at])), (i, at)


def test_reference_adapters():
    import grp_ref as ref
    rng = np.random.default_rng(4)
    x, w, a, b = (rng.standard_normal(s) for s in ((5, 6), (3, 6), (2, 8, 6), (2, 3, 8)))
    index, scale = np.array([1, -1, 0, 2, 1]), np.array([0.5, 2.0])
    y, tol = ref.lora(x, w, a, b, index, scale, np.ones(3), "f16")
    for m, r in enumerate(index):
        own = w + (scale[r] * b[r] @ a[r] if 0 <= r < 2 else 0)
        assert np.abs(y[m] - own @ x[m] - 1).max() < 1e-12
    assert (tol > 0).all() and (tol < 0.1 * (1 + np.abs(y))).all()
