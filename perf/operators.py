"""The feed-forward operators as they are measured: their cases, their inputs, their plain forms and the library's calls.

Five operators of one feed-forward block, from training to serving:

* ``gated``     H = act(X Wg^T) * (X Wu^T)                        (16-bit operands)
* ``train``     the same forward, then its gradients from dH      (H, dX, dWg, dWu)
* ``quantize``  rows to 8-bit integers with one scale a row
* ``gemm_i8``   8-bit integer product, a scale a token and a channel, optional bias
* ``gated_i8``  the gated forward on 8-bit integer operands

With ``own`` false, ``run`` computes in elementary torch operations; with ``own`` true it makes the
library's calls.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _case(name, op, M, N, K, dtype, act="silu", bias=False):
    return {"name": name, "op": op, "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias}


def listed():
    return [
        # One token of one sequence: both weights are streamed once, latency and bandwidth count.
        _case("gated_token", "gated", 1, 8192, 4096, "bf16"),
        # A decoding batch of 64 sequences.
        _case("gated_batch64", "gated", 64, 8192, 8192, "f16"),
        # A prompt whose sizes suit no tile and whose rows start on odd addresses.
        _case("gated_ragged", "gated", 3001, 5003, 1021, "f16", "gelu"),
        # A long prompt through an ordinary block.
        _case("gated_prompt", "gated", 4096, 8192, 4096, "f16"),
        # A fine-tuning step of a small block on a short sequence: launches count.
        _case("train_short", "train", 129, 1000, 264, "f16", "relu"),
        # A training step of an ordinary block.
        _case("train_block", "train", 8192, 8192, 4096, "bf16"),
        # The activations of a decoding batch before an 8-bit product.
        _case("quantize_batch16", "quantize", 16, 1, 8192, "f16"),
        # The activations of a long prompt (or a weight, once, row by row).
        _case("quantize_prompt", "quantize", 8192, 1, 8192, "bf16"),
        # The down projection of a decoding batch in 8 bits.
        _case("i8_batch16", "gemm_i8", 16, 8192, 8192, "f16", "none", True),
        # A long prompt through a square projection in 8 bits.
        _case("i8_prompt", "gemm_i8", 8192, 8192, 8192, "bf16", "none"),
        # The gated half of the block in 8 bits, a decoding batch.
        _case("gated_i8_batch64", "gated_i8", 64, 8192, 4096, "f16"),
        # The same on a prompt whose sizes suit no tile.
        _case("gated_i8_ragged", "gated_i8", 3001, 5003, 1021, "bf16", "gelu"),
    ]


#: Products per output element and pass, in M * N * K multiply-adds.
PRODUCTS = {"gated": 2, "train": 6, "quantize": 0, "gemm_i8": 1, "gated_i8": 2}


def _flops(c):
    return 2 * PRODUCTS[c["op"]] * c["M"] * c["N"] * c["K"]


def _log_size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gated", "train", "quantize", "gemm_i8", "gated_i8"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "quantize":
        c = _case("", op, _log_size(rng, 1, 8192), 1, _log_size(rng, 64, 8192), dtype)
    else:
        act = rng.choice(["silu", "gelu", "relu"]) if op != "gemm_i8" else rng.choice(["none", "relu"])
        while True:
            M = _log_size(rng, 16 if op == "train" else 1, 8192)
            N, K = _log_size(rng, 64, 8192), _log_size(rng, 64, 8192)
            if rng.random() < 0.5:  # widths are multiples of eight as often as not
                N, K = (N + 7) // 8 * 8, (K + 7) // 8 * 8
            c = _case("", op, M, N, K, dtype, act, op == "gemm_i8" and rng.random() < 0.5)
            if _flops(c) <= PRODUCTS[op] * 2 * 8192 * 8192 * 4096:
                break
    c.pop("name")
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _activations(gen, M, K, dtype):
    """Rows of N(0, 1) of differing magnitude, with a few channels ten times as large."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    x *= 0.25 + 1.5 * torch.rand(M, 1, generator=gen, device="cuda")
    loud = torch.rand(K, generator=gen, device="cuda") < 0.01
    return torch.where(loud, 10 * x, x).to(dtype)


def _weight(gen, N, K, dtype):
    return (torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)).to(dtype)


def _codes(x):
    """8-bit codes with rows on 16-byte boundaries, and a scale a row: what a user keeps of a weight."""
    rows, K = x.shape
    x = x.double()
    scale = (x.abs().amax(1) / 127).float()
    stored = torch.zeros(rows, (K + 15) // 16 * 16, dtype=torch.int8, device=x.device)
    stored[:, :K] = torch.round(x / scale.double().clamp_min(1e-300)[:, None]).to(torch.int8)
    return stored[:, :K], scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, M, N, K, dtype = case["op"], case["M"], case["N"], case["K"], TYPES[case["dtype"]]
    s = {"op": op, "act": case["act"], "dtype": dtype}
    x = _activations(gen, M, K, dtype)
    if op in ("gated", "train"):
        s |= {"x": x, "wg": _weight(gen, N, K, dtype), "wu": _weight(gen, N, K, dtype)}
        if op == "train":
            s["dh"] = (0.05 * torch.randn(M, N, generator=gen, device="cuda")).to(dtype)
    elif op == "quantize":
        s["x"] = x * (torch.rand(M, 1, generator=gen, device="cuda") > 0.02)  # padded tokens are rows of zeros
    else:
        s["a"], s["sa"] = _codes(x)
        s["wg"], s["sg"] = _codes(_weight(gen, N, K, torch.float32))
        if op == "gated_i8":
            s["wu"], s["su"] = _codes(_weight(gen, N, K, torch.float32))
        else:
            s["bias"] = torch.randn(N, generator=gen, device="cuda").to(dtype) if case["bias"] else None
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

GELU_A, GELU_B = math.sqrt(2 / math.pi), 0.044715


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1 + torch.tanh(GELU_A * (g + GELU_B * g * g * g)))
    return torch.where(g > 0, g, torch.zeros_like(g))


def _act_slope(g, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-g))
        return sig * (1 + g * (1 - sig))
    if act == "gelu":
        t = torch.tanh(GELU_A * (g + GELU_B * g * g * g))
        return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_A * (1 + 3 * GELU_B * g * g)
    return (g > 0).to(g.dtype)


def _product_i8(a, w):
    """The integer sums, exact in 64 bits."""
    return a.double() @ w.double().T


def _plain(s):
    op, act, dtype = s["op"], s["act"], s["dtype"]
    if op in ("gated", "train"):
        x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
        g, u = x @ wg.T, x @ wu.T
        a = _act(g, act)
        h = (a * u).to(dtype)
        if op == "gated":
            return h
        dh = s["dh"].float()
        dg, du = dh * u * _act_slope(g, act), dh * a
        return h, (dg @ wg + du @ wu).to(dtype), (dg.T @ x).to(dtype), (du.T @ x).to(dtype)
    if op == "quantize":
        x = s["x"].double()
        scale = (x.abs().amax(1) / 127).float()
        ratio = x / torch.where(scale > 0, scale.double(), 1.0)[:, None]
        return torch.round(ratio).to(torch.int8), scale
    sa, sg = s["sa"][:, None], s["sg"][None, :]
    g = _product_i8(s["a"], s["wg"]).float() * sa * sg
    if op == "gated_i8":
        u = _product_i8(s["a"], s["wu"]).float() * sa * s["su"][None, :]
        return (_act(g, act) * u).to(dtype)
    if s["bias"] is not None:
        g = g + s["bias"].float()
    return (torch.where(g > 0, g, torch.zeros_like(g)) if act == "relu" else g).to(dtype)


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _library(s):
    import tiled_dense_gemm_fp16_b200 as tg
    op, act, dtype = s["op"], s["act"], s["dtype"]
    if op == "gated":
        return tg.gated(s["x"], s["wg"], s["wu"], act=act)
    if op == "train":
        h, gate, up = tg.gated(s["x"], s["wg"], s["wu"], act=act, save=True)
        return (h, *tg.gated_backward(s["dh"], s["x"], s["wg"], s["wu"], gate, up, act=act))
    if op == "quantize":
        return tg.quantize_i8(s["x"])
    if op == "gated_i8":
        return tg.gated_i8(s["a"], s["sa"], s["wg"], s["sg"], s["wu"], s["su"], act=act, dtype=dtype)
    return tg.gemm_i8(s["a"], s["sa"], s["wg"], s["sg"], bias=s["bias"], relu=act == "relu", dtype=dtype)


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, M, N, K = case["op"], case["M"], case["N"], case["K"]
    if op == "gated":
        nbytes = 2 * (M * K + 2 * N * K + M * N)
    elif op == "train":  # x, both weights and dH in; H, dX and both weight gradients out
        nbytes = 2 * (M * K + 2 * N * K + M * N) + 2 * (M * N + M * K + 2 * N * K)
    elif op == "quantize":
        nbytes = 2 * M * K + M * K + 4 * M
    else:
        weights = 2 if op == "gated_i8" else 1
        nbytes = M * K + 4 * M + weights * (N * K + 4 * N) + 2 * M * N + (2 * N if case["bias"] else 0)
    return {"bytes": nbytes, "flops": _flops(case) if op != "quantize" else 3 * M * K}


def _sigmoid64(z):
    e = torch.exp(-z.abs())
    return torch.where(z >= 0, 1 / (1 + e), e / (1 + e))


def _gate64(g, act):
    """act(g) and its derivative, both through the logistic function."""
    if act == "relu":
        return g.clamp_min(0), (g > 0).double()
    z, dz = g, torch.ones_like(g)
    if act == "gelu":  # (1 + tanh(y)) / 2 is the logistic function of 2 y
        z = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        dz = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    p = _sigmoid64(z)
    return g * p, p + g * p * (1 - p) * dz


def exact(case, seed):
    s, op, act = prepare(case, seed), case["op"], case["act"]
    if op == "quantize":
        x = s["x"].double()
        scale = (x.abs().max(dim=1).values / 127).to(torch.float32)
        wide = scale.double().unsqueeze(1).expand_as(x)
        q = torch.where(wide > 0, (x / wide).round(), torch.zeros_like(x))
        return q.to(torch.int8), scale.double()
    if op in ("gated", "train"):
        x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
        g, u = torch.einsum("mk,nk->mn", x, wg), torch.einsum("mk,nk->mn", x, wu)
        a, slope = _gate64(g, act)
        if op == "gated":
            return a * u
        dh = s["dh"].double()
        h, dg, du = a * u, dh * u * slope, dh * a
        del g, u, a, slope, dh
        dx = torch.einsum("mn,nk->mk", dg, wg) + torch.einsum("mn,nk->mk", du, wu)
        return h, dx, torch.einsum("mn,mk->nk", dg, x), torch.einsum("mn,mk->nk", du, x)
    a = s["a"].double() * s["sa"].double().unsqueeze(1)
    g = torch.einsum("mk,nk->mn", a, s["wg"].double() * s["sg"].double().unsqueeze(1))
    if op == "gated_i8":
        u = torch.einsum("mk,nk->mn", a, s["wu"].double() * s["su"].double().unsqueeze(1))
        return _gate64(g, act)[0] * u
    if s["bias"] is not None:
        g = g + s["bias"].double()
    return g.clamp_min(0) if act == "relu" else g
