"""Grouped products and low-rank adapters as they are measured: cases, inputs, plain forms and the library's calls.

Three passes over two families, beside the dense feed-forward operators:

* ``grouped``  Y = X W_g^T with each row's group g: the rows of a group lie together (tokens sorted by expert), the
               groups' ends are on the device, as a router leaves them
* ``train``    the same forward, then its gradients from dY      (Y, dX, dW)
* ``lora``     Y = X W^T + s_r (X A_r^T) B_r^T [+ bias] with an adapter r, or none, for each row

With ``own`` false, ``run`` computes in elementary torch operations; with ``own`` true it makes the library's
calls.  ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _grouped(name, op, rows, used, groups, active, N, K, dtype):
    """``rows`` of the buffer, the first ``used`` of them in ``active`` of the ``groups``; weights are N x K."""
    return {"name": name, "op": op, "rows": rows, "used": used, "groups": groups, "active": active, "N": N, "K": K,
            "dtype": dtype}


def _lora(name, rows, N, K, rank, adapters, requests, singles, base, dtype, bias=False):
    """``requests`` with an adapter of their own, ``singles`` of them of one row, and ``base`` requests without one."""
    return {"name": name, "op": "lora", "rows": rows, "N": N, "K": K, "rank": rank, "adapters": adapters,
            "requests": requests, "singles": singles, "base": base, "dtype": dtype, "bias": bias}


def listed():
    return [
        # One token, sent to 8 of 64 experts: their weights are streamed once.
        _grouped("grouped_token", "grouped", 8, 8, 64, 8, 2048, 4096, "bf16"),
        # A decoding batch of 64 tokens with 8 experts each: nearly all experts have a few rows.
        _grouped("grouped_batch64", "grouped", 512, 512, 64, 60, 2048, 4096, "f16"),
        # A prompt whose sizes suit no tile, rows on odd addresses, an expert without rows, a buffer not quite full.
        _grouped("grouped_ragged", "grouped", 3001, 2900, 7, 6, 5003, 1021, "f16"),
        # A long prompt through the experts of the block-scaled benchmark, in 16 bits.
        _grouped("grouped_prompt", "grouped", 8192, 8192, 8, 8, 4096, 7168, "bf16"),
        # A fine-tuning step of small experts on a short sequence: launches count.
        _grouped("train_short", "train", 258, 258, 4, 4, 1000, 264, "f16"),
        # A training step of many narrow experts: short sums for every weight gradient.
        _grouped("train_narrow", "train", 8192, 8192, 64, 63, 1024, 2048, "bf16"),
        # A training step of a few ordinary experts.
        _grouped("train_block", "train", 16384, 16384, 8, 8, 4096, 4096, "bf16"),
        # One token of one request, with its adapter.
        _lora("lora_token", 1, 4096, 4096, 16, 32, 1, 1, 0, "bf16"),
        # A decoding batch of 64 requests, an adapter each.
        _lora("lora_batch64", 64, 8192, 8192, 16, 64, 64, 64, 0, "f16"),
        # A prompt in pieces with a decoding batch behind it, some requests without an adapter, odd sizes.
        _lora("lora_pieces", 1049, 5003, 2048, 32, 64, 40, 36, 3, "f16", True),
        # Prompts of eight requests through a wide projection.
        _lora("lora_prompts", 8192, 8192, 4096, 64, 16, 8, 0, 0, "bf16"),
    ]


def _log_size(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _flops(c):
    if c["op"] == "lora":
        with_adapter = c["rows"] * c["requests"] // (c["requests"] + c["base"])
        return 2 * c["rows"] * c["N"] * c["K"] + 2 * with_adapter * c["rank"] * (c["N"] + c["K"])
    return (6 if c["op"] == "train" else 2) * c["used"] * c["N"] * c["K"]


def draw(rng):
    op = rng.choice(["grouped", "train", "lora"])
    dtype = rng.choice(["f16", "bf16"])
    while True:
        N, K = _log_size(rng, 64, 8192), _log_size(rng, 64, 8192)
        if rng.random() < 0.7:  # widths are multiples of eight more often than not
            N, K = (N + 7) // 8 * 8, (K + 7) // 8 * 8
        if op == "lora":
            K = (K + 7) // 8 * 8  # as adapters' rows are stored
            rows = _log_size(rng, 1, 8192)
            requests = min(rows, _log_size(rng, 1, 64))
            base = min(rows - requests, rng.choice([0, 0, 1, 3]))
            singles = rng.choice([0, requests // 2, requests if rows == requests + base else requests - 1])
            c = _lora("", rows, N, K, 8 * rng.randint(1, 16), requests + rng.randint(0, 16), requests, singles, base,
                      dtype, rng.random() < 0.5)
            if _flops(c) <= 2 * 8192 * 8192 * 4096:
                break
        else:
            rows = _log_size(rng, 16 if op == "train" else 1, 16384)
            groups = _log_size(rng, 1, 64)
            used = rows if rng.random() < 0.7 else rng.randint(rows // 2 + 1, rows)
            active = rng.randint(1, min(groups, used))
            c = _grouped("", op, rows, used, groups, active, N, K, dtype)
            if groups * N * K <= 1 << 28 and _flops(c) <= (3 if op == "train" else 1) * 2 * 8192 * 4096 * 7168:
                break
    c.pop("name")
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _parts(gen, total, n):
    """n positive sizes that add up to ``total``, some several times as large as others."""
    if n == 0:
        return []
    weight = torch.exp(0.7 * torch.randn(n, generator=gen, dtype=torch.float64))
    edges = (torch.cumsum(weight, 0) / weight.sum() * (total - n)).round().long().tolist()
    edges[-1] = total - n
    return [1 + b - a for a, b in zip([0] + edges[:-1], edges)]


def _activations(gen, M, K, dtype):
    """Rows of N(0, 1) of differing magnitude, with a few channels ten times as large."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    x *= 0.25 + 1.5 * torch.rand(M, 1, generator=gen, device="cuda")
    loud = torch.rand(K, generator=gen, device="cuda") < 0.01
    return torch.where(loud, 10 * x, x).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    c, dtype = case, TYPES[case["dtype"]]
    M, N, K = c["rows"], c["N"], c["K"]
    s = {"op": c["op"], "dtype": dtype, "x": _activations(gen, M, K, dtype)}
    if c["op"] != "lora":
        sizes = [0] * c["groups"]
        chosen = torch.randperm(c["groups"], generator=host).tolist()[:c["active"]]
        for g, n in zip(chosen, _parts(host, c["used"], c["active"])):
            sizes[g] = n
        s["sizes"] = sizes  # the plain form's plan; the library's calls read the ends on the device
        s["ends"] = torch.tensor(sizes).cumsum(0).to(torch.int32).cuda()
        s["w"] = torch.empty(c["groups"], N, K, dtype=dtype, device="cuda")
        for w in s["w"]:
            w.copy_(torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K))
        if c["op"] == "train":
            s["dy"] = (0.05 * torch.randn(M, N, generator=gen, device="cuda")).to(dtype)
        return s
    R, rank, requests, base = c["adapters"], c["rank"], c["requests"], c["base"]
    s["w"] = (torch.randn(N, K, generator=gen, device="cuda") / math.sqrt(K)).to(dtype)
    s["a"] = (torch.randn(R, rank, K, generator=gen, device="cuda") / math.sqrt(K)).to(dtype)
    s["b"] = (0.3 * torch.randn(R, N, rank, generator=gen, device="cuda") / math.sqrt(rank)).to(dtype)
    s["scale"] = 0.5 + 1.5 * torch.rand(R, generator=gen, device="cuda")
    s["bias"] = torch.randn(N, generator=gen, device="cuda").to(dtype) if c["bias"] else None
    adapters = torch.randperm(R, generator=host).tolist()[:requests]
    runs = [(r, 1) for r in adapters[:c["singles"]]]
    long = adapters[c["singles"]:] + [-1] * base
    runs = list(zip(long, _parts(host, M - c["singles"], len(long)))) + runs  # prompts first, then the batch
    s["rows"] = []
    start = 0
    for r, n in runs:
        s["rows"].append((r, start, start + n))
        start += n
    s["index"] = torch.tensor([r for r, n in runs for _ in range(n)], dtype=torch.int32).cuda()
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _plain(s):
    x, dtype = s["x"], s["dtype"]
    if s["op"] == "lora":
        x = x.float()
        y = x @ s["w"].float().T
        for r, lo, hi in s["rows"]:
            if r >= 0:
                y[lo:hi] += s["scale"][r] * ((x[lo:hi] @ s["a"][r].float().T) @ s["b"][r].float().T)
        if s["bias"] is not None:
            y += s["bias"].float()
        return y.to(dtype)
    w, train = s["w"], s["op"] == "train"
    y = torch.zeros(x.shape[0], w.shape[1], dtype=dtype, device=x.device)
    dx, dw = (torch.zeros_like(x), torch.zeros_like(w)) if train else (None, None)
    lo = 0
    for g, n in enumerate(s["sizes"]):
        if n:
            rows, wg = x[lo:lo + n].float(), w[g].float()
            y[lo:lo + n] = rows @ wg.T
            if train:
                d = s["dy"][lo:lo + n].float()
                dx[lo:lo + n] = d @ wg
                dw[g] = d.T @ rows
        lo += n
    return (y, dx, dw) if train else y


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _library(s):
    import tiled_dense_gemm_fp16_b200 as tg
    if s["op"] == "lora":
        return tg.lora(s["x"], s["w"], s["a"], s["b"], s["index"], scale=s["scale"], bias=s["bias"])
    y = tg.grouped(s["x"], s["w"], s["ends"])
    if s["op"] == "grouped":
        return y
    return (y, *tg.grouped_backward(s["dy"], s["x"], s["w"], s["ends"]))


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# What a pass cannot do without, and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    c = case
    M, N, K = c["rows"], c["N"], c["K"]
    if c["op"] == "lora":
        values = M * K + N * K + M * N + c["requests"] * c["rank"] * (N + K) + (N if c["bias"] else 0)
        return {"bytes": 2 * values + 4 * M + 4 * c["requests"], "flops": _flops(c)}
    values = c["used"] * K + c["active"] * N * K + M * N
    if c["op"] == "train":  # dY in; dX and all of dW out
        values += c["used"] * N + M * K + c["groups"] * N * K
    return {"bytes": 2 * values + 4 * c["groups"], "flops": _flops(c)}


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if s["op"] == "lora":
        y = torch.einsum("mk,nk->mn", x, s["w"].double())
        index = s["index"].long()
        for r in sorted({int(i) for i in index.tolist()} - {-1}):
            at = torch.nonzero(index == r).flatten()
            inner = torch.einsum("mk,jk->mj", x[at], s["a"][r].double())
            y.index_add_(0, at, torch.einsum("mj,nj->mn", inner, s["b"][r].double()) * s["scale"][r].double())
        return y if s["bias"] is None else y + s["bias"].double()
    w = s["w"]
    ends = [0] + s["ends"].tolist()
    y = torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda")
    dx = torch.zeros_like(x)
    dw = torch.zeros(w.shape, dtype=torch.float64, device="cuda") if s["op"] == "train" else None
    for g in range(w.shape[0]):
        at = slice(ends[g], ends[g + 1])
        wg = w[g].double()
        y[at] = torch.einsum("mk,nk->mn", x[at], wg)
        if dw is not None:
            d = s["dy"][at].double()
            dx[at] = torch.einsum("mn,nk->mk", d, wg)
            dw[g] = torch.einsum("mn,mk->nk", d, x[at])
    return y if dw is None else (y, dx, dw)
