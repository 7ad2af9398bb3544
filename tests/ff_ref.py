"""The feed-forward operators in 64 bits, and how far a right 16-bit result may be from them.

A result may differ from its definition by
  * half a step of its type, relative (fp16 2^-11, bf16 2^-8), or of fp16's subnormals (2^-25);
  * the fp32 sum: the tensor core adds 16 products (32 bytes of K) at a time, each addition off by at
    most 2^-22 of the magnitudes added, so a sum of K products by (K / 16 + 4) 2^-22 sum |a||b|;
  * the activation: |act'| <= 1.13 carries an error of G over, and the fast exponential and division
    and the products around them are good to 2^-19, relative to |act(g)| (g times a logistic value).
"""
import numpy as np

HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}
SLOPE = 1.13        # largest |act'| of the three activations
FAST = 2.0 ** -19   # activation arithmetic, relative
GELU_A, GELU_B = np.sqrt(2 / np.pi), 0.044715


def torch_type(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def f64(t):
    return t.detach().cpu().double().numpy()


def logistic(z):
    e = np.exp(-np.abs(z))
    return np.where(z >= 0, 1 / (1 + e), e / (1 + e))


def act(g, name):
    """act(g) and its derivative."""
    if name == "relu":
        return np.where(g > 0, g, 0.0), (g > 0).astype(np.float64)
    z, dz = (g, 1.0) if name == "silu" else (2 * GELU_A * (g + GELU_B * g ** 3), 2 * GELU_A * (1 + 3 * GELU_B * g ** 2))
    p = logistic(z)
    return g * p, p + g * p * (1 - p) * dz


def sum_error(abs_sum, K):
    return (K / 16 + 4) * 2.0 ** -22 * abs_sum


def round_error(ref, dt):
    return HALF[dt] * np.abs(ref) + TINY[dt]


def gated(x, wg, wu, name, dt):
    """(H, G, U) in 64 bits and their tolerances."""
    K = x.shape[1]
    g, u = x @ wg.T, x @ wu.T
    dg, du = (sum_error(np.abs(x) @ np.abs(w).T, K) for w in (wg, wu))
    return gate(g, u, dg, du, name, dt)


def gate(g, u, dg, du, name, dt):
    a, _ = act(g, name)
    h = a * u
    tol_h = (SLOPE * dg + FAST * np.abs(a)) * (np.abs(u) + du) + np.abs(a) * du
    tol_h = tol_h * (1 + HALF[dt]) + round_error(h, dt)
    return (h, g, u), (tol_h, dg * 1.01 + round_error(g, dt), du * 1.01 + round_error(u, dt))


def gated_backward(dh, x, wg, wu, g, u, name, dt):
    """(dX, dWg, dWu) in 64 bits from the stored 16-bit G and U, and their tolerances.

    dG and dU are rounded to the 16-bit type before the products.  The slope's terms are at most 1.13 in
    all, its arithmetic good to 2^-18 absolutely."""
    M, K = x.shape
    N = wg.shape[0]
    a, s = act(g, name)
    dg, du = dh * u * s, dh * a
    err_g = np.abs(dh * u) * 2.0 ** -18
    err_g = err_g * (1 + HALF[dt]) + round_error(dg, dt)
    err_u = FAST * np.abs(dh * a) + round_error(du, dt)
    dx = dg @ wg + du @ wu
    abs_x = np.abs(dg) @ np.abs(wg) + np.abs(du) @ np.abs(wu)
    tol_x = err_g @ np.abs(wg) + err_u @ np.abs(wu)
    tol_x = 1.01 * (tol_x + sum_error(abs_x, 2 * N)) + round_error(dx, dt)
    outs, tols = [dx], [tol_x]
    for d, err in ((dg, err_g), (du, err_u)):
        w = d.T @ x
        outs.append(w)
        tols.append(1.01 * (err.T @ np.abs(x) + sum_error(np.abs(d).T @ np.abs(x), M)) + round_error(w, dt))
    return outs, tols


def quantize(x):
    """Codes and fp32 scales of the rows of x (64-bit values of a 16-bit type)."""
    scale = np.zeros(x.shape[0], np.float32)
    q = np.zeros(x.shape, np.int8)
    for m, row in enumerate(x):
        if not np.all(np.isfinite(row)):
            scale[m] = np.nan
            continue
        scale[m] = np.float32(np.abs(row).max(initial=0.0)) / np.float32(127)
        if scale[m] > 0:
            q[m] = np.rint(row / np.float64(scale[m])).astype(np.int8)
    return q, scale


def i8_product(a, sa, w, sw):
    """The scaled product in 64 bits and its error in fp32: three roundings of 2^-24."""
    c = (a.astype(np.float64) @ w.astype(np.float64).T) * sa.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :]
    return c, np.abs(c) * 2.0 ** -22


def check(got, ref, tol, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape}, want {ref.shape}"
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (f"{what}: {len(bad)} of {ref.size} outside, first at {tuple(bad[0])}: got {got[tuple(bad[0])]}, "
                           f"want {ref[tuple(bad[0])]} +- {tol[tuple(bad[0])]}")
