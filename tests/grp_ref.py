"""Grouped products and low-rank adapters in 64 bits, and how far a right 16-bit result may be from them.

As in ff_ref: half a step of the type, and the tensor core's fp32 sums, each addition of 16 products off by at most 2^-22
of the magnitudes added: (K / 16 + 4) 2^-22 sum |a||b|.  For the adapters:
  * T = scale A X is such a sum, times scale (2^-24), rounded once to the 16-bit type; its error meets |B|;
  * B T of tokens with different neighbours is summed by fused multiply-adds in two chains of rank / 2, each step off by
    2^-24, so by (rank / 8 + 4) 2^-22 |B||T|, which covers the tensor cores' rank / 16 too;
  * the sum of W X, B T and the bias adds three more roundings of 2^-24 of the magnitudes.
"""
import numpy as np

from ff_ref import check, f64, round_error, sum_error, torch_type  # noqa: F401


def bounds(sizes):
    ends = np.cumsum(sizes)
    return list(zip(ends - np.asarray(sizes), ends))


def grouped(x, w, sizes, dt):
    """Y with zeros in the rows without a group, and its tolerance."""
    y = np.zeros((x.shape[0], w.shape[1]))
    tol = np.zeros_like(y)
    for g, (lo, hi) in enumerate(bounds(sizes)):
        y[lo:hi] = x[lo:hi] @ w[g].T
        tol[lo:hi] = 1.01 * sum_error(np.abs(x[lo:hi]) @ np.abs(w[g]).T, x.shape[1]) + round_error(y[lo:hi], dt)
    return y, tol


def grouped_backward(dy, x, w, sizes, dt):
    """((dX, dW), tolerances)."""
    dx, dw = np.zeros_like(x), np.zeros_like(w)
    tx, tw = np.zeros_like(x), np.zeros_like(w)
    for g, (lo, hi) in enumerate(bounds(sizes)):
        d, r = dy[lo:hi], x[lo:hi]
        dx[lo:hi], dw[g] = d @ w[g], d.T @ r
        tx[lo:hi] = 1.01 * sum_error(np.abs(d) @ np.abs(w[g]), w.shape[1]) + round_error(dx[lo:hi], dt)
        tw[g] = 1.01 * sum_error(np.abs(d).T @ np.abs(r), hi - lo) + round_error(dw[g], dt)
    return (dx, dw), (tx, tw)


def lora(x, w, a, b, index, scale, bias, dt):
    """Y and its tolerance; scale and bias may be None."""
    M, K = x.shape
    rank = a.shape[1]
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    tol = sum_error(mag, K)
    for r in sorted(set(index.tolist())):
        if not 0 <= r < a.shape[0]:
            continue
        at = np.flatnonzero(index == r)
        s = 1.0 if scale is None else float(scale[r])
        t = s * (x[at] @ a[r].T)
        err = abs(s) * sum_error(np.abs(x[at]) @ np.abs(a[r]).T, K) + np.abs(t) * 2.0 ** -23
        err = err * 1.01 + round_error(t, dt)
        product = (np.abs(t) + err) @ np.abs(b[r]).T
        y[at] += t @ b[r].T
        mag[at] += product
        tol[at] += err @ np.abs(b[r]).T + (rank / 8 + 4) * 2.0 ** -22 * product
    if bias is not None:
        y, mag = y + bias, mag + np.abs(bias)
    tol = 1.01 * (tol + 3 * 2.0 ** -24 * mag)
    return y, tol + round_error(y, dt)
