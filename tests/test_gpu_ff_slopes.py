"""Gradients of the gated block against difference quotients of its forward pass, both taken with the library's calls,
in directions where each term of a gradient is at least ten times what the comparison can be off by.

With v = sign of the 64-bit gradient of one operand P, the slope is S = <dP, v> and the quotient Q = <H(P + t v) - H(P -
t v), dH> / 2t.  They may differ by
  * the quotient's curvature, which halving the step shows (central differences: the error falls to a quarter, so it is
    at most 4/3 of the change; 2 is taken);
  * roundings, each off by at most c_i = half a step of its type times what S or Q depends on it: H at both ends, the
    stored G and U, dG and dU, dP.  They are independent, so their sum passes 6 sqrt(sum c_i^2) with a chance below
    2 exp(-18) = 3e-8 (Hoeffding);
  * the fp32 arithmetic (sums, activations), all of one sign at worst: its bounds of ff_ref.py, added up.
"""
import numpy as np
import pytest

import ff_ref as ref

M, N, K = 48, 160, 96
STEP = {"x": 1 / 16, "wg": 1 / 64, "wu": 1 / 64}
GRID = {"x": 1 / 64, "wg": 1 / 512, "wu": 1 / 512}  # of the values, so that both ends are exact in either type


def operands(dt):
    rng = np.random.default_rng(11)
    t = {"x": rng.standard_normal((M, K)), "wg": rng.standard_normal((N, K)) * 0.1, "wu": rng.standard_normal((N, K)) * 0.1}
    # bf16 has 8 bits: values below 2 on a grid of 1/64, weights below 1/2 on one of 1/512.
    most = {"x": 1.75, "wg": 0.4375, "wu": 0.4375}
    t = {n: np.clip(np.round(v / GRID[n]) * GRID[n], -most[n], most[n]) for n, v in t.items()}
    dh = np.round(rng.standard_normal((M, N)) * 16) / 16
    return t, np.clip(dh, -2, 2)


def gradients(t, dh, act):
    """64-bit gradients, term by term, at the 64-bit G and U; and what each depends on."""
    g, u = t["x"] @ t["wg"].T, t["x"] @ t["wu"].T
    a, s = ref.act(g, act)
    dg, du = dh * u * s, dh * a
    return g, u, a, s, dg, du, {"x": (dg @ t["wg"], du @ t["wu"]), "wg": (dg.T @ t["x"],), "wu": (du.T @ t["x"],)}


def allowance(t, dh, act, dt, name, v):
    """(bound, the slope's terms) of one operand in the direction v."""
    half = ref.HALF[dt]
    g, u, a, s, dg, du, terms = gradients(t, dh, act)
    terms = terms[name]
    # What S = sum dG P + dU Q depends on: P and Q are the changes of G and U along v.
    P = {"x": v @ t["wg"].T, "wg": t["x"] @ v.T, "wu": np.zeros_like(g)}[name]
    Q = {"x": v @ t["wu"].T, "wg": np.zeros_like(g), "wu": t["x"] @ v.T}[name]
    e = 1e-5
    bend = (ref.act(g + e, act)[1] - ref.act(g - e, act)[1]) / (2 * e)  # act''
    step = STEP[name]
    ends = [ref.gated(*({**t, name: t[name] + d * step * v}[n] for n in ("x", "wg", "wu")), act, dt) for d in (1, -1)]
    roundings = [half * np.abs(g) * np.abs(dh * (u * bend * P + s * Q)), half * np.abs(u) * np.abs(dh * s * P),
                 half * np.abs(dg * P), half * np.abs(du * Q), half * np.abs(sum(terms)) * np.abs(v)]
    roundings += [ref.round_error(outs[0], dt) * np.abs(dh) / (2 * step) for outs, _ in ends]
    spread = 6 * np.sqrt(sum((c ** 2).sum() for c in roundings))
    arithmetic = sum(((tols[0] - ref.round_error(outs[0], dt)).clip(0) * np.abs(dh)).sum() / (2 * step) for outs, tols in ends)
    arithmetic += (2.0 ** -18 * np.abs(dh * u * P)).sum() + (ref.FAST * np.abs(dh * a * Q)).sum()
    abs_sum = {"x": np.abs(dg) @ np.abs(t["wg"]) + np.abs(du) @ np.abs(t["wu"]), "wg": np.abs(dg).T @ np.abs(t["x"]),
               "wu": np.abs(du).T @ np.abs(t["x"])}[name]
    arithmetic += ref.sum_error(abs_sum, {"x": 2 * N, "wg": M, "wu": M}[name]).sum()

    def quotient(d):
        a, b = (ref.gated(*({**t, name: t[name] + z * d * v}[n] for n in ("x", "wg", "wu")), act, dt)[0][0] for z in (1, -1))
        return ((a - b) * dh).sum() / (2 * d)

    curve = 2 * abs(quotient(step) - quotient(step / 2))
    return 1.01 * (spread + arithmetic + curve), [float((x * v).sum()) for x in terms]


CASES = [(n, a, d) for n in ("x", "wg", "wu") for a in ("silu", "gelu") for d in ("f16", "bf16")]


@pytest.mark.parametrize("name,act,dt", CASES)
def test_directions_tell(name, act, dt):
    """On the CPU: a gradient that misses any of its terms, or has it doubled, would be outside by far."""
    t, dh = operands(dt)
    v = np.sign(sum(gradients(t, dh, act)[-1][name]))
    bound, terms = allowance(t, dh, act, dt, name, v)
    assert all(abs(x) > 10 * bound for x in terms), (bound, terms)


@pytest.mark.gpu
@pytest.mark.parametrize("name,act,dt", CASES)
def test_slopes_are_quotients(name, act, dt):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    t, dh = operands(dt)
    v = np.sign(sum(gradients(t, dh, act)[-1][name]))
    bound, _ = allowance(t, dh, act, dt, name, v)

    def device(a):
        d = torch.from_numpy(a).cuda().to(ref.torch_type(dt))
        assert np.array_equal(ref.f64(d), a)
        return d

    at = {n: device(a) for n, a in t.items()}
    dhd = device(dh)
    _, g, u = tg.gated(*at.values(), act=act, save=True)
    grads = dict(zip(at, tg.gated_backward(dhd, *at.values(), g, u, act=act)))
    ends = [tg.gated(*({**at, name: device(t[name] + d * STEP[name] * v)}).values(), act=act) for d in (1, -1)]
    torch.cuda.synchronize()
    assert tg.device_status()[0] == tg.Status.OK
    slope = float((ref.f64(grads[name]) * v).sum())
    quotient = float(((ref.f64(ends[0]) - ref.f64(ends[1])) * dh).sum() / (2 * STEP[name]))
    assert abs(slope - quotient) <= bound, (slope, quotient, bound)
