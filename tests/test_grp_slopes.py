"""Gradients of the grouped product against difference quotients that tell: the step goes along the gradient's signs, so the
slope is the sum of its magnitudes, far above what roundings allow.  The product is linear in x and in w, so a quotient has no
error of its own.  All values lie on grids on which the steps are exact in either type."""
import numpy as np
import pytest

import grp_ref as ref

M, SIZES, N, K = 101, [40, 0, 56], 64, 48
STEP = {"x": 1.0, "w": 2.0 ** -3}
CASES = [(n, d) for n in ("x", "w") for d in ("f16", "bf16")]


def _operands():
    rng = np.random.default_rng(7)
    grid = lambda shape, sigma, unit: np.clip(np.rint(rng.normal(0, sigma, shape) / unit), -48, 48) * unit  # noqa: E731
    return {"x": grid((M, K), 1.0, 2.0 ** -4), "w": grid((len(SIZES), N, K), K ** -0.5, 2.0 ** -6)}, grid((M, N), 1.0, 2.0 ** -4)


def _gradients(t, dy, dt):
    grads, tols = ref.grouped_backward(dy, t["x"], t["w"], SIZES, dt)
    return dict(zip(("x", "w"), grads)), dict(zip(("x", "w"), tols))


def _allowance(t, dy, dt, name, v):
    """How far a slope along v from right 16-bit gradients may be from a quotient of right 16-bit outputs."""
    allowed = (_gradients(t, dy, dt)[1][name] * np.abs(v)).sum()
    for z in (1, -1):
        _, tol = ref.grouped(*({**t, name: t[name] + z * STEP[name] * v}[n] for n in ("x", "w")), SIZES, dt)
        allowed += (tol * np.abs(dy)).sum() / (2 * STEP[name])
    return 1.01 * allowed


@pytest.mark.parametrize("name,dt", CASES)
def test_directions_tell(name, dt):
    """On the CPU: no gradient, half of it, twice it, its negative, another group's or one that misses a row is outside by far."""
    t, dy = _operands()
    g = _gradients(t, dy, dt)[0][name]
    v = np.sign(g)
    bound = _allowance(t, dy, dt, name, v)
    wrong = {"none": 0 * g, "half": g / 2, "twice": 2 * g, "negative": -g}
    if name == "x":
        lost = g.copy()
        lost[:4] = 0
        other = g.copy()
        other[:40] = dy[:40] @ t["w"][2]
    else:
        lost = g.copy()
        lost[0] -= dy[:4].T @ t["x"][:4]
        other = g[::-1]
    wrong.update(rows=lost, other=other)
    right = (g * v).sum()
    y = [ref.grouped(*({**t, name: t[name] + z * STEP[name] * v}[n] for n in ("x", "w")), SIZES, dt)[0] for z in (1, -1)]
    assert abs(((y[0] - y[1]) * dy).sum() / (2 * STEP[name]) - right) < 1e-9 * right
    for what, w in wrong.items():
        assert abs((w * v).sum() - right) > 2 * bound, (what, (w * v).sum(), right, bound)
    for what in ("none", "half", "twice", "negative"):
        assert abs((wrong[what] * v).sum() - right) > 20 * bound, (what, bound)


@pytest.mark.gpu
@pytest.mark.parametrize("name,dt", CASES)
def test_slopes_are_quotients(name, dt):
    import torch
    import tiled_dense_gemm_fp16_b200 as tg
    t, dy = _operands()
    v = np.sign(_gradients(t, dy, dt)[0][name])
    bound = _allowance(t, dy, dt, name, v)

    def device(a):
        d = torch.from_numpy(a).cuda().to(ref.torch_type(dt))
        assert np.array_equal(ref.f64(d), a)
        return d

    ends = torch.from_numpy(np.cumsum(SIZES).astype(np.int32)).cuda()
    at, dyd = {n: device(a) for n, a in t.items()}, device(dy)
    grads = dict(zip(("x", "w"), tg.grouped_backward(dyd, *at.values(), ends)))
    leaves = {n: a.clone().requires_grad_() for n, a in at.items()}
    tg.grouped_linear(*leaves.values(), ends).backward(dyd)
    y = [tg.grouped(*({**at, name: device(t[name] + z * STEP[name] * v)}).values(), ends) for z in (1, -1)]
    torch.cuda.synchronize()
    assert tg.device_status()[0] == tg.Status.OK
    quotient = float(((ref.f64(y[0]) - ref.f64(y[1])) * dy).sum() / (2 * STEP[name]))
    for g in (grads[name], leaves[name].grad):
        slope = float((ref.f64(g) * v).sum())
        assert abs(slope - quotient) <= bound, (slope, quotient, bound)
