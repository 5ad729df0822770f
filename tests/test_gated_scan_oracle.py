"""Pins of the gated scan's fp64 oracle: closed forms, splitting, and its gradients against
central differences of its forward."""
import numpy as np
import pytest

from oracle import gated_scan as GS


def _inputs(L, D, seed, gated=True):
    g = np.random.default_rng(seed)
    v = {k: g.standard_normal((L, D)) for k in ("x", "r", "g", "dy")}
    v["z"] = g.standard_normal((L, D)) if gated else None
    v["lam"] = g.standard_normal(D) - 3.0
    v["h0"], v["dh"] = g.standard_normal(D), g.standard_normal(D)
    return v


def test_closed_gates_keep_the_state():
    v = _inputs(7, 3, 0, gated=False)
    f = GS.forward(v["lam"], v["x"], np.full((7, 3), -np.inf), v["g"], None, v["h0"])
    assert np.array_equal(f["h"], np.broadcast_to(v["h0"], (7, 3)))


def test_constant_decay_is_a_geometric_sum():
    L, c = 9, 8.0
    lam, r = np.array([-4.0]), np.zeros((L, 1))
    a = np.exp(-c * np.log1p(np.exp(-4.0)) / 2)
    f = GS.forward(lam, np.ones((L, 1)), r, np.full((L, 1), np.inf), c=c)
    want = np.sqrt(1 - a * a) * (1 - a ** np.arange(1, L + 1)) / (1 - a)
    assert np.allclose(f["h"][:, 0], want, rtol=1e-13)


def test_a_split_sequence_goes_on_from_its_state():
    v = _inputs(11, 4, 1)
    whole = GS.forward(v["lam"], v["x"], v["r"], v["g"], v["z"], v["h0"])
    one = GS.forward(v["lam"], v["x"][:5], v["r"][:5], v["g"][:5], v["z"][:5], v["h0"])
    two = GS.forward(v["lam"], v["x"][5:], v["r"][5:], v["g"][5:], v["z"][5:], one["h_end"])
    assert np.allclose(np.concatenate([one["y"], two["y"]]), whole["y"], rtol=1e-13, atol=0)


@pytest.mark.parametrize("gated", [False, True])
def test_gradients_match_differences(gated):
    v = _inputs(6, 3, 2, gated)

    def value(**kw):
        w = {**v, **kw}
        f = GS.forward(w["lam"], w["x"], w["r"], w["g"], w["z"], w["h0"])
        return (f["y"] * v["dy"]).sum() + (f["h_end"] * v["dh"]).sum()

    got = GS.backward(v["lam"], v["x"], v["r"], v["g"], v["dy"], v["z"], v["h0"], v["dh"])
    eps = 1e-6
    for name in ("x", "r", "g", "lam", "h0") + (("z",) if gated else ()):
        num = np.empty_like(v[name])
        for i in np.ndindex(num.shape):
            up, dn = v[name].copy(), v[name].copy()
            up[i] += eps
            dn[i] -= eps
            num[i] = (value(**{name: up}) - value(**{name: dn})) / (2 * eps)
        # central differences: eps^2 of curvature and 1e-16 / eps of rounding
        assert np.allclose(got[name], num, rtol=1e-7, atol=1e-8), name


def test_bounds_are_small_beside_the_results():
    v = _inputs(300, 5, 3)
    f = GS.forward(v["lam"], v["x"], v["r"], v["g"], v["z"], v["h0"])
    assert np.max(f["y_off"]) < 1e-3 * np.max(np.abs(f["y"]))


def _long(L=3000, D=8, seed=9):
    """Decays from 0.99 to 0.9995 and inputs of one sign: nothing cancels, and every error stays."""
    g = np.random.default_rng(seed)
    v = {k: np.abs(g.standard_normal((L, D))) for k in ("x", "dy")}
    v["r"], v["g"] = (np.clip(1 + 0.5 * g.standard_normal((L, D)), -4, 4) for _ in range(2))
    v["lam"] = np.log(np.expm1(-np.log(np.linspace(0.99, 0.9995, D)) / 8.0))
    v["h0"], v["dh"] = np.abs(g.standard_normal(D)), np.abs(g.standard_normal(D))
    return {k: t.astype(np.float32).astype(np.float64) for k, t in v.items()}


def test_closer_bounds_hold_for_fp32_and_see_three_lost_digits():
    v = _long()
    near = GS.memory_bounds(**v)
    f = GS.forward(v["lam"], v["x"], v["r"], v["g"], None, v["h0"])
    # token by token in fp32, from coefficients rounded to it
    _, G, _, a, m = GS._gates(v["lam"], v["r"], v["g"], 8.0)
    a32, b32 = a.astype(np.float32), (m * G * v["x"]).astype(np.float32)
    h, worst = v["h0"].astype(np.float32), 0.0
    for t in range(len(a32)):
        h = (a32[t] * h + b32[t]).astype(np.float32)
        worst = max(worst, np.max(np.abs(h - f["h"][t]) / near["h_off"][t]))
    assert worst < 1
    # a state that has lost three of its digits halfway: the wide bounds let it pass
    lost = f["h"] * (1 + 2.0 ** -12)
    assert np.all(np.abs(lost - f["h"])[-1, -1] <= f["h_off"][-1, -1])
    assert np.all(np.abs(lost - f["h"]) > near["h_off"])
