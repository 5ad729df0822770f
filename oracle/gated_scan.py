"""fp64 oracle of the gated linear recurrence (test infrastructure, no library code).

One sequence, token by token:
    s = softplus(lam)   R = sigmoid(r)   G = sigmoid(g)   la = -c s R
    a = exp(la)   m = sqrt(1 - a^2)   h_t = a h_{t-1} + m G x_t   y_t = h_t [silu(z_t)]
and the gradients of sum(y dy) + sum(h_L dh) by the reverse recurrence
    d_t = dy_t silu(z_t) + a_{t+1} d_{t+1}.

`bounds` gives, beside each result, how far a computation in fp32 may be off: every
factor that enters a product is taken to be off by KAPPA half-steps of fp32, and the
recurrences carry those errors on, over the magnitudes (absolute sums, so that
cancellation is covered).  KAPPA: the argument of sigmoid's exponential is off by
half a step of |r| <= 8, the exponential, the sum and the quotient by one or two
steps each (|r| + 5); la adds two and m, a square root, halves what it is given;
b = m G x has two such factors, and three products: 2 * 13 + 3 < 32.  a = exp(la)
turns la's relative error, |r| + 7 < 16 half-steps, into one of |la| times that, and
adds two steps of its own: KAPPA (1 + |la|) in all.
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24  # half a step of fp32
KAPPA = 32


def _sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def _gates(lam, r, g, c):
    s = np.logaddexp(0.0, lam)
    R, G = _sigmoid(r), _sigmoid(g)
    la = -c * s * R
    return R, G, la, np.exp(la), np.sqrt(-np.expm1(2.0 * la))


def forward(lam, x, r, g, z=None, h0=None, c=8.0):
    """One sequence: x, r, g, z [L, D], lam, h0 [D].  A dict: y, h (all states [L, D]),
    h_end, and the bounds y_off, h_off, h_end_off, with `size` the magnitudes."""
    L, D = x.shape
    R, G, la, a, m = _gates(lam, r, g, c)
    b = m * G * x
    h = np.zeros(D) if h0 is None else h0.astype(np.float64)
    hs, size, off = np.empty((L, D)), np.empty((L, D)), np.empty((L, D))
    M, E = np.abs(h), np.zeros(D)
    for t in range(L):
        h = a[t] * h + b[t]
        aM = a[t] * M
        M = aM + np.abs(b[t])
        E = a[t] * E + KAPPA * U * (M - la[t] * aM)
        hs[t], size[t], off[t] = h, M, E
    out = {"h": hs, "h_end": h, "size": size, "h_off": off, "h_end_off": E}
    if z is None:
        out["y"], out["y_off"] = hs, off
    else:
        gate = z * _sigmoid(z)
        out["y"] = hs * gate
        out["y_off"] = (off + KAPPA * U * size) * np.abs(gate)
    return out


def backward(lam, x, r, g, dy, z=None, h0=None, dh=None, c=8.0):
    """The gradients x, r, g, lam, h0 (and z), each with its bound as "<name>_off"."""
    L, D = x.shape
    R, G, la, a, m = _gates(lam, r, g, c)
    f = forward(lam, x, r, g, None, h0, c)
    h, size, off = f["h"], f["size"], f["h_off"]
    start = np.zeros(D) if h0 is None else h0.astype(np.float64)
    hp = np.concatenate([start[None], h[:-1]]) if L else h
    hp_size = np.concatenate([np.abs(start)[None], size[:-1]]) if L else h
    hp_off = np.concatenate([np.zeros((1, D)), off[:-1]]) if L else h
    out = {}
    ds = dy.astype(np.float64)
    if z is not None:
        sig = _sigmoid(z)
        slope = sig * (1.0 + z * (1.0 - sig))
        out["z"] = dy * h * slope
        # 1 + z (1 - sig) cancels for negative z: its error goes by 1 + |z| (1 - sig)
        wide = sig * (1.0 + np.abs(z) * (1.0 - sig))
        out["z_off"] = np.abs(dy) * (off * wide + KAPPA * U * size * wide)
        ds = dy * z * sig
    e = np.zeros(D) if dh is None else dh.astype(np.float64)
    eM, eE = np.abs(e), np.zeros(D)
    d, dM, dE = np.empty((L, D)), np.empty((L, D)), np.empty((L, D))
    for t in range(L - 1, -1, -1):
        d[t] = ds[t] + e
        dM[t] = np.abs(ds[t]) + eM
        dE[t] = eE + KAPPA * U * dM[t]
        e, eM = a[t] * d[t], a[t] * dM[t]
        eE = a[t] * (dE[t] + KAPPA * U * (1.0 - la[t]) * dM[t])
    out["h0"], out["h0_off"] = e, eE
    out["x"], out["x_off"] = d * m * G, m * G * (dE + KAPPA * U * dM)
    out["g"] = d * m * x * G * (1.0 - G)
    # 1 - G: half a step of one beside its own size
    out["g_off"] = m * np.abs(x) * G * ((1.0 - G) * (dE + KAPPA * U * dM) + KAPPA * U * dM)
    per_m = np.where(m > 0, 1.0 / np.where(m > 0, m, 1.0), 0.0)
    k = a * hp - a * a * per_m * G * x
    k_size = a * (1.0 - la) * hp_size + a * a * (1.0 - la) * per_m * G * np.abs(x)
    dla = d * k
    dla_off = dE * k_size + dM * (a * hp_off + 2 * KAPPA * U * k_size)
    out["r"] = dla * la * (1.0 - R)
    out["r_off"] = np.abs(la) * ((1.0 - R) * dla_off + KAPPA * U * dM * k_size)
    sl = c * _sigmoid(lam)
    out["lam"] = -sl * (dla * R).sum(0)
    # the terms' errors, and those of summing 128 tokens and then the pieces
    out["lam_off"] = sl * (R * (dla_off + (KAPPA + 128 + L / 128) * U * dM * k_size)).sum(0)
    return out


def memory_bounds(lam, x, r, g, h0, dy, dh, c=8.0):
    """Closer bounds for long memories, where `forward` and `backward` allow KAPPA half-steps of
    the whole state at every token: of h (each token's), of d_x and of d_h0 in half-steps counted
    one by one, for |r|, |g| <= 4 and decays near one.

    a = 1 - (1 - a): one rounding of a number in [1/2, 1), half a half-step, and (1 - a) off by
    KAPPA of itself (R: |r| + 7, c softplus(lam) log2(e): 10, their product 1, the polynomial 9).
    Between a token and the state that it enters there is one rounding a token, in the fused
    multiply-add or in the product of a tile's decays: with a's own, 1.5 a token.  Putting
    segments together adds two for every 8 tokens at most (16 in bf16): 2 a token in all, and 8
    once for the parts that the last state is put together from.  b is off by KAPPA.  Back,
    e = a (e + dy) is rounded twice a token: 2.5, and the same for the parts: 3."""
    R, G, la, a, m = _gates(lam, r, g, c)
    b = np.abs(m * G * x)
    M, E = np.abs(h0.astype(np.float64)), np.zeros(len(lam))
    h_off = np.empty(x.shape)
    for t in range(len(x)):
        before = M
        M = a[t] * M + b[t]
        E = a[t] * E + U * (2 * M + KAPPA * ((1 - a[t]) * before + b[t]))
        h_off[t] = E + 8 * U * M
    dM, dE = np.abs(dh.astype(np.float64)), np.zeros(len(lam))
    dx_off = np.empty(x.shape)
    for t in range(len(x) - 1, -1, -1):
        dM = dM + np.abs(dy[t])
        dE = dE + U * dM
        dx_off[t] = m[t] * G[t] * (dE + (KAPPA + 8) * U * dM)
        dE = a[t] * dE + U * (2 * a[t] + KAPPA * (1 - a[t])) * dM
        dM = a[t] * dM
    return {"h_off": h_off, "x_off": dx_off, "h0_off": dE + 8 * U * dM}
