"""The paged key-value cache's operators in plain 64-bit arithmetic (numpy), and
the rounding bounds that the tests hold the kernels to."""

import numpy as np

U = 2.0 ** -24  # half a step of fp32, relative


def visible(p, n, window, sinks):
    """Slots that a query at position p sees in a cache of n slots."""
    t = np.arange(n)
    ok = t <= p
    if window:
        ok &= (t > p - window) | (t < sinks)
    return ok


def attend(q, k, v, there, p, scale, window, sinks, u_p, u_out):
    """One query row: q [heads, dim]; k, v [kv heads, n, dim] (float64; rows of slots
    that are not there may hold anything); there [n] whether the slot's page exists;
    position p. Returns (out [heads, dim], weights [kv heads, n], tolerance of out,
    tolerance of the weights).

    u_p: relative rounding of a weight that enters the second product; u_out: of
    the output. The fp32 errors counted: a score is a sum of dim exact products
    (dim roundings of sums bounded by sum |q k|), times the scale, minus the
    maximum, through an exponential of 2 ulp; a score's error is the weight's
    relative error, once itself and once through the normalizer; the sums over the
    slots add one rounding per slot each; rescaling a handful more. In fp16 a weight
    below 2^-14 of the maximum is off by up to 2^-25 absolutely."""
    heads, dim = q.shape
    kv, n, _ = k.shape
    group = heads // kv
    ok = visible(p, n, window, sinks) & there
    out, tol = np.zeros((heads, dim)), np.zeros((heads, dim))
    w_all, w_tol = np.zeros((kv, n)), np.zeros((kv, n))
    idx = np.nonzero(ok)[0]
    if p < 0 or idx.size == 0:
        return out, w_all, tol, w_tol
    for h in range(heads):
        g = h // group
        kk, vv = k[g, idx], v[g, idx]
        s = scale * (kk @ q[h])
        mass = abs(scale) * (np.abs(kk) @ np.abs(q[h]))
        w = np.exp(s - s.max())
        w /= w.sum()
        d_s = dim * U * mass.max() + 8 * U * max(1.0, np.abs(s).max())
        rel = 2 * d_s + (2 * idx.size + 64) * U
        out[h] = w @ vv
        tol[h] = (u_p + rel) * (w @ np.abs(vv)) + 2.0 ** -25 * np.abs(vv).sum(0) + u_out * np.abs(out[h]) + 1e-30
        w_all[g, idx] += w
        w_tol[g, idx] += w * rel + 2.0 ** -126
    return out, w_all, tol, w_tol


def gather(cache, row, n):
    """[kv heads, n, dim] of one sequence and [n] whether the slot's page exists
    (slots on no page read as 0)."""
    pages, kv, ps, dim = cache.shape
    out, there = np.zeros((kv, n, dim)), np.zeros(n, dtype=bool)
    for t in range(n):
        p = int(row[t // ps])
        if 0 <= p < pages:
            out[:, t] = cache[p, :, t % ps]
            there[t] = True
    return out, there


def evict_kept(w, n, budget, sinks, recent):
    """Slots that stay, of one sequence and head with weights w (n > budget)."""
    held = list(range(sinks)) + list(range(n - recent, n))
    rest = range(sinks, n - recent)
    key = [(0 if np.isnan(w[t]) else 1, 0.0 if np.isnan(w[t]) else -float(w[t]), t) for t in rest]
    best = [t for _, _, t in sorted(key)[:budget - sinks - recent]]
    return sorted(held + best)
