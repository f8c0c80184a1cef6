"""Plain 64-bit implementations of the operators of a prompt's pass (head norms with rotary positions, causal
attention over packed prompts, the gated delta rule, log probabilities), for the tests: numpy, one row or one
token at a time, sharing nothing with the library."""
import numpy as np

import spec_reference as R

f64 = R.f64


def norm_rope(x, w, eps, positions, table, interleaved):
    """x [N, heads, D] -> (the normed rows, what they turn into)."""
    n = x * (np.mean(x * x, -1, keepdims=True) + eps) ** -0.5 * w
    return n, R.rope(n, positions, table, interleaved, False)


def attention(q, k, v, starts, scale):
    """q [N, Hq, D], k, v [N, Hk, D]. Returns (out, lse, the largest scale sum|q||k| of each row, sum p |v|); rows
    of no sequence are NaN."""
    N, hq, d = q.shape
    g = hq // k.shape[1]
    out, mass = (np.full((N, hq, v.shape[2]), np.nan) for _ in range(2))
    lse, size = (np.full((N, hq), np.nan) for _ in range(2))
    for lo, hi in zip(starts[:-1], starts[1:]):
        for t in range(lo, hi):
            for h in range(hq):
                kk, vv = k[lo:t + 1, h // g], v[lo:t + 1, h // g]
                x = scale * (kk @ q[t, h])
                m = x.max()
                p = np.exp(x - m)
                lse[t, h] = m + np.log(p.sum())
                p /= p.sum()
                out[t, h] = p @ vv
                mass[t, h] = p @ np.abs(vv)
                size[t, h] = abs(scale) * (np.abs(kk) @ np.abs(q[t, h])).max()
    return out, lse, size, mass


def delta(q, k, v, decay, beta, state, scale, norm_eps):
    """One sequence: q, k [T, Hk, D], v [T, Hv, D], decay, beta [T, Hv], state [Hv, D, D]. Returns (out, state,
    the largest norm that a column of the state had, with |v|'s largest, [Hv, D])."""
    T, hv, d = v.shape
    g = hv // q.shape[1]
    if norm_eps is not None:
        q = q / np.sqrt((q * q).sum(-1, keepdims=True) + norm_eps)
        k = k / np.sqrt((k * k).sum(-1, keepdims=True) + norm_eps)
    out, S = np.zeros((T, hv, d)), state.copy()
    size = np.sqrt((S * S).sum(1))
    for t in range(T):
        for h in range(hv):
            S[h] *= np.exp(decay[t, h])
            u = beta[t, h] * (v[t, h] - S[h].T @ k[t, h // g])
            S[h] += np.outer(k[t, h // g], u)
            out[t, h] = scale * (S[h].T @ q[t, h // g])
            size[h] = np.maximum(size[h], np.sqrt((S[h] * S[h]).sum(0)) + np.abs(v[t, h]))
    return out, S, size


def logprobs(row):
    """One row: (log probabilities, entropy, log Z, sum p (x - m)^2, the order: best first, of equal ones the lowest index)."""
    m = row.max()
    with np.errstate(divide="ignore", invalid="ignore"):
        d = row - m
        e = np.exp(d)
        z = e.sum()
        lp = d - np.log(z)
        p = e / z
        h = -np.where(p > 0, p * lp, 0.0).sum()
        spread = np.where(p > 0, p * d * d, 0.0).sum()
    return lp, h, np.log(z), spread, np.argsort(-row, kind="stable")
