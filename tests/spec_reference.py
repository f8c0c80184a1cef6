"""Plain 64-bit implementations of the speculative decoding step's operators (rotary positions, the
quantised paged cache, tree attention, draft verification), for the tests: numpy and Python, one row
at a time where that is simplest, sharing nothing with the library."""
import math

import numpy as np
import torch


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- rotary positions

def rope_frequencies(rot, theta, kind="plain", factor=1.0, original=0.0, fast=0.0, slow=0.0):
    i = np.arange(rot // 2, dtype=np.float64)
    if kind == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    f = theta ** (-2 * i / rot)
    if kind == "linear":
        f = f / factor
    if kind == "by_parts":
        turns = original * f / (2 * math.pi)
        keep = np.clip((turns - slow) / (fast - slow), 0, 1)
        f = keep * f + (1 - keep) * f / factor
    return f


def rope(x, positions, table, interleaved, inverse):
    """x [N, heads, D], table [max_pos, rot/2, 2], all 64 bits."""
    half = table.shape[1]
    y = x.copy()
    sign = -1.0 if inverse else 1.0
    for n, pos in enumerate(positions):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            c, s = table[pos, i, 0], sign * table[pos, i, 1]
            y[n, :, a] = x[n, :, a] * c - x[n, :, b] * s
            y[n, :, b] = x[n, :, a] * s + x[n, :, b] * c
    return y


# ---- the cache's formats

E4M3 = np.array([(-1.0) ** (b >> 7) * ((b & 7) * 2.0 ** -9 if (b >> 3) & 15 == 0 else (1 + (b & 7) / 8) * 2.0 ** (((b >> 3) & 15) - 7))
                 for b in range(256)])
E4M3[[127, 255]] = np.nan


def round_half_even(x):
    return np.rint(x)


def fp8_row(x):
    """(codes, scale byte, values) of one row (64 bits)."""
    if not np.isfinite(x).all():
        return None, 255, np.full_like(x, np.nan)
    top = np.abs(x).max()
    e = -117
    while top > 448 * 2.0 ** e:
        e += 1
    y = x / 2.0 ** e
    grid = E4M3[:127]  # 0 and the positive values, ascending
    mag = np.abs(y)
    hi = np.clip(np.searchsorted(grid, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    below, above = mag - grid[lo], grid[hi] - mag
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = np.where(mag >= grid[126], 126, code)
    code = code + 128 * np.signbit(y)
    return code.astype(np.uint8), e + 127, E4M3[code] * 2.0 ** e


def int4_row(x, group):
    """(codes, scales, biases, values) of one row; scales and biases as fp16."""
    n = len(x) // group
    q, s, b = np.zeros(len(x), np.uint8), np.zeros(n, np.float16), np.zeros(n, np.float16)
    v = np.zeros(len(x))
    for g in range(n):
        y = x[g * group:(g + 1) * group]
        if not np.isfinite(y).all():
            s[g], v[g * group:(g + 1) * group] = np.nan, np.nan
            continue
        lo, hi = np.clip(y.min(), -57344, 57344), np.clip(y.max(), -57344, 57344)
        s[g], b[g] = np.float16((hi - lo) / 15), np.float16(lo)
        sd, bd = float(s[g]), float(b[g])
        c = np.clip(round_half_even((y - bd) / sd), 0, 15) if sd > 0 else np.zeros(group)
        q[g * group:(g + 1) * group] = c
        v[g * group:(g + 1) * group] = c * sd + bd
    return q, s, b, v


def stored(x, kind, group=0):
    """The values that rows x [..., D] (64 bits) come back as."""
    flat = x.reshape(-1, x.shape[-1])
    if kind == "bf16":
        return x
    out = np.stack([fp8_row(r)[2] if kind == "fp8" else int4_row(r, group)[3] for r in flat])
    return out.reshape(x.shape)


# ---- trees

def sees(parents):
    """[T, T]: what each node sees (itself and its ancestors); an absent node nothing."""
    t = len(parents)
    m = np.zeros((t, t), bool)
    for i in range(t):
        chain, node = [], i
        while node > 0 and parents[node] >= 0:
            chain.append(node)
            node = parents[node]
        if node == 0:
            m[i, chain + [0]] = True
    return m


def depths(parents):
    return [max(int(row.sum()) - 1, 0) for row in sees(parents)]


def words(m):
    """Mask words int32 [T, ceil(T/32)] of a [T, T] truth array."""
    t = m.shape[0]
    w = np.zeros((t, (t + 31) // 32), np.uint32)
    for i, j in zip(*np.nonzero(m)):
        w[i, j // 32] |= np.uint32(1 << (j % 32))
    return torch.from_numpy(w.view(np.int32))


def attention(q, k, v, ctx, see, scale):
    """One sequence: q [T, Hq, D], k, v [keys, Hk, D], see [T, T]. Returns out, lse, and per row what the
    error bounds need: sum p |v| and the largest |q||k| sum, times scale."""
    t, hq, d = q.shape
    g = hq // k.shape[1]
    out, lse = np.zeros((t, hq, d)), np.full((t, hq), -np.inf)
    weight, reach = np.zeros((t, hq, d)), np.zeros((t, hq))
    for i in range(t):
        at = np.concatenate([np.arange(ctx), ctx + np.nonzero(see[i])[0]]).astype(int)
        if not len(at):
            continue
        for h in range(hq):
            kk, vv = k[at, h // g], v[at, h // g]
            x = scale * (kk @ q[i, h])
            m = x.max()
            p = np.exp(x - m)
            out[i, h] = p @ vv / p.sum()
            lse[i, h] = m + np.log(p.sum())
            weight[i, h] = p @ np.abs(vv) / p.sum()
            reach[i, h] = abs(scale) * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, lse, weight, reach


# ---- verification

def verify(logits, tokens, parents, temp, draft=None, u=None, noise=None):
    """One sequence, all 64 bits. Returns (count, path, next, margin): margin is how near (relatively) any
    decision came to the other one."""
    margin = [np.inf]

    def near(a, b):
        margin.append(abs(a - b) / max(abs(a), abs(b), 1e-300))

    greedy = draft is None or not temp > 0

    def target(node):
        x = logits[node]
        if greedy:
            return x
        e = np.exp((x - x.max()) / temp)
        return e / e.sum()

    cur, path = 0, [0]
    r, s = target(0), 1.0
    for i in range(1, len(tokens)):
        if (parents[i] if parents is not None else i - 1) != cur or not 0 <= tokens[i] < logits.shape[1]:
            continue
        x = tokens[i]
        if greedy:
            ok = x == int(np.argmax(r))
        else:
            a, b = u[i] * s * draft[cur][x], r[x]
            near(a, b)
            ok = a < b
        if ok:
            cur = i
            path.append(i)
            r, s = target(i), 1.0
        elif not greedy:
            r = np.maximum(r - s * draft[cur], 0)
            s = r.sum()
    if greedy:
        return len(path) - 1, path, int(np.argmax(r)), np.inf
    if not s > 0:
        r = target(cur)
    race = r / noise
    two = np.sort(race)[-2:]
    if len(race) > 1:
        near(two[0], two[1])
    return len(path) - 1, path, int(np.argmax(race)), min(margin)
