"""GPU tests of the operators of a prompt's pass through the binding, against 64-bit implementations
(prompt_reference).

Tolerances, from the number formats (unit roundoffs: u16 = 2^-8 of bf16, u32 = 2^-24):
  head norms  a row's sum of D squares is off by at most D u32 of itself, its root by half of that; with the
              products and the turn's two products and sum, and one rounding to bf16:
                |err| <= u16 |y| + (D + 16) u32 (|n0| + |n1|), n the normed elements of the pair
  attention   the scores are off by at most d = (D + 8) u32 max_j scale sum|q||k| (a sum of D products in fp32; the
              8 for the scale, the maximum and the exponential), so that each weight is off by a factor of
              1 + 2 d; weights are rounded to bf16 (u16 of p |v|), the result to bf16: with A = sum p |v|
                |err| <= (1.5 u16 + 4 d + 64 u32) A + u16 |out| + 2^-24,  lse: 2 d + 64 u32 (1 + |lse|)
  delta rule  columns of the state do not meet. With keys of norm 1 at most and beta <= 1, I - beta k k^T makes no
              column's error longer, and a token adds at most (D + 16) u32 M to it: M the largest that a column's
              norm plus |v| was, D u32 of it from the sum over the keys, the rest from the decay (expf is within
              two units of the last place), the norms and the update. After T tokens and from an output's own sum:
                |state err| <= T (D + 16) u32 M + u32 |S|
                |out err| <= u16 |out| + scale |q| (T + 1) (D + 16) u32 M
              In chunks, an operand on the way to the state is the sum of two fp16, off by 2^-22 of itself or 2^-38 of
              the largest of its column. With the state's columns and the values within M, X and so R are off by
              (2^-22 + D u32) M a token (keys of norm 1), U = T R by that and two more 2^-22 of up to sqrt(64) terms
              of size M times what T does to them (2 or so), U's 64 terms' sums by 64 u32; the state takes that
              on, and its own errors: (D + 16) u32 M a token as above, over a chunk's 64, bound them. For the outputs
              the state and U are rounded to 11 bits, P too: three roundings of 2^-12, of sums within M
                |out err| <= u16 |out| + scale (3 2^-12 + (T + 64) (D + 16) u32) M
  log probabilities  e^d is off by 2 |d| u32 (the product with log2 e) and 2^-22 (the function) of itself, sums
              run over V/1024 elements a thread and then 40 joins: log Z is off by at most
              r = (V/1024 + 100) u32 (the |d| weighted with p add up to less than the entropy, at most 21), so
                |logp err| <= r + 4 u32 (|x - m| + |logp|)
                |entropy err| <= r (1 + H + log Z) + 4 u32 sum p d^2 + 4 u32 H
              (S = sum d e^d has terms of one sign, each off by 4 |d| u32 + 2^-22 of itself)
"""
import numpy as np
import pytest
import torch

import prompt_reference as P
from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B

pytestmark = pytest.mark.gpu
U16, U32 = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def within(got, want, limit, what):
    got = P.f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, what
    assert np.all(np.isfinite(got)), what
    ratio = np.abs(got - want) / limit
    assert ratio.max(initial=0.0) <= 1.0, f"{what}: {ratio.max():.3g} of the limit at {np.unravel_index(ratio.argmax(), ratio.shape)}"


def fine():
    assert B.device_status() == B.TS_OK


# ------------------------------------------------------------------ head norms and rotary positions

def check_norm_rope(n, hq, hk, d, rot, interleaved, seed, *, in_place=False, scale=1.7, eps=1e-6):
    g = gen(seed)
    x = randn(g, n, hq + 2 * hk, d, scale=scale)
    x[0, 0] = 0  # a head of zeros
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    table = B.rope_table(500, rot, 10000.0)
    pos = torch.randint(0, 500, (n,), generator=g, device="cuda", dtype=torch.int32)
    inputs = [P.f64(t) if t is not None else None for t in (q, k)]
    rest = x[:, hq + hk:].clone()
    out = B.hc_qk_norm_rope(q, k, pos, table, w[0], w[1] if hk else None, eps=eps, interleaved=interleaved,
                            **(dict(q_out=q, k_out=k) if in_place else {}))
    for got, xin, wt in zip(out, inputs, w):
        if xin is None:
            assert got is None
            continue
        normed, want = P.norm_rope(xin, P.f64(wt), eps, pos.cpu().numpy(), P.f64(table), interleaved)
        size, r = np.abs(normed), rot // 2
        pair = size.copy()
        i0, i1 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(r), np.arange(r) + r)
        pair[..., i0] = pair[..., i1] = size[..., i0] + size[..., i1]
        within(got, want, U16 * np.abs(want) + (d + 16) * U32 * pair + 1e-38, "head norms")
    assert torch.equal(rest, x[:, hq + hk:])
    fine()


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 64), (128, 32), (256, 256), (256, 64), (128, 20), (80, 80),
                                   (80, 32), (8, 2), (1024, 1024), (32, 32), (200, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_heads(d, rot, interleaved):
    check_norm_rope(5, 4, 2, d, rot, interleaved, d + rot)


@pytest.mark.parametrize("n,hq,hk", [(1, 1, 0), (1, 20, 4), (3, 1, 1), (67, 5, 1), (700, 32, 8), (1, 64, 3), (257, 7, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope_counts(n, hq, hk, in_place):
    check_norm_rope(n, hq, hk, 128, 64, False, n, in_place=in_place)


@pytest.mark.parametrize("d,rot", [(128, 128), (80, 20)])
@pytest.mark.parametrize("scale,eps", [(1e-20, 1e-6), (1e15, 1e-6), (1.0, 10.0)])
def test_norm_rope_magnitudes(d, rot, scale, eps):
    check_norm_rope(3, 2, 1, d, rot, True, 5, scale=scale, eps=eps)


@pytest.mark.parametrize("d,rot", [(128, 64), (80, 20)])
def test_norm_rope_positions_out_of_range(d, rot):
    g = gen(1)
    q, w, table = randn(g, 4, 3, d), torch.ones(d, device="cuda").bfloat16(), B.rope_table(10, rot, 10000.0)
    good = torch.tensor([0, 3, 9, 5], device="cuda", dtype=torch.int32)
    want, _ = B.hc_qk_norm_rope(q, None, good, table, w)
    fine()
    got, _ = B.hc_qk_norm_rope(q, None, torch.tensor([0, -1, 10, 5], device="cuda", dtype=torch.int32), table, w)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert torch.equal(got[[0, 3]], want[[0, 3]])
    assert not got[1:3, :, :rot].any() and torch.equal(got[1:3, :, rot:], want[1:3, :, rot:])


def test_norm_rope_nan_stays_in_its_head():
    g = gen(2)
    for d, rot in ((128, 128), (80, 80)):
        q, w, table = randn(g, 3, 4, d), torch.ones(d, device="cuda").bfloat16(), B.rope_table(10, rot, 10000.0)
        pos = torch.arange(3, device="cuda", dtype=torch.int32)
        want, _ = B.hc_qk_norm_rope(q, None, pos, table, w)
        q[1, 2, 7] = float("nan")
        got, _ = B.hc_qk_norm_rope(q, None, pos, table, w)
        assert got[1, 2].isnan().all()
        got[1, 2] = want[1, 2]
        assert torch.equal(got, want)


# ------------------------------------------------------------------ attention over packed prompts

def prompts(lens, hq, hk, d, seed, *, behind=0, q_scale=1.5):
    """Slices of one projection's output, the sequences' starts, and rows of no sequence behind them."""
    g = gen(seed)
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    x = randn(g, at[-1] + behind, hq + 2 * hk, d)
    x[:, :hq] *= q_scale
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], torch.tensor(at, device="cuda", dtype=torch.int32), at


def check_attention(q, k, v, at, got, scale=None, rows=None):
    """``rows``: the heads that are looked at."""
    d = q.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    out, lse, size, mass = P.attention(P.f64(q), P.f64(k), P.f64(v), at, scale)
    err = (d + 8) * U32 * size
    in_use = slice(at[0], at[-1])
    a, z = P.f64(got[0])[in_use], P.f64(got[1])[in_use]
    out, lse, err, mass = out[in_use], lse[in_use], err[in_use], mass[in_use]
    limit = (1.5 * U16 + 4 * err + 64 * U32)[..., None] * mass + U16 * np.abs(out) + 2.0 ** -24
    within(a, out, limit, "out")
    within(z, lse, 2 * err + 64 * U32 * (1 + np.abs(lse)), "lse")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (6, 2), (8, 1), (5, 1)])
@pytest.mark.parametrize("lens", [[1], [2, 1], [127, 128, 129], [0, 17, 0, 0, 64, 0], [255, 1, 256, 257], [300]])
def test_attention_lengths(d, hq, hk, lens):
    q, k, v, starts, at = prompts(lens, hq, hk, d, sum(lens) + hq)
    check_attention(q, k, v, at, B.hc_prompt_attention(q, k, v, starts))
    fine()


@pytest.mark.parametrize("hq,hk", [(40, 1), (33, 1), (37, 1), (128, 2), (3, 1), (7, 7), (48, 16)])
def test_attention_heads(hq, hk):
    q, k, v, starts, at = prompts([70, 3, 150], hq, hk, 64, hq)
    check_attention(q, k, v, at, B.hc_prompt_attention(q, k, v, starts))
    fine()


@pytest.mark.parametrize("d", [64, 128])
def test_attention_long(d):
    q, k, v, starts, at = prompts([1100, 1500], 2, 1, d, 5)
    check_attention(q, k, v, at, B.hc_prompt_attention(q, k, v, starts))
    fine()


def test_attention_many_sequences():
    """More than one round of the blocks' order, sequences of no tokens among them."""
    r = np.random.default_rng(3)
    lens = [int(x) for x in r.integers(0, 9, 700)]
    lens[5], lens[400], lens[699] = 300, 0, 140
    q, k, v, starts, at = prompts(lens, 2, 1, 64, 6)
    check_attention(q, k, v, at, B.hc_prompt_attention(q, k, v, starts))
    fine()


def test_attention_leaves_rows_behind():
    q, k, v, starts, at = prompts([50, 200], 4, 2, 128, 7, behind=60)
    k[250:], v[250:] = float("nan"), float("inf")
    out, lse = torch.full(q.shape, 7.0, device="cuda").bfloat16(), torch.full(q.shape[:2], 7.0, device="cuda")
    got = B.hc_prompt_attention(q, k, v, starts, out=out, lse=lse)
    assert got[0] is out and got[1] is lse and (out[250:] == 7).all() and (lse[250:] == 7).all()
    check_attention(q[:250], k[:250], v[:250], at, (out[:250], lse[:250]))
    fine()


@pytest.mark.parametrize("scale", [1e-3, 0.3, 4.0])
def test_attention_scale(scale):
    q, k, v, starts, at = prompts([200, 90], 2, 1, 64, 8, q_scale=3.0)
    check_attention(q, k, v, at, B.hc_prompt_attention(q, k, v, starts, scale=scale), scale)


def test_attention_growing_scores():
    """Keys whose scores grow with their place, so that a row's maximum does in every tile."""
    q, k, v, starts, at = prompts([700], 2, 1, 128, 9)
    q[:] = q.abs()
    k[:] = (torch.arange(700, device="cuda")[:, None, None] * 0.02 * torch.ones_like(k)).bfloat16()
    check_attention(q, k, v, at, B.hc_prompt_attention(q, k, v, starts))
    k[:] = k.flip(0)
    check_attention(q, k, v, at, B.hc_prompt_attention(q, k, v, starts))


@pytest.mark.parametrize("what", ["k nan", "v nan", "v inf", "k inf", "q nan"])
@pytest.mark.parametrize("token", [0, 40, 130, 299])
def test_attention_what_is_not_seen_does_not_reach(what, token):
    """An infinity or a NaN at a token of the second sequence: earlier tokens and other sequences are as without."""
    q, k, v, starts, at = prompts([90, 300, 45], 4, 2, 64, 10)
    want, want_lse = B.hc_prompt_attention(q, k, v, starts)
    t = at[1] + token
    bad = float(what.split()[1])
    dict(q=q, k=k, v=v)[what[0]][t, 1, 5] = bad
    got, lse = B.hc_prompt_attention(q, k, v, starts)
    for now, then in ((got, want), (lse, want_lse)):
        assert torch.equal(now[:t], then[:t]) and torch.equal(now[at[2]:], then[at[2]:])
    heads = slice(1, 2) if what[0] == "q" else slice(2, 4)  # the query heads of key head 1
    rows = slice(t, t + 1) if what[0] == "q" else slice(t, at[2])
    if what == "v nan":
        assert got[rows, heads, 5].isnan().all()
        got[rows, heads, 5] = want[rows, heads, 5]
    elif what == "v inf":
        assert (got[rows, heads, 5] == float("inf")).all()
        got[rows, heads, 5] = want[rows, heads, 5]
    else:
        if what != "k inf":
            assert got[rows, heads].isnan().all()
        got[rows, heads], lse[rows, heads] = want[rows, heads], want_lse[rows, heads]
    assert torch.equal(got, want) and torch.equal(lse, want_lse)
    fine()


def test_attention_starts_out_of_range():
    q, k, v, starts, at = prompts([50, 60, 70], 2, 1, 64, 11)
    want, _ = B.hc_prompt_attention(q, k, v, starts)
    for bad in ([0, 50, 110, 181], [-1, 50, 110, 180], [0, 120, 110, 180]):
        out = torch.full_like(q, 7.0).contiguous()
        got, _ = B.hc_prompt_attention(q, k, v, torch.tensor(bad, device="cuda", dtype=torch.int32), out=out)
        assert B.device_status() == B.TS_ERR_INVALID_ARG
        if bad[1] == 50:
            assert torch.equal(got[50:110], want[50:110])
        # (rows 110 .. 119 are two sequences' with the last of these)
        assert (got[110:] == 7).all() if bad[3] == 181 else torch.equal(got[120:], want[120:])
        if bad[0] == -1:
            assert (got[:50] == 7).all()


def test_attention_is_the_same_every_time_and_over_the_cache():
    """The same bits each time, replayed too; and what the attention over a paged cache gives for the same rows."""
    q, k, v, starts, at = prompts([512, 512], 8, 2, 128, 12)
    out, lse = B.hc_prompt_attention(q, k, v, starts)
    graph = torch.cuda.CUDAGraph()
    o2, l2 = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.graph(graph):
        B.hc_prompt_attention(q, k, v, starts, out=o2, lse=l2)
    for _ in range(5):
        o2.zero_(), l2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)
    cache = B.kv_cache("bf16", 2 * 8, 2, 64, 128, torch.arange(16, device="cuda", dtype=torch.int32).view(2, 8))
    ctx = torch.zeros(2, device="cuda", dtype=torch.int32)
    B.hc_kv_write(k.unflatten(0, (2, 512)), v.unflatten(0, (2, 512)), cache, ctx)
    tree, tree_lse = B.hc_tree_attention(q.unflatten(0, (2, 512)), cache, ctx)
    assert (tree.flatten(0, 1).float() - out.float()).abs().max() < 0.05
    assert (tree_lse.flatten(0, 1) - lse).abs().max() < 1e-4
    fine()


# ------------------------------------------------------------------ the gated delta rule

def gates(g, *shape):
    decay = -torch.rand(*shape, generator=g, device="cuda") ** 3 * 4
    return decay, torch.rand(*shape, generator=g, device="cuda")


def delta_limits(out, state, size, scale, T, d):
    """Of one sequence: out [T, Hv, D], state [Hv, D, D], size [Hv, D] (the columns'); |q| <= 1."""
    step = (d + 16) * U32 * size
    return U16 * np.abs(out) + scale * (T + 1) * step + 1e-38, T * step[:, None] + U32 * np.abs(state) + 1e-38


def step_case(b, t, hk, hv, d, seed, norm_eps=1e-6):
    g = gen(seed)
    x = randn(g, b, t, 2 * hk + hv, d, scale=1.0 if norm_eps is not None else 0.7 * d ** -0.5)
    q, k, v = x[:, :, :hk], x[:, :, hk:2 * hk], x[:, :, 2 * hk:]
    if norm_eps is None:  # norms of 1 at most
        for y in (q, k):
            y /= y.float().norm(dim=-1, keepdim=True).clamp(min=0.99).bfloat16() * 1.02
    decay, beta = gates(g, b, t, hv)
    return q, k, v, decay, beta, torch.randn(b, hv, d, d, generator=g, device="cuda") * 0.3


def check_step(args, got, state, counts, norm_eps, scale=None):
    q, k, v, decay, beta, before = (P.f64(x) for x in args)
    d = v.shape[-1]
    scale = d ** -0.5 if scale is None else scale
    for i, n in enumerate(counts):
        out, after, size = P.delta(q[i, :n], k[i, :n], v[i, :n], decay[i, :n], beta[i, :n], before[i], scale, norm_eps)
        lo, ls = delta_limits(out, after, size, abs(scale), n, d)
        if n:
            within(got[i, :n], out, lo, "out")
        within(state[i], after, ls, "state")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b,t,hk,hv", [(1, 1, 1, 1), (1, 1, 2, 4), (3, 1, 1, 3), (2, 4, 2, 2), (1, 7, 3, 6), (9, 3, 1, 2), (1, 70, 1, 1)])
@pytest.mark.parametrize("norm_eps", [1e-6, 0.5, None])
def test_delta_step(d, b, t, hk, hv, norm_eps):
    args = step_case(b, t, hk, hv, d, b + t + hv, norm_eps)
    before = args[5].clone()
    apart = torch.empty_like(before)
    out, same = B.hc_delta_step(*args, norm_eps=norm_eps, state_out=apart)
    assert same is apart and torch.equal(args[5], before)
    check_step(args, out, apart, [t] * b, norm_eps)
    again, state = B.hc_delta_step(*args[:5], before, norm_eps=norm_eps)  # in place
    assert state is before and torch.equal(state, apart) and torch.equal(again, out)
    fine()


@pytest.mark.parametrize("d", [64, 128])
def test_delta_step_counts(d):
    b, t = 6, 5
    args = step_case(b, t, 2, 4, d, 3)
    out = torch.full((b, t, 4, d), 7.0, device="cuda").bfloat16()
    counts = [0, 1, 2, 3, 4, 5]
    apart = torch.full_like(args[5], 9.0)
    B.hc_delta_step(*args, counts=torch.tensor(counts, device="cuda", dtype=torch.int32), out=out, state_out=apart)
    check_step(args, out, apart, counts, 1e-6)
    for i, n in enumerate(counts):
        assert (out[i, n:] == 7).all()
    assert torch.equal(apart[0], args[5][0])
    fine()
    # a count out of range is the nearest one in it
    wild, _ = B.hc_delta_step(*args, counts=torch.tensor([-3, 9, 5, 5, 5, 5], device="cuda", dtype=torch.int32), out=out.fill_(7.0),
                              state_out=torch.empty_like(apart))
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert (wild[0] == 7).all() and not (wild[1] == 7).all()


def test_delta_step_continues():
    """A step of five tokens is the same, bit for bit, as one of two and one of three."""
    args = step_case(2, 5, 1, 2, 128, 4)
    whole, state = B.hc_delta_step(*args, state_out=torch.empty_like(args[5]))
    half = args[5].clone()
    parts = [B.hc_delta_step(*(x[:, a:z].contiguous() for x in args[:5]), half)[0] for a, z in ((0, 2), (2, 5))]
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(half, state)


def test_delta_step_decays_that_keep_nothing():
    for low in (-200.0, float("-inf"), torch.finfo(torch.float32).min):
        args = list(step_case(1, 3, 1, 2, 64, 6))
        args[3][:, 1] = low
        out, state = B.hc_delta_step(*args, state_out=torch.empty_like(args[5]))
        fresh, want = B.hc_delta_step(*(x[:, 1:].contiguous() for x in args[:3]), *(x[:, 1:].contiguous() for x in args[3:5]),
                                      torch.zeros_like(args[5]))
        assert torch.equal(state, want) and torch.equal(out[:, 1:], fresh)


def prompt_case(lens, hk, hv, d, seed, *, behind=0, low=4.0):
    g = gen(seed)
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    n = at[-1] + behind
    x = randn(g, n, 2 * hk + hv, d)
    decay = -torch.rand(n, hv, generator=g, device="cuda") ** 3 * low
    return (x[:, :hk], x[:, hk:2 * hk], x[:, 2 * hk:], decay, torch.rand(n, hv, generator=g, device="cuda"),
            torch.randn(len(lens), hv, d, d, generator=g, device="cuda") * 0.3, torch.tensor(at, device="cuda", dtype=torch.int32)), at


def check_prompt(args, at, out, state, norm_eps=1e-6):
    q, k, v, decay, beta, before = (P.f64(x) for x in args[:6])
    d = v.shape[-1]
    scale = d ** -0.5
    for i, (lo, hi) in enumerate(zip(at[:-1], at[1:])):
        want, after, size = P.delta(q[lo:hi], k[lo:hi], v[lo:hi], decay[lo:hi], beta[lo:hi], before[i], scale, norm_eps)
        step = (d + 16) * U32 * size * (hi - lo + 64)
        if hi > lo:
            within(out[lo:hi], want, U16 * np.abs(want) + scale * (3 * 2.0 ** -12 * size + step) + 1e-38, "out")
        within(state[i], after, step[:, None] + U32 * np.abs(after) + 1e-38, "state")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 4), (1, 3)])
@pytest.mark.parametrize("lens", [[1], [64], [65, 63], [0, 5, 0, 130, 0], [200, 1, 64, 128]])
def test_delta_prompt(d, hk, hv, lens):
    args, at = prompt_case(lens, hk, hv, d, sum(lens) + hv)
    before = args[5].clone()
    apart = torch.empty_like(before)
    out, same = B.hc_delta_prompt(*args, state_out=apart)
    assert same is apart and torch.equal(args[5], before)
    check_prompt(args, at, out, apart)
    again, state = B.hc_delta_prompt(*args[:5], before, args[6])  # in place
    assert state is before and torch.equal(state, apart) and torch.equal(again, out)
    fine()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low", [0.01, 1.0, 60.0])
def test_delta_prompt_long(d, low):
    args, at = prompt_case([700], 1, 2, d, 3, low=low)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state)
    fine()


@pytest.mark.parametrize("hk,hv", [(1, 9), (3, 51), (2, 16)])
def test_delta_prompt_heads(hk, hv):
    args, at = prompt_case([70, 3], hk, hv, 64, hv)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state)
    fine()


def test_delta_prompt_many_sequences():
    r = np.random.default_rng(4)
    lens = [int(x) for x in r.integers(0, 90, 70)]
    args, at = prompt_case(lens, 1, 2, 64, 5)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state)
    fine()


@pytest.mark.parametrize("norm_eps", [0.5, None])
def test_delta_prompt_norms(norm_eps):
    args, at = prompt_case([150, 20], 2, 2, 128, 6)
    if norm_eps is None:  # norms of 1 at most
        for y in args[:2]:
            y /= y.float().norm(dim=-1, keepdim=True).bfloat16() * 1.02
    out, state = B.hc_delta_prompt(*args, norm_eps=norm_eps, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state, norm_eps)


def test_delta_prompt_equal_keys():
    """All keys the same, beta 1: each token's update takes back the one before."""
    args, at = prompt_case([130], 1, 1, 64, 7, low=0.0)
    args[1][:] = args[1][0].clone()
    args[4].fill_(1.0)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state)


@pytest.mark.parametrize("decay", [-200.0, float("-inf"), torch.finfo(torch.float32).min, -90.0])
def test_delta_prompt_strong_decays(decay):
    """After a token that keeps nothing all is as from a state of zeros, weak decays after strong ones among it."""
    args, at = prompt_case([190], 1, 2, 64, 8, low=0.05)
    args[3][[3, 40, 41, 100]] = decay
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    bounded = list(args)
    bounded[3] = args[3].clamp(min=-1e4)
    check_prompt(bounded, at, out, state)


def test_delta_prompt_leaves_rows_behind():
    args, at = prompt_case([50, 100], 1, 2, 128, 9, behind=40)
    for x in args[:5]:
        x[150:] = float("nan")
    out = torch.full((190, 2, 128), 7.0, device="cuda").bfloat16()
    _, state = B.hc_delta_prompt(*args, out=out, state_out=torch.empty_like(args[5]))
    assert (out[150:] == 7).all()
    check_prompt([x[:150] if i < 5 else x for i, x in enumerate(args)], at, out[:150], state)
    fine()


@pytest.mark.parametrize("what", ["q", "k", "v", "decay", "beta", "state"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("token", [0, 17, 64, 90, 149])
def test_delta_prompt_what_came_before_is_not_reached(what, bad, token):
    args, at = prompt_case([70, 150, 66], 2, 4, 64, 10)
    want, want_state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    t, x = at[1] + token, float(bad)
    if what == "state":
        args[5][1, 2, 3, 5] = x
        t = at[1]
    else:
        args[dict(q=0, k=1, v=2, decay=3, beta=4)[what]][(t, 1, 5) if what in "qkv" else (t, 1)] = x
    got, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    heads = dict(q=slice(2, 4), k=slice(2, 4), v=slice(1, 2), decay=slice(1, 2), beta=slice(1, 2), state=slice(2, 3))[what]
    cols = slice(5, 6) if what in ("v", "state") else slice(None)
    rows = slice(t, t + 1) if what == "q" else slice(t, at[2])
    assert not torch.isfinite(got[rows, heads, cols]).any()
    got[rows, heads, cols] = want[rows, heads, cols]
    assert torch.equal(got, want)
    if what != "q":
        assert not torch.isfinite(state[1, heads, :, cols]).any()
        state[1, heads, :, cols] = want_state[1, heads, :, cols]
    assert torch.equal(state, want_state)
    fine()


def test_delta_prompt_is_the_same_every_time_and_as_token_by_token():
    args, at = prompt_case([200, 200], 2, 4, 128, 11)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    ws = B.delta_prompt_workspace(400, 2, 2, 4, 128)
    o2, s2 = torch.zeros_like(out), torch.zeros_like(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.hc_delta_prompt(*args, out=o2, state_out=s2, ws=ws)
    for _ in range(3):
        o2.zero_(), s2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(s2, state)
    step = [x.unflatten(0, (2, 200)) for x in args[:5]]
    o3, s3 = B.hc_delta_step(*step, args[5], state_out=torch.empty_like(state))
    assert (s3 - state).norm() <= 1e-4 * state.norm()
    assert (o3.flatten(0, 1).float() - out.float()).norm() <= 2e-3 * out.float().norm()
    fine()


def test_delta_prompt_starts_out_of_range():
    args, at = prompt_case([50, 60, 70], 1, 1, 64, 12)
    want, want_state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    out = torch.full_like(want, 7.0)
    state = torch.zeros_like(want_state)
    B.hc_delta_prompt(*args[:6], torch.tensor([-1, 50, 110, 181], device="cuda", dtype=torch.int32), out=out, state_out=state)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert (out[:50] == 7).all() and (out[110:] == 7).all() and torch.equal(out[50:110], want[50:110])
    assert torch.equal(state[0], args[5][0]) and torch.equal(state[2], args[5][2]) and torch.equal(state[1], want_state[1])


# ------------------------------------------------------------------ log probabilities

def logit_rows(kind, n, v, seed, dtype):
    g = gen(seed)
    x = torch.randn(n, v, generator=g, device="cuda") * (torch.rand(n, 1, generator=g, device="cuda") * 4 + 0.5)
    if kind == "ruled out":
        out = torch.rand(n, v, generator=g, device="cuda") < 0.9
        out[:, v // 2] = False
        x = x.masked_fill(out, float("-inf"))
    elif kind == "lowest":  # masks of the type's lowest value
        x = x.masked_fill(torch.rand(n, v, generator=g, device="cuda") < 0.5, torch.finfo(dtype).min)
        x[:, v // 3] = 1.0
    elif kind == "equal":
        x = torch.full_like(x, 2.5)
    elif kind == "rising":
        x = x.sort(-1).values
    elif kind == "falling":
        x = x.sort(-1, descending=True).values
    elif kind == "few values":
        x = (x * 2).round() / 2
        x[:, ::2] *= -1.0  # zeros of both signs
    elif kind == "one":
        x = x - 60.0
        x[:, v - 1] = 3.0
    elif kind == "large":
        x = x * 1e4
    return x.to(dtype)


def check_logprobs(x, tokens, top, got):
    logp, entropy, ids, best = got
    n, v = x.shape
    rows = P.f64(x.float())
    r = (v / 1024 + 100) * U32
    for i in range(n):
        lp, h, log_z, spread, order = P.logprobs(rows[i])
        d = rows[i] - rows[i].max()
        if tokens is not None:
            t = tokens[i].cpu().numpy()
            for j, tok in enumerate(t):
                have = float(logp[i, j])
                if tok < 0:
                    assert have == 0
                elif np.isneginf(lp[tok]):
                    assert have == -np.inf
                else:
                    assert abs(have - lp[tok]) <= r + 4 * U32 * (abs(d[tok]) + abs(lp[tok])), (i, j)
        assert abs(float(entropy[i]) - h) <= r * (1 + h + log_z) + 4 * U32 * (spread + h), (i, float(entropy[i]), h)
        if top:
            assert ids[i].tolist() == order[:top].tolist(), i
            want = lp[order[:top]]
            have = P.f64(best[i])
            assert np.array_equal(np.isneginf(want), np.isneginf(have))
            ok = np.isfinite(want)
            assert np.all(np.abs(have - want)[ok] <= (r + 4 * U32 * (np.abs(d[order[:top]]) + np.abs(want)))[ok])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [1, 2, 7, 33, 1000, 2047, 4096, 8191, 8193, 32768, 50001])
@pytest.mark.parametrize("n", [1, 3, 160])
def test_logprobs_sizes(dtype, v, n):
    if n * v > 2_000_000 and n > 3:
        n = 80  # rows shared by two blocks
    x = logit_rows("plain", n, v, v + n, dtype)
    j = 1 + v % 3
    tokens = torch.randint(0, v, (n, j), generator=gen(v), device="cuda", dtype=torch.int32)
    top = min(v, 20)
    check_logprobs(x, tokens, top, B.hc_logprobs(x, tokens, top=top))
    fine()


@pytest.mark.parametrize("kind", ["ruled out", "lowest", "equal", "rising", "falling", "few values", "one", "large"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v,top", [(2, 40000, 32), (1, 128001, 32), (155, 20003, 7), (3, 40, 32), (1, 32, 32), (4, 70001, 1)])
def test_logprobs_distributions(kind, dtype, n, v, top):
    x = logit_rows(kind, n, v, 11, dtype)
    tokens = torch.randint(-1, v, (n, 3), generator=gen(v), device="cuda", dtype=torch.int32)
    tokens[:, 0] = -1
    check_logprobs(x[:6], tokens[:6], top, [t[:6] for t in B.hc_logprobs(x, tokens, top=top)])
    fine()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [3, 170])
def test_logprobs_rows_anywhere(dtype, n):
    """Rows at a stride, from any element on, and more tokens than a block has threads; rows' neighbours are not read
    as theirs."""
    wide = torch.full((n, 9100), float("nan"), device="cuda", dtype=dtype)
    for first, v in ((0, 9001), (1, 9000), (3, 8999), (5, 17), (7, 9)):
        x = wide[:, first:first + v]
        x.copy_(logit_rows("plain", n, v, first, dtype))
        tokens = torch.randint(0, v, (n, 700), generator=gen(v), device="cuda", dtype=torch.int32)
        got = B.hc_logprobs(x, tokens, top=5)
        check_logprobs(x[-3:], tokens[-3:], 5, [t[-3:] for t in got])
        wide.fill_(float("nan"))
    fine()


def test_logprobs_outputs_that_are_left_out():
    x = logit_rows("plain", 6, 3000, 1, torch.float32).view(2, 3, 3000)
    tokens = torch.randint(0, 3000, (2, 3, 2), generator=gen(1), device="cuda", dtype=torch.int32)
    logp, entropy, ids, best = B.hc_logprobs(x, tokens, top=4)
    assert logp.shape == (2, 3, 2) and entropy.shape == (2, 3) and ids.shape == best.shape == (2, 3, 4)
    a = B.hc_logprobs(x)
    assert a[0] is a[2] is a[3] is None and torch.equal(a[1], entropy)
    a = B.hc_logprobs(x, top=4)
    assert a[0] is None and torch.equal(a[2], ids) and torch.equal(a[3], best)
    a = B.hc_logprobs(x, tokens)
    assert torch.equal(a[0], logp) and a[2] is None
    fine()


@pytest.mark.parametrize("n", [5, 200])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_logprobs_rows_that_are_no_distribution(n, dtype):
    v = 9000
    x = logit_rows("plain", n, v, 2, dtype)
    tokens = torch.randint(0, v, (n, 2), generator=gen(3), device="cuda", dtype=torch.int32)
    want = B.hc_logprobs(x, tokens, top=3)
    fine()
    x[1, 8500] = float("nan")
    x[2, 3] = float("inf")
    x[3] = float("-inf")
    got = B.hc_logprobs(x, tokens, top=3)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    for g, w in zip(got, want):
        bad, keep = g[1:4], [0] + list(range(4, n))
        assert (bad == -1).all() if g.dtype == torch.int32 else bad.isnan().all()
        assert torch.equal(g[keep], w[keep])
    tokens[0, 1] = v
    got = B.hc_logprobs(x[:1], tokens[:1], top=3)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert got[0][0, 1].isnan() and torch.equal(got[0][0, 0], want[0][0, 0])


def test_logprobs_match_the_exit():
    """On the logits that the exit writes, the most probable token is what a greedy verification takes."""
    x = logit_rows("plain", 4, 32768, 5, torch.float32)
    _, _, ids, best = B.hc_logprobs(x, top=1)
    _, _, token = B.hc_verify(x[:, None].contiguous(), torch.zeros(4, 1, device="cuda", dtype=torch.int32))
    assert torch.equal(ids[:, 0], token)
    logp, *_ = B.hc_logprobs(x, ids)
    assert torch.equal(logp, best)
