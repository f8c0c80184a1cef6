"""GPU tests of the prompt operators on a busy GPU and in the branches that only some sizes take; limits are
test_gpu_prompt's, or stand beside the test."""
import numpy as np
import pytest
import torch

import prompt_reference as P
from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B
from test_gpu_prompt import U16, U32, check_logprobs, check_prompt, fine, gen, logit_rows, prompt_case, prompts, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


# ------------------------------------------------------------------ head norms

@pytest.mark.parametrize("n,hq,hk,d,rot", [(9001, 9, 0, 128, 64), (9001, 32, 8, 128, 128), (17401, 7, 2, 64, 32), (2500, 16, 1, 256, 256),
                                           (5003, 16, 1, 128, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_norm_rope_threads_that_walk_over_heads(n, hq, hk, d, rot, interleaved, in_place):
    """Tokens and heads enough that a thread walks over up to eight heads, an odd number of them too: the same bits as of 100
    tokens at a time, where it has one; and some rows against the formula (test_gpu_prompt's limit)."""
    g = gen(n)
    x = randn(g, n, hq + 2 * hk, d, scale=1.7)
    q, k = x[:, :hq], x[:, hq:hq + hk] if hk else None
    w = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    table = B.rope_table(500, rot, 10000.0)
    pos = torch.randint(0, 500, (n,), generator=g, device="cuda", dtype=torch.int32)
    rows = [0, 1, n // 2, n - 2, n - 1]
    before = [P.f64(t[rows]) if t is not None else None for t in (q, k)]
    parts = [B.hc_qk_norm_rope(q[a:a + 100], k[a:a + 100] if hk else None, pos[a:a + 100], table, w[0], w[1] if hk else None,
                               interleaved=interleaved) for a in range(0, n, 100)]
    rest = x[:, hq + hk:].clone()
    out = B.hc_qk_norm_rope(q, k, pos, table, w[0], w[1] if hk else None, interleaved=interleaved,
                            **(dict(q_out=q, k_out=k) if in_place else {}))
    for i in range(2 if hk else 1):
        assert torch.equal(out[i], torch.cat([p[i] for p in parts]))
        normed, want = P.norm_rope(before[i], P.f64(w[i]), 1e-6, pos[rows].cpu().numpy(), P.f64(table), interleaved)
        pair, r = np.abs(normed), rot // 2
        i0, i1 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(r), np.arange(r) + r)
        pair[..., i0] = pair[..., i1] = pair[..., i0] + pair[..., i1]
        within(out[i][rows], want, U16 * np.abs(want) + (d + 16) * U32 * pair + 1e-38, "head norms")
    assert torch.equal(rest, x[:, hq + hk:])
    fine()


# ------------------------------------------------------------------ attention over packed prompts

@pytest.mark.parametrize("n,s,hq", [(5000, 3, 1), (3000, 601, 1), (700, 65535, 32)])
def test_attention_sequences_that_overlap(n, s, hq):
    """Each other sequence claims all rows, those between end before they begin: recorded, rows hold the result or what was
    there, and nothing beside them is written."""
    q, k, v, starts, at = prompts([n], hq, 1, 64, 61)
    want, want_lse = B.hc_prompt_attention(q, k, v, starts)
    fine()
    wide, lse = torch.full((n + 512, hq, 64), 7.0, device="cuda").bfloat16(), torch.full((n + 512, hq), 7.0, device="cuda")
    over = torch.arange(s + 1, device="cuda", dtype=torch.int32) % 2 * n
    B.hc_prompt_attention(q, k, v, over, out=wide[256:256 + n], lse=lse[256:256 + n])
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    for got, right in ((wide, want), (lse, want_lse)):
        assert (got[:256] == 7).all() and (got[256 + n:] == 7).all()
        mine = got[256:256 + n]
        assert ((mine == right) | (mine == 7)).all() and (mine == right).any()


# ------------------------------------------------------------------ the delta rule's segments

@pytest.mark.parametrize("hk,hv,d,lens", [(1, 1, 64, [16000]), (2, 4, 128, [9000]), (1, 2, 64, [5000, 7000])])
def test_segments_on_a_busy_gpu(hk, hv, d, lens):
    """Other work on another stream holds SMs, so that some of a launch's walks start late: the same bits as alone."""
    args, at = prompt_case(lens, hk, hv, d, 21, low=0.1)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    ws = B.delta_prompt_workspace(sum(lens), len(lens), hk, hv, d)
    side = torch.cuda.Stream()
    x = torch.randn(4096, 4096, device="cuda").bfloat16()
    outs = [torch.zeros_like(out) for _ in range(8)]
    states = [torch.zeros_like(state) for _ in range(8)]
    y = torch.empty_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(40):
            torch.mm(x, x, out=y)
    for o, s in zip(outs, states):
        B.hc_delta_prompt(*args, out=o, state_out=s, ws=ws)
    torch.cuda.synchronize()
    for o, s in zip(outs, states):
        assert torch.equal(o, out) and torch.equal(s, state)
    fine()


@pytest.mark.parametrize("hk,hv,d,n", [(1, 1, 64, 2700), (4, 8, 128, 5000)])
def test_segments_read_what_was_just_written(hk, hv, d, n):
    """All inputs are written by the kernels just before, other ones each time, in a graph and without; the workspace
    holds all ones before, as it may."""
    cases = [prompt_case([n], hk, hv, d, 41 + i, low=0.1)[0] for i in range(3)]
    want = [B.hc_delta_prompt(*c, state_out=torch.empty_like(c[5])) for c in cases]
    args = [torch.zeros_like(x) for x in cases[0]]
    ws = B.delta_prompt_workspace(n, 1, hk, hv, d)
    ws.view(torch.int32)[:] = 1
    out, state = torch.zeros_like(want[0][0]), torch.zeros_like(args[5])
    kept = [(torch.zeros_like(out), torch.zeros_like(state)) for _ in cases]

    def all_cases():
        for c, (o, s) in zip(cases, kept):
            for mine, x in zip(args, c):
                mine.copy_(x)
            B.hc_delta_prompt(*args, out=out, state_out=state, ws=ws)
            for mine in args:  # nobody reads them any more
                mine.zero_()
            o.copy_(out)
            s.copy_(state)

    def check():
        torch.cuda.synchronize()
        for (o, s), (wo, w) in zip(kept, want):
            assert torch.equal(o, wo) and torch.equal(s, w)
            o.zero_(), s.zero_()

    for _ in range(5):
        all_cases()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        all_cases()
    for _ in range(5):
        ws.view(torch.int32)[:] = 1
        graph.replay()
    check()
    fine()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low", [0.0, 0.02, 0.5])
@pytest.mark.parametrize("hv,lens", [(60, [130]), (2, [700]), (2, [1800]), (1, [2000, 4]), (1, [2700])])
def test_states_have_22_bits(d, low, hv, lens):
    """The states' relative error in the Frobenius norm, of chunks in one walk, in segments, and in segments whose last are
    prepared beside the walks. What goes into a state is off by 2^-23 of its column's largest at most, uniformly: an operand
    by some 2^-24 rms, five of them on the way (the state, M, R, T, U); the tensor cores' fp32 sums of 64 to 128 terms by some
    sqrt(128) 2^-25. Together 4e-7 of what a chunk adds, and the state holds the chunks' errors as it holds what they added: 1e-6
    over the dozens here, with the segments' joins twice that. A part of 11 bits left out, 2^-12 rms of an operand, would be 1e-4; two
    parts of bf16 (16 bits), 2^-18 rms of each operand, 9e-6. The limit is between: 2^-18."""
    args, at = prompt_case(lens, 1, hv, d, d + hv + lens[0], low=low)
    _, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    q, k, v, decay, beta, before = (P.f64(x) for x in args[:6])
    heads = [0, hv - 1] if hv > 2 else list(range(hv))
    for i, (lo, hi) in enumerate(zip(at[:-1], at[1:])):
        _, after, _ = P.delta(q[lo:hi], k[lo:hi], v[lo:hi][:, heads], decay[lo:hi][:, heads], beta[lo:hi][:, heads], before[i][heads], 1.0, 1e-6)
        err = np.linalg.norm(P.f64(state[i, heads]) - after) / np.linalg.norm(after)
        print(f"D {d} low {low} {hi - lo} tokens: {err:.3g}")
        assert err <= 2.0 ** -18
    fine()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-30])
def test_keys_of_zeros_leave_the_others_their_bits(d, eps):
    """Keys and queries of zeros, as padding has them, beside others, whatever the epsilon that their norms are: the limits of
    test_states_have_22_bits, and of test_gpu_prompt for the outputs."""
    args, at = prompt_case([200], 1, 2, d, 81, low=0.1)
    for x in args[:2]:
        x[[0, 5, 70, 71, 150, 199]] = 0
    out, state = B.hc_delta_prompt(*args, norm_eps=eps, state_out=torch.empty_like(args[5]))
    q, k, v, decay, beta, before = (P.f64(x) for x in args[:6])
    _, after, _ = P.delta(q, k, v, decay, beta, before[0], 1.0, eps)
    assert np.linalg.norm(P.f64(state[0]) - after) <= 2.0 ** -18 * np.linalg.norm(after)
    check_prompt(args, at, out, state, eps)
    fine()


@pytest.mark.parametrize("token", [0, 70, 129])
def test_keys_and_queries_past_the_range_of_their_squares(token):
    """They count as zeros, in chunks and token by token; without an epsilon zeros have no direction."""
    args, at = prompt_case([130], 1, 2, 64, 71)
    huge, zero = [x.clone() for x in args[:6]], [x.clone() for x in args[:6]]
    for i in range(2):
        huge[i][token] = args[i][token] * 2.0 ** 70
        zero[i][token] = 0
    a, sa = B.hc_delta_prompt(*huge, args[6], state_out=torch.empty_like(args[5]))
    z, sz = B.hc_delta_prompt(*zero, args[6], state_out=torch.empty_like(args[5]))
    assert torch.equal(a, z) and torch.equal(sa, sz) and not a[token].any()
    a, sa = B.hc_delta_step(*(x[None] for x in huge[:5]), huge[5], state_out=torch.empty_like(args[5]))
    z, sz = B.hc_delta_step(*(x[None] for x in zero[:5]), zero[5], state_out=torch.empty_like(args[5]))
    assert torch.equal(a, z) and torch.equal(sa, sz) and not a[0, token].any()
    a, sa = B.hc_delta_prompt(*zero, args[6], norm_eps=0.0, state_out=torch.empty_like(args[5]))
    z, sz = B.hc_delta_step(*(x[None] for x in zero[:5]), zero[5], norm_eps=0.0, state_out=torch.empty_like(args[5]))
    for out, state in ((a, sa), (z[0], sz)):
        assert out[token:].isnan().all() and state.isnan().all() and torch.isfinite(out[:token]).all()
    fine()


def test_one_workspace_serves_smaller_calls():
    ws = B.delta_prompt_workspace(6000, 6, 1, 2, 64)
    for lens in ([6000], [3000, 2900], [100, 5, 1, 0, 9, 300], [1], [2000, 1, 1, 1, 1, 1]):
        args, at = prompt_case(lens, 1, 2, 64, 51, low=0.1)
        want, want_state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
        out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]), ws=ws)
        assert torch.equal(out, want) and torch.equal(state, want_state)
    fine()


# ------------------------------------------------------------------ log probabilities

@pytest.mark.parametrize("kind", ["plain", "ruled out", "lowest", "equal", "rising", "falling", "few values", "one", "large"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [3, 5, 32])
def test_logprobs_second_threshold(kind, dtype, top):
    """Rows of seven chunks a CTA, two blocks a SM: the alternatives' second threshold, from the fourth chunk on, in any
    order of a row's elements; and the same bits call after call."""
    n, v = 330, 50001
    x = logit_rows(kind, n, v, 31, dtype)
    tokens = torch.randint(0, v, (n, 1), generator=gen(v), device="cuda", dtype=torch.int32)
    got = B.hc_logprobs(x, tokens, top=top)
    for rows in (slice(0, 2), slice(303, 306), slice(n - 1, n)):
        check_logprobs(x[rows], tokens[rows], top, [t[rows] for t in got])
    for _ in range(4):
        for a, z in zip(B.hc_logprobs(x, tokens, top=top), got):
            assert torch.equal(a, z)
    # the other rows against one sort (stable: of equal ones the lowest index)
    order = (x.float() + 0.0).sort(dim=-1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(got[2].long(), order)
    fine()


@pytest.mark.parametrize("kind", ["plain", "ruled out", "lowest", "equal", "rising", "falling", "few values", "one"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(20, 20003), (60, 20003), (10, 131072), (38, 100003)])
def test_logprobs_rows_of_two_and_four_ctas(kind, dtype, n, v):
    """Clusters of two and of four CTAs, some with a second threshold in each CTA's part."""
    x = logit_rows(kind, n, v, 32, dtype)
    tokens = torch.randint(0, v, (n, 2), generator=gen(v), device="cuda", dtype=torch.int32)
    got = B.hc_logprobs(x, tokens, top=20)
    check_logprobs(x[-3:], tokens[-3:], 20, [t[-3:] for t in got])
    order = (x.float() + 0.0).sort(dim=-1, descending=True, stable=True).indices[:, :20]
    assert torch.equal(got[2].long(), order)
    fine()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(1, 32768), (1, 40), (3, 7681), (20, 128001), (60, 20003), (330, 50001)])
@pytest.mark.parametrize("top", [0, 3])
def test_logprobs_of_a_token_that_is_nearly_certain(dtype, n, v, top):
    """Log probabilities and entropies near 0 keep their relative precision. All terms but the largest one's 1 are added up
    apart from it: with test_gpu_prompt's r for the sums, and e^d off by 2 |d| u32 + 2^-22 of itself (|d| of 64 at most), log Z is off
    by (r + 132 u32) of itself; from Z = 1.25 on, where it is the logarithm of a sum with the 1 in it, by r (1 + 1 / log 1.25) < 6 r of
    itself. S = sum d e^d likewise, with d's own error twice."""
    g, r = gen(n + v), (v / 1024 + 100) * U32
    x = torch.randn(n, v, generator=g, device="cuda")
    at = torch.randint(0, v, (n,), generator=g, device="cuda")
    at[0], at[-1] = 0, v - 1
    x[torch.arange(n, device="cuda"), at] = torch.linspace(13.0, 40.0, n, device="cuda") if n > 1 else 20.0
    x = x.to(dtype)
    logp, entropy, ids, best = B.hc_logprobs(x, at.int()[:, None], top=top)
    e = x.double() - x.double().amax(-1, keepdim=True)
    assert (e[torch.arange(n, device="cuda"), at] == 0).all() and (e < 0).sum() == n * (v - 1)
    z = torch.where(e < 0, e.exp(), 0.0).sum(-1)
    want = torch.log1p(z)
    h = want - (e * e.exp()).sum(-1) / (1 + z)
    assert ((logp[:, 0].double() + want).abs() <= (6 * r + 132 * U32) * want).all()
    assert ((entropy.double() - h).abs() <= (6 * r + 264 * U32) * h).all()
    if top:
        assert torch.equal(ids[:, 0].long(), at) and torch.equal(best[:, 0], logp[:, 0])
    fine()
