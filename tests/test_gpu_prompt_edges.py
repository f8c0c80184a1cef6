"""GPU tests of the prompt operators on a busy GPU and in the branches that only some sizes take; limits are
test_gpu_prompt's, or stand beside the test."""
import pytest
import torch

from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B
from test_gpu_prompt import check_logprobs, check_prompt, fine, gen, logit_rows, prompt_case, prompts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


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
