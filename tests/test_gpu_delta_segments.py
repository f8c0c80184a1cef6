"""The gated delta rule over long prompts of few heads, whose sequences the library cuts into segments (of eight
chunks of 64 tokens or more, from 24 chunks a sequence on) that are walked side by side: at the segments' ends,
beside short sequences, with bad values, strong decays and starts out of range, in place and in a graph. Against the
64-bit implementation, with test_gpu_prompt's limits: their term of the steps counts a rounding of the state a token
and 64 more, and a state that goes through a segment's F and B is rounded d + 16 times a segment more at the most,
which is fewer than a segment's 512 tokens."""
import pytest
import torch

from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B
from test_gpu_prompt import check_prompt, fine, prompt_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 4), (1, 3)])
@pytest.mark.parametrize("lens", [[1537], [2048], [2049], [1599], [3400, 5]])
def test_segments(d, hk, hv, lens):
    args, at = prompt_case(lens, hk, hv, d, sum(lens) + hv, low=0.2)
    before = args[5].clone()
    apart = torch.empty_like(before)
    out, _ = B.hc_delta_prompt(*args, state_out=apart)
    assert torch.equal(args[5], before)
    check_prompt(args, at, out, apart)
    again, state = B.hc_delta_prompt(*args[:5], before, args[6])  # in place
    assert state is before and torch.equal(state, apart) and torch.equal(again, out)
    fine()


@pytest.mark.parametrize("lens", [[0, 1, 6300, 0], [700, 1300, 0, 60, 7300, 512, 1024]])
def test_segments_beside_short_sequences(lens):
    args, at = prompt_case(lens, 1, 1, 64, len(lens), low=0.05)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state)
    fine()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low", [0.001, 60.0])
def test_segments_decays(d, low):
    args, at = prompt_case([1800], 1, 2, d, 3, low=low)
    args[3][[3, 511, 512, 1023, 1500]] = torch.tensor([float("-inf"), -200.0, -90.0, torch.finfo(torch.float32).min, -60.0], device="cuda")[:, None]
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    bounded = list(args)
    bounded[3] = args[3].clamp(min=-1e4)
    check_prompt(bounded, at, out, state)
    fine()


def test_segments_equal_keys():
    """All keys the same, beta 1 and no decay: what a segment makes of a state, it makes of it exactly once."""
    args, at = prompt_case([1700], 1, 1, 64, 7, low=0.0)
    args[1][:] = args[1][0].clone()
    args[4].fill_(1.0)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state)


def test_segments_leave_rows_behind():
    args, at = prompt_case([50, 3100], 1, 2, 128, 9, behind=300, low=0.2)
    for x in args[:5]:
        x[3150:] = float("nan")
    out = torch.full((3450, 2, 128), 7.0, device="cuda").bfloat16()
    _, state = B.hc_delta_prompt(*args, out=out, state_out=torch.empty_like(args[5]))
    assert (out[3150:] == 7).all()
    check_prompt([x[:3150] if i < 5 else x for i, x in enumerate(args)], at, out[:3150], state)
    fine()


@pytest.mark.parametrize("what", ["q", "k", "v", "decay", "beta", "state"])
@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("token", [0, 511, 512, 700, 1536, 4799])
def test_segments_what_came_before_is_not_reached(what, bad, token):
    args, at = prompt_case([70, 4800, 66], 2, 4, 64, 10, low=0.2)
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


def test_segments_are_the_same_every_time_and_as_token_by_token():
    args, at = prompt_case([1700], 2, 4, 128, 11, low=0.2)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    ws = B.delta_prompt_workspace(1700, 1, 2, 4, 128)
    ws.fill_(255)  # it need not be initialised
    o2, s2 = torch.zeros_like(out), torch.zeros_like(state)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.hc_delta_prompt(*args, out=o2, state_out=s2, ws=ws)
    for _ in range(3):
        o2.zero_(), s2.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(s2, state)
    step = [x[None] for x in args[:5]]
    o3, s3 = B.hc_delta_step(*step, args[5], state_out=torch.empty_like(state))
    assert (s3 - state).norm() <= 1e-4 * state.norm()
    assert (o3[0].float() - out.float()).norm() <= 2e-3 * out.float().norm()
    fine()


@pytest.mark.parametrize("first,last", [(-1, 5181), (-100000, 2**30)])
def test_segments_starts_out_of_range(first, last):
    args, at = prompt_case([50, 5060, 70], 1, 1, 64, 12)
    want, want_state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    out = torch.full_like(want, 7.0)
    state = torch.zeros_like(want_state)
    B.hc_delta_prompt(*args[:6], torch.tensor([first, 50, 5110, last], device="cuda", dtype=torch.int32), out=out, state_out=state)
    assert B.device_status() == B.TS_ERR_INVALID_ARG
    assert (out[:50] == 7).all() and (out[5110:] == 7).all() and torch.equal(out[50:5110], want[50:5110])
    assert torch.equal(state[0], args[5][0]) and torch.equal(state[2], args[5][2]) and torch.equal(state[1], want_state[1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hk,hv,lens", [(2, 4, [2600]), (1, 1, [5000, 2700, 300]), (4, 8, [2561])])
def test_segments_whose_last_are_prepared_beside_the_walks(d, hk, hv, lens):
    """From 40 chunks a sequence on and with SMs left idle; the same bits call after call, without a pause, on two streams."""
    args, at = prompt_case(lens, hk, hv, d, sum(lens), low=0.1)
    out, state = B.hc_delta_prompt(*args, state_out=torch.empty_like(args[5]))
    check_prompt(args, at, out, state)
    ws = [B.delta_prompt_workspace(sum(lens), len(lens), hk, hv, d) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    many = [B.hc_delta_prompt(*args, state_out=torch.zeros_like(args[5]), ws=ws[i % 2], stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for o, s in many:
        assert torch.equal(o, out) and torch.equal(s, state)
    # other inputs in between, in the same workspace: nothing of one call is left for the next
    other, _ = prompt_case(lens, hk, hv, d, 77, low=0.1)
    first = B.hc_delta_prompt(*other, state_out=torch.zeros_like(args[5]), ws=ws[0])
    again = B.hc_delta_prompt(*args, state_out=torch.zeros_like(args[5]), ws=ws[0])
    third = B.hc_delta_prompt(*other, state_out=torch.zeros_like(args[5]), ws=ws[0])
    assert torch.equal(again[0], out) and torch.equal(again[1], state)
    assert torch.equal(first[0], third[0]) and torch.equal(first[1], third[1])
    fine()


def test_segments_prepared_beside_the_walks_in_a_graph():
    """Inputs that the kernels just before have written, replay after replay."""
    args, at = prompt_case([3000], 2, 4, 128, 5, low=0.1)
    k, v = args[1].clone(), args[2].clone()
    out, state = torch.empty(3000, 4, 128, device="cuda").bfloat16(), torch.empty_like(args[5])
    ws = B.delta_prompt_workspace(3000, 1, 2, 4, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for scale in (1.0, 0.5):
            torch.mul(v, scale, out=args[2].copy_(v))
            args[1].copy_(k)
            B.hc_delta_prompt(*args, out=out, state_out=state, ws=ws)
    for _ in range(3):
        out.zero_(), state.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want, want_state = B.hc_delta_prompt(args[0], k, v * 0.5, *args[3:], state_out=torch.empty_like(state))
        assert torch.equal(out, want) and torch.equal(state, want_state)
    fine()
