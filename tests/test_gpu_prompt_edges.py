"""GPU tests of the prompt operators on a busy GPU and in the branches that only some sizes take; limits are
test_gpu_prompt's, or stand beside the test."""
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
