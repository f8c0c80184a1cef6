"""The operators together, as examples/speculative_decode.py runs them: drafted trees through the stack."""
import os
import sys

import pytest
import torch

from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import speculative_decode as S  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def model():
    require_gpu()
    B.device_status()
    return S.Decoder(V=512)


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_greedy_tokens_are_the_targets_own(model, kind):
    """Every token is the argmax of what one pass over the whole sequence, as a chain, has after the tokens
    before it. The two passes differ by the roundings of bf16 activations (2^-8 each, some ten in a row, against
    logits of standard deviation about 1): a token may fall short of the largest logit by 0.1 at most."""
    prompt = torch.randint(model.V, (3, 21), generator=torch.Generator().manual_seed(2)).int().cuda()
    made, caches, ctx, steps = S.generate(model, prompt, 30, kind=kind)
    assert steps < 30 and all(len(m) >= 30 for m in made)
    for i, row in enumerate(made):
        assert int(ctx[i]) == prompt.shape[1] + len(row) - 1  # the last token is the next step's root
        tokens = torch.cat([prompt[i].cpu(), torch.tensor(row[:-1], dtype=torch.int32)])[None].cuda()
        n = tokens.shape[1]
        fresh = model.caches(kind, 1, n)
        zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        logits = model.logits(tokens, fresh, zero, torch.arange(n, dtype=torch.int32, device="cuda")[None])[0]
        after = logits[prompt.shape[1] - 1:]
        short = after.max(-1).values - after[torch.arange(len(row)), torch.tensor(row, device="cuda")]
        assert float(short.max()) <= 0.1
        # and the cache holds the accepted tokens' rows, in order: those of the one pass, up to the same roundings
        if kind == "bf16":
            where = torch.zeros(3, dtype=torch.int32, device="cuda")
            for a, z in zip(caches, fresh):
                have, want = B.hc_kv_read(a, where, n)[0][i], B.hc_kv_read(z, zero, n)[0][0]
                assert float((have.float() - want.float()).abs().max()) <= 0.1 * float(want.float().abs().max())
    assert B.device_status() == B.TS_OK


def test_sampled_tokens_follow_the_seed(model):
    prompt = torch.randint(model.V, (2, 9), generator=torch.Generator().manual_seed(3)).int().cuda()
    a = S.generate(model, prompt, 20, kind="fp8", temperature=0.8, seed=5)[0]
    b = S.generate(model, prompt, 20, kind="fp8", temperature=0.8, seed=5)[0]
    c = S.generate(model, prompt, 20, kind="fp8", temperature=0.8, seed=6)[0]
    assert a == b and a != c
    assert all(0 <= x < model.V for row in a for x in row)
