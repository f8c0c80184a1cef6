"""GPU tests of the speculative decoding step's operators at the ends of their ranges. Tolerances are
test_gpu_spec's, with what a test adds to them derived beside it."""
import numpy as np
import pytest
import torch

import spec_reference as R
from gpu_common import require_gpu
from hyper_connection_residual_call_gb300 import binding as B
from test_gpu_spec import U16, gen, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()
    B.device_status()


def bf16_bits(*bits):
    return torch.tensor(np.array(bits, np.uint16).view(np.int16)).cuda().view(torch.bfloat16)


def zeros(n=1):
    return torch.zeros(n, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ the cache's largest finite values

@pytest.mark.parametrize("group", [32, 64, 128])
def test_int4_largest_finite_values_saturate(group):
    """The lowest and the highest finite bf16, each beside ordinary elements and both in one group."""
    g = gen(40)
    cache = make_cache(g, "int4", 1, 16, 1, 16, 128, group)
    x = randn(g, 1, 6, 1, 128)
    low, high, next_low = bf16_bits(0xFF7F, 0x7F7F, 0xFF7E)
    x[0, 0, 0, 5], x[0, 1, 0, 70], x[0, 2, 0, 3] = low, high, next_low
    x[0, 3, 0, 9], x[0, 3, 0, 10] = low, high
    x[0, 4], x[0, 5] = low, high
    B.hc_kv_write(x, x, cache, zeros())
    want = R.stored(R.f64(x), "int4", group)
    assert np.isfinite(want).all()
    for got in B.hc_kv_read(cache, zeros(), 6):
        assert (np.abs(R.f64(got) - want) <= U16 * np.abs(want) + 1e-6).all()
    out, lse = B.hc_tree_attention(x[:, :1] * 0, cache, zeros() + 5)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    assert B.device_status() == B.TS_OK
