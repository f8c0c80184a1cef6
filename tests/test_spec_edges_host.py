"""Refusals of the speculative decoding step's entry points that test_spec_host does not have: every call here
fails argument validation, so no CUDA call is made."""
import pytest

from hyper_connection_residual_call_gb300 import binding as B
from hyper_connection_residual_call_gb300.build import build

FAKE = 0x10000  # an aligned address that is never dereferenced: validation fails first


@pytest.fixture(scope="module", autouse=True)
def lib():
    build()
    return B.library()


@pytest.mark.parametrize("at,needle", [(0x20000, "new_len overlaps n_accepted"), (0x20004, "new_len overlaps n_accepted"),
                                       (0x30000, "new_len overlaps path"), (0x3005C, "new_len overlaps path"), (0xFFF8, "new_len overlaps ctx_len")])
def test_compact_refuses_a_new_len_that_is_still_read(at, needle):
    """Three sequences of eight nodes: n_accepted has 12 bytes at 0x20000, path 96 at 0x30000."""
    c = B.TsHcKvCache(B.TS_KV_BF16, 0, 16, 4, 128, 10, 100, FAKE, FAKE, None, None, None, None, FAKE)
    assert B.ts_hc_kv_compact(c, FAKE, 0x30000, 0x20000, at, 3, 8, None) == B.TS_ERR_INVALID_ARG
    assert needle in B.ts_hc_last_error()
