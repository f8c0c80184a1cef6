"""The verification tests' inputs, on the CPU: a sequence whose decisions are nearer than 1e-4 is passed over
there, so none may be."""
import numpy as np
import pytest

import spec_reference as R
from test_gpu_spec import verify_inputs

CASES = [(b, t, v, tree, [0.7, 1.0, 0.0, 1.3], {}, b + t)
         for b, t, v in [(1, 1, 1000), (1, 5, 32768), (3, 9, 50), (40, 6, 1), (7, 40, 2049), (160, 4, 501), (20, 5, 70001)]
         for tree in (False, True)]
CASES += [(2, t, v, tree, [0.9, 0.0], dict(agree=0.3), t) for t, v, tree in [(1024, 60, True), (1025, 60, False), (1500, 300, True), (4096, 20, True)]]


@pytest.mark.parametrize("b,t,v,tree,temps,kw,seed", CASES)
def test_no_sequence_is_passed_over(b, t, v, tree, temps, kw, seed):
    logits, tokens, parents, temp, draft, u, noise = verify_inputs(seed, b, t, v, tree, temps, **kw)
    for i in range(b):
        d64 = lambda x: x[i].astype(np.float64)  # noqa: E731
        assert R.verify(d64(logits), tokens[i], parents[i], float(temp[i]), d64(draft), d64(u), d64(noise))[3] >= 1e-4
