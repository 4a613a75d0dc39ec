"""The packed-sequence operators on inputs where a score, a weight or a code is at the end of its range.

Tolerances as in test_gpu_operators.py: bounds from the arithmetic, u = 2^-24.
"""
import math

import pytest
import torch

import test_gpu_operators as ops
from test_gpu_operators import run_prefill

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ prefill
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["infinite", "overflow"])
def test_prefill_rows_whose_every_score_is_minus_infinity(kind, d, causal, dtype):
    """They have no softmax, wherever the row is and however many whole steps of keys it sees: NaN.  Every other row has
    the bits it has beside ordinary rows."""
    h, hkv, n = 4, 2, 400
    q, k, v = ops.prefill_inputs(h, hkv, d, n, n, dtype, 200)
    k = k.abs() + 0.5
    clean, out = torch.empty_like(q), torch.empty_like(q)
    run_prefill(q, k, v, clean, [n], [n], dtype, causal)
    rows = [0, 1, 63, 64, 65, 127, 128, 129, 200, 255, 256, 300, 383, 384, 399]
    bad = torch.zeros(n, h, dtype=torch.bool, device="cuda")
    for i, r in enumerate(rows):
        bad[r, i % h] = True
    # -3e38 in every dim: a score below -3e38 * 0.5 * 64, past fp32's range
    q[bad] = -math.inf if kind == "infinite" else -3e38
    run_prefill(q, k, v, out, [n], [n], dtype, causal)
    assert bool(torch.isnan(out[bad]).all())
    assert torch.equal(out[~bad], clean[~bad])
