"""The packed-sequence operators on inputs where a score, a weight or a code is at the end of its range.

Tolerances as in test_gpu_operators.py: bounds from the arithmetic, u = 2^-24.
"""
import math

import pytest
import torch

import test_gpu_operators as ops
from persistent_sm_decode_02_b200 import dec as D_
from test_gpu_operators import DT, U, Pool, gen, run_paged, run_prefill

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


# ------------------------------------------------------------------------------------------------ paged attention
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,first", [(40, 16), (40, 17), (33, 32), (600, 100), (600, 590), (9000, 4000), (40, 40), (9000, 9000)])
def test_paged_scores_that_overflow_weigh_nothing(n, first, dtype):
    """The first positions' scores pass fp32's range (-infinity), the others' are 0: the mean of the others' values, to the
    rounding of equal weights (none: powers of two) and their sum; NaN where there are no others."""
    h, hkv, d, ps = 4, 2, 64, 16
    pool = Pool([n, n], hkv, d, ps, 210).fill([n, n], 211)
    for b in range(2):
        ids = pool.table[b].long()
        pool.k[ids, :, :, 0] = 0
        flat = torch.arange(len(ids) * ps, device="cuda").view(-1, ps)
        low = (flat < first)[:, None, :].expand(-1, hkv, -1)
        page = pool.k[ids]
        page[..., 0] = torch.where(low, 0x7E, 0).to(torch.uint8)  # 448
        pool.k[ids] = page
        pool.ks[ids] = 2.0 ** 30
    q = torch.zeros(2, h, d, device="cuda")
    q[0, :, 0] = -1e30  # score -1e30 * 448 * 2^30 / 8
    q = q.to(DT[dtype][0])
    out = torch.empty_like(q)
    run_paged(pool, q, out, [n, n], dtype)
    if first == n:
        assert bool(torch.isnan(out[0]).all())
    else:
        _, v = pool.rows(0, n)
        v = v[:, first:].repeat_interleave(h // hkv, 0)
        ref, a = v.mean(1), v.abs().mean(1)
        assert bool(((out[0].double() - ref).abs() <= DT[dtype][2] * ref.abs() + a * (2.0 ** -20 + n * U)).all())
    _, v = pool.rows(1, n)  # scores of 0 throughout
    v = v.repeat_interleave(h // hkv, 0)
    ref, a = v.mean(1), v.abs().mean(1)
    assert bool(((out[1].double() - ref).abs() <= DT[dtype][2] * ref.abs() + a * (2.0 ** -20 + n * U)).all())


def test_paged_no_page_to_read_gives_zeros():
    """A sequence whose every page id is bad has no position to see."""
    h, hkv, d, ps, lens = 4, 2, 64, 16, [40, 700]
    pool = Pool(lens, hkv, d, ps, 212).fill(lens, 213)
    table = pool.table.clone()
    table[1] = pool.n_pages
    q = torch.randn(2, h, d, generator=gen(214), device="cuda")
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    run_paged(pool, q, out, lens, "f32", table=table, status=status)
    assert int(status) == D_.DEC_SEQ_BAD_PAGE and bool((out[1] == 0).all())
    ops.check_paged(pool, q[:1], out[:1], lens[:1], "f32")


@pytest.mark.parametrize("dtype,down", [("bf16", 20), ("bf16", 26), ("f32", 20), ("f32", 29)])
def test_paged_small_weights_keep_their_bits(dtype, down):
    """One key takes the weight and has the value zero; what is left are weights about 2^-down of it.  Sequences as many as
    there are pieces of the line, so that one piece sees both."""
    h, hkv, d, ps, n, n_seqs = 4, 1, 64, 16, 63 * 16, 1776
    pool = Pool([32], hkv, d, ps, 220).fill([32], 221)
    strong, weak = (int(x) for x in pool.table[0])
    pool.table = torch.full((n_seqs, n // ps), weak, dtype=torch.int32, device="cuda")
    pool.table[:, 0] = strong
    pool.width, pool.n_pages = n // ps, pool.k.shape[0]
    pool.k[[strong, weak]] = 0
    pool.k[strong, :, 5, 0] = 0x38  # 1
    pool.v[strong] = 0
    pool.ks[[strong, weak]] = 1.0
    pool.vs[[strong, weak]] = 1.0
    score = torch.linspace(down - 1, down, 37, dtype=torch.float64, device="cuda") * math.log(2)
    q = torch.zeros(n_seqs, h, d, device="cuda")
    q[:, :, 0] = (score[torch.arange(n_seqs, device="cuda") % 37] * 8).float()[:, None]
    q = q.to(DT[dtype][0])
    out = torch.empty_like(q)
    run_paged(pool, q, out, [n] * n_seqs, dtype)
    w = torch.exp(-q[:, :, 0].double() / 8)  # of each of the others, against the one's 1
    _, v = pool.rows(0, 32)
    ref = (w * (n // ps - 1))[..., None] * v[0, 16:].sum(0) / (1 + w * (n - 1))[..., None]
    a = (w * (n // ps - 1))[..., None] * v[0, 16:].abs().sum(0) / (1 + w * (n - 1))[..., None]
    # a score is off by (scaling by log2 e, the hardware's 2^x) 2 u of itself
    tol = DT[dtype][2] * ref.abs() + a * ((2.0 ** -11 if dtype == "bf16" else 2.0 ** -20) + 4 * U * down + 2.0 ** -20 + n * U)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
