"""The packed-sequence operators on inputs where a score, a weight or a code is at the end of its range.

Tolerances as in test_gpu_operators.py: bounds from the arithmetic, u = 2^-24.
"""
import math

import pytest
import torch

import persistent_sm_decode_02_b200 as pkg
import test_gpu_operators as ops
from persistent_sm_decode_02_b200 import dec as D_
from test_gpu_operators import DT, U, Pool, gen, ints, offsets, run_append, run_paged, run_prefill

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


@pytest.mark.parametrize("d,n", [(64, 5000), (128, 5000), (128, 30000)])
@pytest.mark.parametrize("what", ["value", "value_inf", "key", "late"])
def test_prefill_bf16_values_that_are_not_finite_in_a_long_prompt(what, d, n):
    """A NaN that nearly every row of a long prompt sees shows in its dim (value) or row (key) there; every other result of
    that prompt, and the prompt beside it, have the bits they have without it, and no wait runs out meanwhile."""
    h, hkv, lens = 4, 2, [n, 700]
    q, k, v = ops.prefill_inputs(h, hkv, d, sum(lens), sum(lens), "bf16", 260)
    clean, out = torch.empty_like(q), torch.empty_like(q)
    run_prefill(q, k, v, clean, lens, lens, "bf16")
    at = n // 2 + 3 if what == "late" else 0
    if what == "key":
        k[at, 0, 9] = math.nan
    else:
        v[at, 0, 9] = math.inf if what == "value_inf" else math.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_prefill(q, k, v, out, lens, lens, "bf16", status=status)
    assert int(status) == 0
    bad = torch.zeros_like(out, dtype=torch.bool)
    if what == "key":
        bad[at:n, :2] = True
    else:
        bad[at:n, :2, 9] = True
    if what == "value_inf":  # the weight of a far key may round to zero
        assert not bool(torch.isfinite(out[bad]).any()) and bool((out[at, :2, 9] == math.inf).all())
    else:
        assert bool(torch.isnan(out[bad]).all())
    same = ~bad
    tile = slice(at - at % 128, at)  # rows that share a step with it and do not see it are computed once more
    same[tile, :2] = False
    assert torch.equal(out[same], clean[same])
    if tile.stop > tile.start:
        k, v = k[:at], v[:at]
        seen = torch.arange(at, device="cuda")[None, :] <= torch.arange(tile.start, tile.stop, device="cuda")[:, None]
        ref, a, s = ops.attend64(*(t.double().transpose(0, 1) for t in (q[tile, :2], k[:, :1], v[:, :1])), d ** -0.5, seen)
        tol = ops.attend_tol(ref, a, s, at, d, "bf16", 2.0 ** -8)
        assert bool(((out[tile, :2].double().transpose(0, 1) - ref).abs() <= tol).all())


@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("h,hkv,d", [(4, 2, 64), (3, 1, 64), (4, 2, 128), (3, 3, 128)])
def test_prefill_bf16_bits_do_not_depend_on_what_lies_around(h, hkv, d, causal):
    """NaN and infinities in every key and value of the other prompts, and behind the last: the same bits."""
    lq, lk = [700, 77, 128, 333, 15, 250], [700, 77, 128, 400, 16, 257]
    q, k, v = ops.prefill_inputs(h, hkv, d, sum(lq), sum(lk) + 40, "bf16", 263)
    clean = torch.empty_like(q)
    run_prefill(q, k, v, clean, lq, lk, "bf16", causal, n_k=sum(lk) + 40)
    ops.check_prefill(q, k, v, clean, lq, lk, "bf16", causal)
    for b in range(len(lq)):
        q0, k0 = offsets(lq)[b], offsets(lk)[b]
        kk, vv = torch.full_like(k, math.nan), torch.full_like(v, math.nan)
        vv[::3] = math.inf
        kk[k0:k0 + lk[b]], vv[k0:k0 + lk[b]] = k[k0:k0 + lk[b]], v[k0:k0 + lk[b]]
        out = torch.empty_like(q)
        run_prefill(q, kk, vv, out, lq, lk, "bf16", causal, n_k=sum(lk) + 40)
        assert torch.equal(out[q0:q0 + lq[b]], clean[q0:q0 + lq[b]]), b


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_bf16_some_values_seen_some_not(d):
    """NaN in dim 3 of the first key, which every row sees, in dim 7 of a key inside the last tile, and in all dims of the
    next prompt's first keys: dim 3 is NaN, dim 7 from that key's row on, and all else is finite and right."""
    h, hkv, lens, at = 2, 1, [1000, 60], 950
    q, k, v = ops.prefill_inputs(h, hkv, d, sum(lens), sum(lens), "bf16", 261)
    v[0, 0, 3] = v[at, 0, 7] = math.nan
    v[1000:1003] = math.nan
    out = torch.empty_like(q)
    run_prefill(q, k, v, out, lens, lens, "bf16")
    assert bool(torch.isnan(out[:1000, :, 3]).all()) and bool(torch.isnan(out[at:1000, :, 7]).all())
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:1000, :, 3] = bad[at:1000, :, 7] = True
    v[0, 0, 3] = v[at, 0, 7] = 0.0
    n = 1000
    seen = torch.arange(n, device="cuda")[None, :] <= torch.arange(n, device="cuda")[:, None]
    ref, a, s = ops.attend64(*(t[:n].double().transpose(0, 1) for t in (q, k, v)), d ** -0.5, seen)
    ok = (out[:n].double().transpose(0, 1) - ref).abs() <= ops.attend_tol(ref, a, s, n, d, "bf16", 2.0 ** -8)
    assert bool((ok | bad[:n].transpose(0, 1)).all())
    assert bool(torch.isnan(out[1000:]).all())


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_bf16_largest_values(d):
    """Values of 1e36: weights count up to 2^8 of the row's largest, and their sum passes fp32's range; the result does not."""
    h, hkv, n = 2, 1, 300
    q, k, v = ops.prefill_inputs(h, hkv, d, n, n, "bf16", 262)
    v = (v.float().abs().clamp(0.5, 1.0) * 1e36).bfloat16()
    k[:200] *= 0.1
    out = torch.empty_like(q)
    run_prefill(q, k, v, out, [n], [n], "bf16")
    ops.check_prefill(q, k, v, out, [n], [n], "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6, 1e8, 1e10, 1e15])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_scores_of_any_finite_size(d, size, dtype):
    """Keys along one direction: the longest seen has all the weight, its value is the result (rounded once; sums of one
    weight of any size and zeros are exact to 2^-20 and, on the tensor cores, the weight's rounding)."""
    h, hkv, n = 4, 2, 300
    g = gen(270)
    sign = torch.randint(0, 2, (d,), generator=g, device="cuda") * 2.0 - 1.0
    length = torch.full((n,), 0.25, device="cuda")
    length[1::3] = 0.5
    best = [0, 40, 130, 200]  # 1, 2, 4, 8
    for i, t in enumerate(best):
        length[t] = 2.0 ** i
    q = (size * sign).expand(n, h, d).to(DT[dtype][0]).contiguous()
    k = (length[:, None, None] * sign).expand(n, hkv, d).to(DT[dtype][0]).contiguous()
    v = torch.randn(n, hkv, d, generator=g, device="cuda").to(DT[dtype][0])
    out = torch.empty_like(q)
    run_prefill(q, k, v, out, [n], [n], dtype)
    of = torch.tensor([max(t for t in best if t <= i) for i in range(n)], device="cuda")
    ref = v[of].double().repeat_interleave(h // hkv, 1)
    tol = (DT[dtype][2] + 2.0 ** -20 + (2.0 ** -8 if dtype == "bf16" else 0.0)) * ref.abs()
    assert bool(((out.double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("low", [-1e9, -1e15, -1e30])
def test_prefill_first_scores_far_below_the_others(low, d, dtype):
    """A first step of scores of enormous size and ordinary ones behind it: these alone have weight."""
    h, hkv, n, first = 4, 2, 400, 130
    q, k, v = ops.prefill_inputs(h, hkv, d, n, n, dtype, 274)
    q = q.abs() + 0.5
    k[:first] = low
    out = torch.empty_like(q)
    run_prefill(q, k, v, out, [n], [n], dtype)
    ops.check_prefill(q[first:], k[first:], v[first:], out[first:], [n - first], [n - first], dtype)


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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6, 1e7])
@pytest.mark.parametrize("n,d", [(70, 64), (900, 128), (9000, 64)])
def test_paged_scores_of_large_size(n, d, size, dtype):
    """Keys along one direction, V's scales of all sizes: the longest key has all the weight, and its value is the result,
    rounded once (besides 2^-20, and fp16's 2^-11 for bf16, of the weight)."""
    h, hkv, ps = 4, 2, 16
    g = gen(271)
    lens = [n] * 4
    pool = Pool(lens, hkv, d, ps, 272).fill(lens, 273)
    sign = torch.randint(0, 2, (d,), generator=g, device="cuda") * 2.0 - 1.0
    best = [0, 20, n // 2, n - 1]
    for b, t in enumerate(best):
        length = torch.full((len(pool.table[b]) * ps,), 0.25, device="cuda")
        length[1::3] = 0.5
        length[t] = 1.0
        codes = (length[:, None] * sign).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, 1, ps, d)
        pool.k[pool.table[b].long()] = codes.expand(-1, hkv, -1, -1)
    pool.ks[pool.table.long()] = 1.0
    q = (size * sign).expand(4, h, d).to(DT[dtype][0]).contiguous()
    out = torch.empty_like(q)
    run_paged(pool, q, out, lens, dtype)
    for b, t in enumerate(best):
        _, v = pool.rows(b, n)
        ref = v[:, t].repeat_interleave(h // hkv, 0)
        tol = (DT[dtype][2] + 2.0 ** -20 + (2.0 ** -11 if dtype == "bf16" else 0.0)) * ref.abs()
        assert bool(((out[b].double() - ref).abs() <= tol).all()), b


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


def test_paged_workspace_after_a_wait_that_ran_out():
    """With a limit of a microsecond the join of a long sequence gives up on blocks that end later: flagged, and the next
    call on the same workspace, on other values, waits for its own blocks' parts.  With the usual limit nothing is flagged."""
    h, hkv, d, ps, lens = 8, 2, 128, 64, [150_000, 70_000]
    pool = Pool([ps] * 8, hkv, d, ps, 250).fill([ps] * 8, 251)
    ids = pool.table[:, 0].clone()
    pool.width = -(-max(lens) // ps)
    pool.table = ids[torch.randint(0, 8, (2, pool.width), generator=gen(252), device="cuda")].to(torch.int32)
    q = torch.randn(2, 2, h, d, generator=gen(253), device="cuda")
    space = torch.empty(pool.cache().workspace_bytes(2, h), dtype=torch.uint8, device="cuda")
    want, out, status = torch.empty_like(q), torch.empty_like(q[0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    for i in range(2):
        run_paged(pool, q[i], want[i], lens, "f32")
    table, at = pool.table, ints(lens)
    short = pkg.PagedCache(pool.k.data_ptr(), pool.v.data_ptr(), pool.ks.data_ptr(), pool.vs.data_ptr(), n_pages=pool.n_pages,
                           page_size=ps, n_kv_heads=hkv, head_dim=d, wait_timeout_us=1)
    late = 0
    for _ in range(20):
        status.zero_()
        short.attention(q[0].data_ptr(), out.data_ptr(), at.data_ptr(), table.data_ptr(), table_stride=pool.width, n_seqs=2,
                        n_heads=h, dtype=D_.DEC_F32, workspace=space.data_ptr(), workspace_bytes=space.numel(),
                        status=status.data_ptr(), stream=ops.stream())
        late += int(status) == D_.DEC_SEQ_TIMEOUT
        status.zero_()
        run_paged(pool, q[1], out, lens, "f32", status=status, space=space)
        assert int(status) == 0 and torch.equal(out, want[1])
    assert late > 0


# ------------------------------------------------------------------------------------------------ append
def _border_keys(rows, hkv, d, pos, fr, pairs, factor, dtype, seed):
    """Keys whose rotation is as near as the type allows to the middles between E4M3 codes (scale 1: one value of 400 a
    head), the two of a pair in one binade."""
    g = gen(seed)
    r = d // 2
    shape = (rows, hkv, r)
    e = torch.randint(-3, 7, shape, generator=g, device="cuda").double()
    x, y = (torch.ldexp((8.5 + torch.randint(0, 7, shape, generator=g, device="cuda").double()) / 8, e)
            * (torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1) for _ in range(2))
    i = torch.arange(r, device="cuda")
    i, j = (i, i + r) if pairs == "half" else (2 * i, 2 * i + 1)
    c, s = (f(pos.double()[:, None, None] * fr) / factor for f in (torch.cos, torch.sin))
    k = torch.empty(rows, hkv, d, dtype=torch.float64, device="cuda")
    k[..., i], k[..., j] = x * c + y * s, y * c - x * s
    k[0, :, int(i[-1])] = 400.0 / factor  # the slowest pair of the first row: the scale's value
    k[0, :, int(j[-1])] = 0.0
    return k.to(DT[dtype][0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs,factor,d,ps,hkv,n", [("half", 1.0, 128, 64, 8, 64), ("neighbour", 0.75, 64, 16, 2, 16),
                                                      ("half", 0.75, 128, 128, 4, 128), ("neighbour", 1.0, 128, 16, 24, 3)])
def test_append_keys_between_two_codes(pairs, factor, d, ps, hkv, n, dtype):
    """Every key of the call at a border, far more than a handful in a block: each code is the exact value's nearest, and
    two calls give the same bits."""
    fr = ops.freqs(d, 100.0)
    old = 5 * ps  # a page of its own
    pos = torch.arange(old, old + n, device="cuda")
    k = _border_keys(n, hkv, d, pos, fr, pairs, factor, dtype, 230)
    h = hkv
    x = torch.zeros(n, (h + 2 * hkv) * d, dtype=k.dtype, device="cuda")
    x[:, h * d:(h + hkv) * d] = k.view(n, -1)
    q_out = torch.empty(n, h, d, dtype=k.dtype, device="cuda")
    pools = [Pool([old + n], hkv, d, ps, 231) for _ in range(3)]
    for p in pools:
        run_append(p, x, q_out, h, [n], [old + n], fr, pairs, dtype, factor)
    turned = ops.rotate64(k.double(), pos, fr, pairs, factor).transpose(0, 1)
    page = int(pools[0].table[0, 5])
    assert bool((pools[0].ks[page] == 1.0).all())
    have = pools[0].k[page, :, :n].view(torch.float8_e4m3fn).double()
    want = ops.e4m3_64(turned)
    _, e = torch.frexp(turned)
    gap = torch.remainder(turned.abs() * torch.ldexp(torch.ones_like(turned), 4 - e), 1.0) - 0.5
    sure = gap.abs() > 2.0 ** -38  # past what the float64 forms agree to
    if dtype == "f32":  # what the pass is for: most are too near for fp32 to tell
        assert float(((gap.abs() < 2.0 ** -19) & sure).double().mean()) > 0.5
    wrong = (have != want) & sure
    assert int(wrong.sum()) == 0, (int(wrong.sum()), wrong.numel())
    for p in pools[1:]:
        assert torch.equal(p.k, pools[0].k) and torch.equal(p.ks.nan_to_num(-5.0), pools[0].ks.nan_to_num(-5.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairs,factor,d,ps,hkv,n", [("half", 1.0, 128, 64, 8, 64), ("neighbour", 0.75, 64, 16, 2, 16)])
def test_append_rotated_keys_between_two_codes(pairs, factor, d, ps, hkv, n, dtype):
    """The same keys with the rotated ones asked for, apart and in place: what the cache holds does not depend on it, and
    both are the rotated keys, rounded once (fp32: three units of the pair's size besides, where fp32 was near enough)."""
    fr = ops.freqs(d, 100.0)
    old, h = 5 * ps, hkv
    pos = torch.arange(old, old + n, device="cuda")
    k = _border_keys(n, hkv, d, pos, fr, pairs, factor, dtype, 232)
    x = torch.zeros(n, (h + 2 * hkv) * d, dtype=k.dtype, device="cuda")
    x[:, h * d:(h + hkv) * d] = k.view(n, -1)
    q_out, apart, inside = torch.empty(n, h, d, dtype=k.dtype, device="cuda"), torch.empty_like(k), x.clone()
    pools = [Pool([old + n], hkv, d, ps, 233) for _ in range(3)]
    run_append(pools[0], x, q_out, h, [n], [old + n], fr, pairs, dtype, factor)
    run_append(pools[1], x, q_out, h, [n], [old + n], fr, pairs, dtype, factor, k_out=apart)
    run_append(pools[2], inside, q_out, h, [n], [old + n], fr, pairs, dtype, factor, k_out=inside[:, h * d:])
    for p in pools[1:]:
        assert torch.equal(p.k, pools[0].k) and torch.equal(p.v, pools[0].v)
    assert torch.equal(inside[:, h * d:(h + hkv) * d].reshape_as(apart), apart)
    exact = ops.rotate64(k.double(), pos, fr, pairs, factor)
    size = torch.empty_like(exact)
    i = torch.arange(d // 2, device="cuda")
    i, j = (i, i + d // 2) if pairs == "half" else (2 * i, 2 * i + 1)
    size[..., i] = size[..., j] = torch.hypot(k[..., i].double(), k[..., j].double()) * factor
    assert bool(((apart.double() - exact).abs() <= DT[dtype][2] * exact.abs() + 3 * 2.0 ** -23 * size).all())


@pytest.mark.parametrize("dtype,d,ps", [("bf16", 128, 64), ("f32", 64, 16), ("bf16", 64, 128)])
def test_append_key_codes_are_the_nearest(dtype, d, ps):
    """Prompts from position 0 on (there the rotation is the identity, and bf16 keys are exact middles one time in 16),
    half of the frequencies 0 besides: the nearest code wherever the float64 value is further from a middle than fp32's
    rotation is off (2^-22 of the pair's size, four units), and at exact middles (where it is exact)."""
    h, hkv, n = 8, 8, 200
    fr = ops.freqs(d)
    fr[d // 4:] = 0.0
    pool = Pool([n], hkv, d, ps, 240)
    x = (torch.randn(n, (h + 2 * hkv) * d, generator=gen(241), device="cuda") * 1.28).to(DT[dtype][0])
    q_out = torch.empty(n, h, d, dtype=x.dtype, device="cuda")
    run_append(pool, x, q_out, h, [n], [n], fr, "half", dtype)
    k = x.double().view(n, h + 2 * hkv, d)[:, h:h + hkv]
    turned = ops.rotate64(k, torch.arange(n, device="cuda"), fr, "half", 1.0)
    size = torch.hypot(k[..., :d // 2], k[..., d // 2:]).repeat(1, 1, 2)
    for p in range(-(-n // ps)):
        lo, hi = p * ps, min(n, (p + 1) * ps)
        page = int(pool.table[0, p])
        s = pool.ks[page].double()[:, None, None]
        y, z = (t[lo:hi].transpose(0, 1) / s for t in (turned, size))
        have = pool.k[page, :, :hi - lo].view(torch.float8_e4m3fn).double()
        _, e = torch.frexp(y)
        step = torch.ldexp(torch.ones_like(y), (e - 1).clamp(min=-6) - 3)
        gap = (torch.remainder(y.abs() / step, 1.0) - 0.5).abs() * step
        sure = (gap > 2.0 ** -22 * z) | (y == k[lo:hi].transpose(0, 1) / s)
        assert float(sure.double().mean()) > 0.99
        assert torch.equal(torch.where(sure, have, 0.0), torch.where(sure, ops.e4m3_64(y), 0.0))


@pytest.mark.parametrize("h,hkv,d,ps,old,new", [(160, 160, 64, 16, 5, [90] * 24), (300, 150, 64, 128, 0, [500, 3, 260]),
                                                (129, 129, 128, 16, 30, [1] * 40)])
def test_append_more_kv_heads_than_a_block_takes(h, hkv, d, ps, old, new):
    old = [old] * len(new)
    pool = Pool([a + b for a, b in zip(old, new)], hkv, d, ps, 295).fill(old, 296)
    x = torch.randn(sum(new), (h + 2 * hkv) * d, generator=gen(297), device="cuda")
    q_out = torch.empty(sum(new), h, d, device="cuda")
    before = pool.state()
    run_append(pool, x, q_out, h, new, [a + b for a, b in zip(old, new)], ops.freqs(d), "half", "f32")
    ops.check_append(pool, before, x, q_out, h, old, new, ops.freqs(d), "half", "f32")


# ------------------------------------------------------------------------------------------------ streams and graphs
def test_prefill_on_several_streams_at_once():
    """Calls of both head sizes and types under way together: the bits of each alone."""
    sets = [("bf16", 64, [900, 30, 700]), ("bf16", 128, [1500, 400]), ("f32", 64, [300, 200]), ("bf16", 64, [64] * 40)]
    args, want, out = [], [], []
    for i, (dtype, d, lens) in enumerate(sets):
        args.append(ops.prefill_inputs(8, 4, d, sum(lens), sum(lens), dtype, 280 + i))
        want.append(torch.empty_like(args[i][0]))
        out.append(torch.empty_like(args[i][0]))
        run_prefill(*args[i], want[i], lens, lens, dtype)
    cu = [ints(offsets(s[2])) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(15):
        for i, (dtype, d, lens) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                run_prefill(*args[i], out[i], cu[i], cu[i], dtype, max_q=max(lens))
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d,ps", [(64, 16), (128, 64)])
def test_prompts_in_a_captured_graph(d, ps):
    """Append and prompt attention captured together and replayed on other values and other lengths: the bits of the same calls
    outside a graph."""
    h, hkv, total = 8, 2, 700
    lens = [[400, 1, 299], [17, 683, 0], [233, 233, 234]]
    fr = ops.freqs(d)
    x = (torch.randn(3, total, (h + 2 * hkv) * d, generator=gen(290), device="cuda") * 1.28).bfloat16()
    row, e = x.stride(1), 2

    def once(pool, xin, cu, at, q, k, out):
        p = xin.data_ptr()
        st = ops.stream()
        pool.cache().append(p, p + h * d * e, p + (h + hkv) * d * e, q.data_ptr(), cu.data_ptr(), at.data_ptr(),
                            pool.table.data_ptr(), table_stride=pool.width, n_seqs=3, n_tokens=total, max_new=total,
                            n_heads=h, strides=(row, row, row, h * d), inv_freq=fr.data_ptr(), rot_dim=d,
                            k_out=k.data_ptr(), stream=st)
        pkg.attention_prefill(q.data_ptr(), k.data_ptr(), p + (h + hkv) * d * e, out.data_ptr(), cu.data_ptr(),
                              cu.data_ptr(), n_seqs=3, n_q=total, n_k=total, max_q=total, n_heads=h, n_kv_heads=hkv,
                              head_dim=d, strides=(h * d, hkv * d, row, h * d), stream=st)

    def buffers():
        pool = Pool([total] * 3, hkv, d, ps, 291)
        q = torch.empty(total, h, d, dtype=torch.bfloat16, device="cuda")
        return pool, q, torch.empty(total, hkv, d, dtype=q.dtype, device="cuda"), torch.empty_like(q)

    pool, q, k, out = buffers()
    xin, cu, at = x[0].clone(), ints(offsets(lens[0])), ints(lens[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(pool, xin, cu, at, q, k, out)
    for i in range(3):
        xin.copy_(x[i])
        cu.copy_(ints(offsets(lens[i])))
        at.copy_(ints(lens[i]))
        before = pool.state()
        graph.replay()
        torch.cuda.synchronize()
        p2, q2, k2, out2 = buffers()
        p2.k, p2.v, p2.ks, p2.vs = before
        once(p2, x[i], ints(offsets(lens[i])), ints(lens[i]), q2, k2, out2)
        torch.cuda.synchronize()
        for a, b in ((q, q2), (k, k2), (out, out2), (pool.k, p2.k), (pool.v, p2.v), (pool.ks.nan_to_num(-5.0), p2.ks.nan_to_num(-5.0))):
            assert torch.equal(a, b), i
