"""dec_kv_append, dec_attention_paged and dec_attention_prefill against plain float64 forms.

Tolerances are bounds, written down from the arithmetic.  With u = 2^-24 (fp32), A = sum_t p_t |v_t| and
S = max_t sum_d |q_d k_d| * scale (both of the float64 form): a score is off by at most (D + 4) u S, so a weight by a
factor of 1 + 2 (D + 4) u S + 2^-20 (scaling by log2 e, the hardware's 2^x, the rescales), and a sum of n weighted values by n u
more; the result is rounded once, by 2^-8 of its value in bf16, u in fp32.  Weights that meet 8-bit values on the
tensor cores are rounded to fp16 (2^-11) for bf16 results and to an fp16 pair (2^-20) for fp32 ones; weights that meet
bf16 values are rounded to bf16 (2^-8).
"""
import math

import pytest
import torch

import persistent_sm_decode_02_b200 as pkg
from persistent_sm_decode_02_b200 import dec as D_

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": (torch.bfloat16, D_.DEC_BF16, 2.0 ** -8), "f32": (torch.float32, D_.DEC_F32, U)}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def stream():
    return torch.cuda.current_stream().cuda_stream


class Pool:
    """Pages, scales and a page table with every sequence's pages in random order; unused bytes are E4M3 NaN."""

    def __init__(self, lens, hkv, d, ps, seed, extra=2, width=None):
        g = gen(seed)
        need = [-(-n // ps) for n in lens]
        self.n_pages = sum(need) + extra
        self.ps, self.hkv, self.d, self.lens = ps, hkv, d, list(lens)
        order = torch.randperm(self.n_pages, generator=g, device="cuda").to(torch.int32)
        self.width = width or max(1, max(need, default=1))
        self.table = torch.full((max(1, len(lens)), self.width), -7, dtype=torch.int32, device="cuda")
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        shape = (self.n_pages, hkv, ps, d)
        self.k = torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda")
        self.v = self.k.clone()
        self.ks = torch.full(shape[:2], math.nan, device="cuda")
        self.vs = self.ks.clone()

    def fill(self, lens, seed, std=1.28):
        """Codes of normal values in every position below lens, the scales powers of two around 2^-6."""
        g = gen(seed)
        for b, n in enumerate(lens):
            for p in range(-(-n // self.ps)):
                page, rows = int(self.table[b, p]), min(self.ps, n - p * self.ps)
                for codes, scales in ((self.k, self.ks), (self.v, self.vs)):
                    e = torch.randint(-8, -5, (self.hkv,), generator=g, device="cuda")
                    s = torch.ldexp(torch.ones(self.hkv, device="cuda"), e)
                    x = torch.randn(self.hkv, rows, self.d, generator=g, device="cuda") * std / s[:, None, None]
                    codes[page, :, :rows] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    scales[page] = s
        return self

    def cache(self):
        return pkg.PagedCache(self.k.data_ptr(), self.v.data_ptr(), self.ks.data_ptr(), self.vs.data_ptr(),
                              n_pages=self.n_pages, page_size=self.ps, n_kv_heads=self.hkv, head_dim=self.d)

    def rows(self, b, n):
        """float64 K and V [hkv, n, d] of sequence b."""
        if n == 0:
            return torch.zeros(2, self.hkv, 0, self.d, dtype=torch.float64, device="cuda").unbind(0)
        ids = self.table[b, :-(-n // self.ps)].long()
        return tuple((c[ids].view(torch.float8_e4m3fn).double() * s[ids].double()[:, :, None, None])
                     .transpose(0, 1).reshape(self.hkv, -1, self.d)[:, :n] for c, s in ((self.k, self.ks), (self.v, self.vs)))

    def state(self):
        return [t.clone() for t in (self.k, self.v, self.ks, self.vs)]


def attend64(q, k, v, scale, seen=None):
    """q [h, m, d], k, v [hkv, n, d] float64 -> out, A, S (see above); rows that see nothing give 0."""
    gs = q.shape[0] // k.shape[0]
    k, v = k.repeat_interleave(gs, 0), v.repeat_interleave(gs, 0)
    if k.shape[1] == 0:
        z = torch.zeros_like(q)
        return z, z, 0.0
    sc = q @ k.transpose(1, 2) * scale
    big = (q.abs() @ k.abs().transpose(1, 2) * scale)
    if seen is not None:
        sc = sc.masked_fill(~seen, -math.inf)
        big = big.masked_fill(~seen, 0.0)
    p = torch.softmax(sc, -1).nan_to_num(0.0)
    return p @ v, p @ v.abs(), float(big.max())


def attend_tol(ref, a, s, n, d, dtype, weight):
    return DT[dtype][2] * ref.abs() + a * (weight + 2 * (d + 4) * U * s + 2.0 ** -20 + n * U) + 1e-30


# ------------------------------------------------------------------------------------------------ append
def e4m3_64(x):
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def scale64(x):
    """Scale [hkv] of new values x [rows, hkv, d]."""
    a = torch.where(torch.isfinite(x), x.abs(), 0.0).amax((0, 2)).clamp(min=2.0 ** -140)
    e = torch.ceil(torch.log2(a / 448.0)).clamp(-120, 120)
    return ((e.long() + 1023) << 52).view(torch.float64)  # 2^e exactly (the device's pow may be an ulp off)


def rotate64(x, pos, inv_freq, pairs, factor):
    r = 2 * inv_freq.numel()
    ang = pos.double()[:, None, None] * inv_freq
    c, s = torch.cos(ang) * factor, torch.sin(ang) * factor
    i = torch.arange(r // 2, device="cuda")
    i, j = (i, i + r // 2) if pairs == "half" else (2 * i, 2 * i + 1)
    y = x.clone()
    y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., i] * s + x[..., j] * c
    return y


def run_append(pool, qkv, q_out, h, new, lens, inv_freq, pairs, dtype, factor=1.0, status=None, max_new=None, with_q=True,
               n_tokens=None, k_out=None):
    hkv, d = pool.hkv, pool.d
    x, e, row = qkv.data_ptr(), qkv.element_size(), qkv.stride(0)
    cu = new if isinstance(new, torch.Tensor) else ints(offsets(new))
    n_seqs = cu.numel() - 1
    pool.cache().append(x if with_q else None, x + h * d * e, x + (h + hkv) * d * e, q_out.data_ptr() if with_q else None,
                        cu.data_ptr(), ints(lens).data_ptr(), pool.table.data_ptr(), table_stride=pool.width,
                        n_seqs=n_seqs, n_tokens=qkv.shape[0] if n_tokens is None else n_tokens,
                        max_new=max(new) if max_new is None else max_new, n_heads=h,
                        dtype=DT[dtype][1], strides=(row, row, row, q_out.stride(0)), inv_freq=inv_freq.data_ptr(),
                        rot_dim=2 * inv_freq.numel(), neighbour_pairs=pairs == "neighbour", factor=factor,
                        k_out=None if k_out is None else k_out.data_ptr(),
                        k_out_stride=None if k_out is None else k_out.stride(0), status=None if status is None else status.data_ptr(), stream=stream())
    torch.cuda.synchronize()


def freqs(r, theta=10000.0):
    return theta ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / max(1, r))


def check_append(pool, before, qkv, q_out, h, old, new, inv_freq, pairs, dtype, factor=1.0):
    hkv, d, ps = pool.hkv, pool.d, pool.ps
    k, v, ks, vs = [t.clone() for t in before]
    at = 0
    for b, (o, n) in enumerate(zip(old, new)):
        if n == 0:
            continue
        x = qkv[at:at + n].double().view(n, h + 2 * hkv, d)
        pos = torch.arange(o, o + n, device="cuda")
        turned = rotate64(x[:, :h + hkv], pos, inv_freq, pairs, factor)
        size = x.abs().amax() * max(1.0, factor)  # |a| + |b| <= 2 size; cos and sin within 2^-21, products and sums by u each
        got = q_out[at:at + n].double()
        assert bool(((got - turned[:, :h]).abs() <= DT[dtype][2] * turned[:, :h].abs() + 2.0 ** -19 * size).all())
        at += n
        for p in range(o // ps, -(-(o + n) // ps)):
            lo, hi = max(o, p * ps), min(o + n, (p + 1) * ps)
            page = int(pool.table[b, p])
            for codes, scales, got_c, got_s, y, slack in ((k, ks, pool.k, pool.ks, turned[:, h:], 2.0 ** -19 * size),
                                                          (v, vs, pool.v, pool.vs, x[:, h + hkv:], 0.0)):
                y = y[lo - o:hi - o]
                now = scale64(y)
                if lo > p * ps:
                    now = torch.maximum(now, scales[page].double())
                    f = (scales[page].double() / now)[:, None, None]
                    part = codes[page, :, :lo - p * ps].view(torch.float8_e4m3fn).double()
                    want = torch.where(torch.isfinite(part), e4m3_64(part * f), part)
                    have = got_c[page, :, :lo - p * ps].view(torch.float8_e4m3fn).double()
                    assert torch.equal(have.nan_to_num(999.0), want.nan_to_num(999.0))
                assert torch.equal(got_s[page].double(), now)
                have = got_c[page, :, lo - p * ps:hi - p * ps].view(torch.float8_e4m3fn).double() * now[:, None, None]
                y = y.transpose(0, 1)
                lim = 448.0 * now[:, None, None]
                want = torch.maximum(torch.minimum(y, lim), -lim)
                assert torch.equal(torch.isnan(have), torch.isnan(y))
                # half a step: 2^-4 of the value, 2^-10 of the scale where the code is subnormal
                ok = (have - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 * now[:, None, None] + slack
                assert bool((ok | torch.isnan(y)).all())
                # and the nearest code itself wherever rounding cannot hinge on the last bits of the rotation
                if slack == 0.0:
                    exact = e4m3_64(y / now[:, None, None])
                    assert torch.equal(torch.where(torch.isnan(y), 0.0, exact),
                                       torch.where(torch.isnan(y), 0.0, have / now[:, None, None]))
                codes[page, :, :hi - p * ps] = got_c[page, :, :hi - p * ps]
                scales[page] = got_s[page]
    # nothing else moved
    for got, want in zip((pool.k, pool.v), (k, v)):
        assert torch.equal(got, want)
    for got, want in zip((pool.ks, pool.vs), (ks, vs)):
        assert torch.equal(got.nan_to_num(-5.0), want.nan_to_num(-5.0))


APPENDS = [
    # dtype, h, hkv, d, page, rot, pairs, old, new
    ("bf16", 32, 8, 128, 64, 128, "half", [0], [1]),
    ("bf16", 32, 8, 128, 64, 128, "half", [63, 64, 65, 0, 700], [1, 1, 1, 1, 1]),
    ("bf16", 6, 2, 64, 16, 64, "neighbour", [0, 5, 16, 31], [77, 0, 33, 1]),
    ("f32", 4, 4, 64, 32, 32, "half", [3, 0, 90], [40, 31, 129]),
    ("bf16", 16, 2, 128, 128, 64, "neighbour", [1, 127, 128], [300, 2, 128]),
    ("f32", 4, 2, 128, 128, 128, "half", [0, 100], [129, 257]),
    ("bf16", 8, 1, 64, 32, 0, "half", [10, 0], [50, 3]),
    ("f32", 7, 7, 128, 16, 16, "neighbour", [15, 2], [1, 2]),
]


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: "%s_h%d_%d_d%d_p%d_r%d_%s" % c[:7])
@pytest.mark.parametrize("factor", [1.0, 0.75])
def test_append(case, factor):
    dtype, h, hkv, d, ps, rot, pairs, old, new = case
    pool = Pool([a + b for a, b in zip(old, new)], hkv, d, ps, 1).fill(old, 2)
    qkv = (torch.randn(sum(new) + 3, (h + 2 * hkv) * d, generator=gen(3), device="cuda") * 1.28).to(DT[dtype][0])
    q_out = torch.full((sum(new) + 3, h, d), 7.0, dtype=DT[dtype][0], device="cuda")
    before = pool.state()
    k_out = torch.full((sum(new) + 3, hkv, d), 7.0, dtype=qkv.dtype, device="cuda")
    run_append(pool, qkv, q_out, h, new, [a + b for a, b in zip(old, new)], freqs(rot), pairs, dtype, factor, k_out=k_out)
    check_append(pool, before, qkv, q_out, h, old, new, freqs(rot), pairs, dtype, factor)
    # the rotated keys, rounded as the queries are
    pos = torch.cat([torch.arange(a, a + n, device="cuda") for a, n in zip(old, new)])
    k = rotate64(qkv[:sum(new)].double().view(-1, h + 2 * hkv, d)[:, h:h + hkv], pos, freqs(rot), pairs, factor)
    err = (k_out[:sum(new)].double() - k).abs()
    assert bool((err <= DT[dtype][2] * k.abs() + 2.0 ** -19 * qkv.double().abs().amax() * max(1.0, factor)).all())
    assert bool((k_out[sum(new):] == 7.0).all())
    assert bool((q_out[sum(new):] == 7.0).all())  # rows behind the last sequence


def test_append_token_by_token_grows_the_scale():
    """A page filled one token at a time, each louder than the last: the scale grows and earlier rows are rounded again."""
    h, hkv, d, ps, n = 4, 2, 64, 16, 20
    pool = Pool([n], hkv, d, ps, 4)
    x = torch.randn(n, (h + 2 * hkv) * d, generator=gen(5), device="cuda") * (
        2.0 ** torch.arange(-4, n - 4, device="cuda", dtype=torch.float32) / 4)[:, None]
    q_out = torch.empty(1, h, d, device="cuda")
    for t in range(n):
        before = pool.state()
        run_append(pool, x[t:t + 1], q_out, h, [1], [t + 1], freqs(d), "half", "f32")
        check_append(pool, before, x[t:t + 1], q_out, h, [t], [1], freqs(d), "half", "f32")


def test_append_extreme_values():
    """Zeros, infinities, NaN, the largest and smallest finite values of the type."""
    h, hkv, d, ps = 2, 2, 64, 16
    new = [16, 16, 16, 16, 5]
    pool = Pool(new, hkv, d, ps, 6)
    x = torch.randn(sum(new), (h + 2 * hkv) * d, generator=gen(7), device="cuda").to(torch.bfloat16)
    x[:16] = 0
    x[16:32] *= 1e-38
    x[32:48, ::3] = torch.finfo(torch.bfloat16).max
    x[48:64, 1::5] = math.inf
    x[64:, 2::7] = math.nan
    x[64:, 3::11] = -math.inf
    q_out = torch.empty(sum(new), h, d, dtype=torch.bfloat16, device="cuda")
    before = pool.state()
    run_append(pool, x, q_out, h, new, new, freqs(0), "half", "bf16")
    check_append_codes_only(pool, before, x, h, new)
    assert torch.equal(q_out.nan_to_num(5.0), x.view(-1, h + 2 * hkv, d)[:, :h].nan_to_num(5.0))


def check_append_codes_only(pool, before, x, h, new):
    hkv, d, ps = pool.hkv, pool.d, pool.ps
    at = 0
    for b, n in enumerate(new):
        y = x[at:at + n].double().view(n, h + 2 * hkv, d)[:, h:]
        at += n
        page = int(pool.table[b, 0])
        for c, (codes, scales) in enumerate(((pool.k, pool.ks), (pool.v, pool.vs))):
            z = y[:, c * hkv:(c + 1) * hkv]
            s = scale64(z)
            assert torch.equal(scales[page].double(), s)
            have = codes[page, :, :n].view(torch.float8_e4m3fn).double()
            z = z.transpose(0, 1) / s[:, None, None]
            want = torch.where(torch.isnan(z), 999.0, e4m3_64(z.clamp(-448, 448)))
            assert torch.equal(have.nan_to_num(999.0), want.nan_to_num(999.0))


def test_append_many_sequences():
    """400 sequences with 0 to 3 new tokens behind lengths around page ends."""
    h, hkv, d, ps = 4, 2, 64, 16
    old, new = [(5 * i) % 35 for i in range(400)], [i % 4 for i in range(400)]
    lens = [a + b for a, b in zip(old, new)]
    pool = Pool(lens, hkv, d, ps, 80).fill(old, 81)
    x = torch.randn(sum(new), (h + 2 * hkv) * d, generator=gen(82), device="cuda")
    q_out = torch.empty(sum(new), h, d, device="cuda")
    before = pool.state()
    run_append(pool, x, q_out, h, new, lens, freqs(d), "half", "f32")
    check_append(pool, before, x, q_out, h, old, new, freqs(d), "half", "f32")


def test_append_whole_prompts_in_full_pages():
    """Pages that fill a block (queries and keys are launches of their own there), a prompt that starts inside a page."""
    for dtype, d, ps in (("bf16", 128, 64), ("f32", 128, 128), ("bf16", 64, 128)):
        h, hkv, old, new = 16, 8, [0, 37, 64], [700, 260, 1]
        lens = [a + b for a, b in zip(old, new)]
        pool = Pool(lens, hkv, d, ps, 83).fill(old, 84)
        x = (torch.randn(sum(new), (h + 2 * hkv) * d, generator=gen(85), device="cuda") * 1.28).to(DT[dtype][0])
        q_out = torch.empty(sum(new), h, d, dtype=x.dtype, device="cuda")
        before = pool.state()
        run_append(pool, x, q_out, h, new, lens, freqs(d), "half", dtype)
        check_append(pool, before, x, q_out, h, old, new, freqs(d), "half", dtype)


def test_append_in_place_and_without_q():
    h, hkv, d, ps, n = 6, 2, 64, 32, 45
    x = (torch.randn(n, (h + 2 * hkv) * d, generator=gen(8), device="cuda")).to(torch.bfloat16)
    pools = [Pool([n], hkv, d, ps, 9) for _ in range(5)]
    out = torch.empty(n, h * d, dtype=torch.bfloat16, device="cuda")
    run_append(pools[0], x, out, h, [n], [n], freqs(d), "half", "bf16")
    y = x.clone()
    z = x.clone()
    run_append(pools[1], y, y, h, [n], [n], freqs(d), "half", "bf16")  # q_out is q, inside the fused buffer
    k_apart = torch.empty(n, hkv * d, dtype=torch.bfloat16, device="cuda")
    run_append(pools[3], z, z, h, [n], [n], freqs(d), "half", "bf16", k_out=z[:, h * d:])  # k_out is k, too
    run_append(pools[4], x, out, h, [n], [n], freqs(d), "half", "bf16", k_out=k_apart)
    assert torch.equal(z[:, :h * d], out) and torch.equal(z[:, h * d:(h + hkv) * d], k_apart)
    run_append(pools[2], x, out, h, [n], [n], freqs(d), "half", "bf16", with_q=False)
    assert torch.equal(y[:, :h * d], out) and torch.equal(y[:, h * d:], x[:, h * d:])
    for p in pools[1:]:
        for a, b in zip(p.state(), pools[0].state()):
            assert torch.equal(a.nan_to_num(-5.0) if a.is_floating_point() else a,
                               b.nan_to_num(-5.0) if b.is_floating_point() else b)


def test_append_far_position():
    """Position 2,000,003: the angle is reduced in fp64."""
    h, hkv, d, ps, o = 2, 1, 128, 128, 2_000_003
    pool = Pool([1], hkv, d, ps, 10, extra=4, width=o // ps + 1)
    pool.table[0] = -1
    pool.table[0, o // ps] = 2
    x = torch.randn(1, (h + 2 * hkv) * d, generator=gen(11), device="cuda")
    q_out = torch.empty(1, h, d, device="cuda")
    before = pool.state()
    run_append(pool, x, q_out, h, [1], [o + 1], freqs(d), "half", "f32")
    # the page's earlier rows are NaN codes and its scale NaN: the new scale takes over
    want = rotate64(x.double().view(1, h + 2 * hkv, d)[:, :h + hkv], torch.tensor([o], device="cuda"), freqs(d), "half", 1.0)
    size = x.double().abs().amax()
    assert bool(((q_out.double() - want[:, :h]).abs() <= U * want[:, :h].abs() + 2.0 ** -19 * size).all())
    s = scale64(want[:, h:])
    assert torch.equal(pool.ks[2].double(), s)
    have = pool.k[2, :, o % ps].view(torch.float8_e4m3fn).double() * s[:, None]
    assert bool(((have - want[0, h:]).abs() <= 2.0 ** -4 * want[0, h:].abs() + 2.0 ** -10 * s[:, None] + 2.0 ** -19 * size).all())
    others = [0, 1, 3, 4][:pool.n_pages - 1]
    assert torch.equal(pool.k[others], before[0][others])


@pytest.mark.parametrize("what", ["page", "decreasing", "past_rows", "short_len", "past_table", "above_max"])
def test_append_inconsistent_sequences_are_skipped(what):
    """Sequence 1 of three is inconsistent: flagged and left out; the others are as if alone."""
    h, hkv, d, ps = 4, 2, 64, 16
    old, new = [4, 10, 20], [20, 9, 7]
    lens = [a + b for a, b in zip(old, new)]
    cu, max_new, bits = offsets(new), 20, D_.DEC_SEQ_BAD_RANGE
    pool = Pool(lens, hkv, d, ps, 12).fill(old, 13)
    x = torch.randn(sum(new), (h + 2 * hkv) * d, generator=gen(14), device="cuda")
    q_out = torch.full((sum(new), h, d), 7.0, device="cuda")
    table = pool.table.clone()
    keep = [0, 2]
    if what == "page":
        pool.table[1, 0] = pool.n_pages
        bits = D_.DEC_SEQ_BAD_PAGE
    elif what == "decreasing":
        cu[1], cu[2] = cu[2], cu[1]  # sequence 1 has -9 rows; 0 has 29, 2 has 16: both above max_new 15
        max_new, keep = 15, []
    elif what == "past_rows":
        cu = [0, 20, 29, 2 ** 31 - 1]
        keep = [0, 1]
    elif what == "short_len":
        lens[1] = 8
    elif what == "past_table":
        lens[1] = pool.width * ps + 1
    elif what == "above_max":
        max_new, keep = 9, [1, 2]
    before = pool.state()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k_out = torch.full((sum(new), hkv, d), 7.0, device="cuda")
    run_append(pool, x, q_out, h, ints(cu), lens, freqs(d), "half", "f32", status=status, max_new=max_new, k_out=k_out)
    assert int(status) == bits
    pool.table = table
    if what == "page":  # slots 0..15 of sequence 1 are left out, 16..18 and every rotated query and key are there
        assert not bool((k_out == 7.0).all(-1).any())
        assert not bool((q_out == 7.0).all(-1).any())
        first = int(table[1, 0])
        assert torch.equal(pool.k[first], before[0][first])
        return
    new_kept = [n if i in keep else 0 for i, n in enumerate(new)]
    rows = torch.cat([x[offsets(new)[i]:offsets(new)[i + 1]] for i in keep]) if keep else x[:0]
    outs = torch.cat([q_out[offsets(new)[i]:offsets(new)[i + 1]] for i in keep]) if keep else q_out[:0]
    check_append(pool, before, rows, outs, h, old, new_kept, freqs(d), "half", "f32")


# ------------------------------------------------------------------------------------------------ paged attention
def run_paged(pool, q, out, lens, dtype, table=None, scale=None, status=None, space=None):
    c = pool.cache()
    h, n = q.shape[1], q.shape[0]
    table = pool.table if table is None else table
    lens = lens if isinstance(lens, torch.Tensor) else ints(lens)
    if space is None:
        space = torch.full((c.workspace_bytes(n, h),), 0xFF, dtype=torch.uint8, device="cuda")
    c.attention(q.data_ptr(), out.data_ptr(), lens.data_ptr(), table.data_ptr(), table_stride=pool.width, n_seqs=n,
                n_heads=h, dtype=DT[dtype][1], q_stride=q.stride(0), out_stride=out.stride(0), scale=scale,
                workspace=space.data_ptr(), workspace_bytes=space.numel(),
                status=None if status is None else status.data_ptr(), stream=stream())


def check_paged(pool, q, out, lens, dtype, scale=None):
    scale = pool.d ** -0.5 if scale is None else scale
    for b, n in enumerate(lens):
        k, v = pool.rows(b, n)
        ref, a, s = attend64(q[b].double()[:, None], k, v, scale)
        tol = attend_tol(ref, a, s, n, pool.d, dtype, 2.0 ** -11 if dtype == "bf16" else 2.0 ** -20)
        err = (out[b].double()[:, None] - ref).abs()
        assert bool((err <= tol).all()), (b, n, float((err / tol).max()))


PAGED = [
    # h, hkv, d, page, lens
    (6, 2, 64, 16, [1]),
    (6, 2, 64, 16, [77]),
    (32, 8, 128, 64, [0, 1, 63, 64, 65, 128, 1000, 0]),
    (16, 2, 128, 32, [5000, 3, 31, 33, 0, 2048]),
    (8, 1, 64, 128, [127, 128, 129, 4097]),
    (4, 4, 64, 64, [300]),
    (4, 2, 128, 16, [15, 16, 17, 500]),
    (7, 1, 128, 64, [130, 7]),
    (32, 8, 128, 64, [8193]),
    (3, 3, 64, 32, list(range(70))),
    (2, 2, 128, 128, [20000]),
    (1, 1, 64, 16, [0]),
    (4, 1, 64, 16, [17] * 32),                                    # as many sequences as one warp counts
    (4, 1, 64, 16, [17] * 16 + [0] + [300] + [16] * 15),          # one more
    (2, 1, 128, 16, [(7 * i) % 41 for i in range(1000)]),         # several for a thread, empty ones among them
    (1, 1, 64, 32, [3] * 2500),                                   # more than there are warps
    (8, 8, 128, 16, [1, 2000, 1, 1, 700, 0, 33]),                 # one query head a kv head; long between short
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", PAGED, ids=lambda c: "h%d_%d_d%d_p%d_n%d_max%d" % (*c[:4], len(c[4]), max(c[4])))
def test_paged(case, dtype):
    """The rows of every page behind the length hold NaN codes, unused table entries are negative."""
    h, hkv, d, ps, lens = case
    pool = Pool(lens, hkv, d, ps, 20).fill(lens, 21)
    wide = torch.randn(len(lens), h * d + 64, generator=gen(22), device="cuda").to(DT[dtype][0]) * 1.28
    q = wide[:, 32:32 + h * d].unflatten(1, (h, d))  # rows are not contiguous
    out = torch.full((len(lens) + 1, h, d), 7.0, dtype=DT[dtype][0], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_paged(pool, q, out[:-1], lens, dtype, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    check_paged(pool, q, out, lens, dtype)
    assert bool((out[-1] == 7.0).all())
    again = torch.empty_like(out[:-1])
    run_paged(pool, q, again, lens, dtype)
    assert torch.equal(again, out[:-1])  # the same bits every time


def test_paged_everything_empty():
    pool = Pool([0, 0, 0], 2, 64, 16, 18)
    q = torch.randn(3, 4, 64, generator=gen(19), device="cuda")
    out = torch.full_like(q, 7.0)
    run_paged(pool, q, out, [0, 0, 0], "f32")
    assert bool((out == 0).all())


def test_paged_scales_far_apart():
    """V's scales of one head span 2^40 between pages (a page of zeros has the smallest there is): the small ones' share
    of the result is kept where the large ones' weights vanish."""
    h, hkv, d, ps, lens = 4, 2, 64, 16, [96]
    pool = Pool(lens, hkv, d, ps, 16).fill(lens, 17)
    for p, e in enumerate((-120, -30, -6, 10, -20, -7)):
        page = int(pool.table[0, p])
        pool.vs[page] = 2.0 ** e
        if e == -120:
            pool.v[page] = 0
    q = torch.randn(1, h, d, generator=gen(15), device="cuda")
    k, _ = pool.rows(0, 96)
    for g in range(hkv):  # queries that avoid the page with the large values: scores around -64 there
        q[0, 2 * g:2 * g + 2] = -200.0 * k[g, 48:64].mean(0).float() / k[g, 48:64].mean(0).norm().float()
    for dtype in ("f32", "bf16"):
        x = q.to(DT[dtype][0])
        out = torch.empty_like(x)
        run_paged(pool, x, out, lens, dtype)
        check_paged(pool, x, out, lens, dtype)


def test_paged_two_streams_at_once():
    """Calls under way together, each with a workspace of its own."""
    h, hkv, d, ps = 8, 2, 128, 32
    sets = [[4000, 10, 900], [50] * 40, [20000]]
    pools = [Pool(lens, hkv, d, ps, 90 + i).fill(lens, 93 + i) for i, lens in enumerate(sets)]
    q = [torch.randn(len(l), h, d, generator=gen(96), device="cuda") for l in sets]
    out = [torch.empty_like(x) for x in q]
    space = [torch.full((p.cache().workspace_bytes(len(l), h),), 0x5A, dtype=torch.uint8, device="cuda")
             for p, l in zip(pools, sets)]
    lens = [ints(l) for l in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                run_paged(pools[i], q[i], out[i], lens[i], "f32", space=space[i])
    torch.cuda.synchronize()
    for i, l in enumerate(sets):
        check_paged(pools[i], q[i], out[i], l, "f32")


def test_paged_scales_and_large_scores():
    """Scores in the hundreds (one key takes nearly all), tiny ones, and a softmax scale of the caller's."""
    h, hkv, d, ps, lens = 8, 2, 128, 32, [200, 1500]
    for std, scale in ((30.0, None), (1e-3, None), (1.0, 0.02)):
        pool = Pool(lens, hkv, d, ps, 23).fill(lens, 24, std=min(std, 3.0))
        q = torch.randn(2, h, d, generator=gen(25), device="cuda") * std
        out = torch.empty_like(q)
        run_paged(pool, q, out, lens, "f32", scale=scale)
        check_paged(pool, q, out, lens, "f32", scale)
        qb, ob = q.bfloat16(), out.bfloat16()
        run_paged(pool, qb, ob, lens, "bf16", scale=scale)
        check_paged(pool, qb, ob, lens, "bf16", scale)


def test_paged_shared_prefix():
    """Two sequences whose tables share their first pages."""
    h, hkv, d, ps, lens = 8, 2, 64, 16, [100, 90]
    pool = Pool(lens, hkv, d, ps, 26).fill(lens, 27)
    pool.table[1, :4] = pool.table[0, :4]
    q = torch.randn(2, h, d, generator=gen(28), device="cuda")
    out = torch.empty_like(q)
    run_paged(pool, q, out, lens, "f32")
    check_paged(pool, q, out, lens, "f32")


def test_paged_nan_stays_in_its_sequence_and_head():
    h, hkv, d, ps, lens = 8, 2, 64, 16, [100, 90, 33]
    pool = Pool(lens, hkv, d, ps, 29).fill(lens, 30)
    pool.v[int(pool.table[1, 2]), 1, 3, 5] = 0x7F
    q = torch.randn(3, h, d, generator=gen(31), device="cuda")
    out = torch.empty_like(q)
    run_paged(pool, q, out, lens, "f32")
    bad = torch.isnan(out)
    assert bool(bad[1, 4:, 5].all()) and int(bad.sum()) == 4
    q[2] = math.nan
    run_paged(pool, q, out, lens, "f32")
    assert bool(torch.isnan(out[2]).all()) and not bool(torch.isnan(out[0]).any())


@pytest.mark.parametrize("what", ["page_low", "page_high", "negative", "past_table"])
def test_paged_inconsistent_sequences(what):
    h, hkv, d, ps, lens = 8, 2, 64, 16, [100, 90, 33]
    pool = Pool(lens, hkv, d, ps, 32).fill(lens, 33)
    q = torch.randn(3, h, d, generator=gen(34), device="cuda")
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    table, given, bits = pool.table.clone(), list(lens), D_.DEC_SEQ_BAD_RANGE
    if what.startswith("page"):
        table[1, 2] = -1 if what == "page_low" else pool.n_pages
        bits = D_.DEC_SEQ_BAD_PAGE
    else:
        given[1] = -5 if what == "negative" else pool.width * ps + 1
    run_paged(pool, q, out, given, "f32", table=table, status=status)
    torch.cuda.synchronize()
    assert int(status) == bits
    for b in (0, 2):
        k, v = pool.rows(b, lens[b])
        ref, a, s = attend64(q[b].double()[:, None], k, v, d ** -0.5)
        assert bool(((out[b].double()[:, None] - ref).abs() <= attend_tol(ref, a, s, lens[b], d, "f32", 2.0 ** -20)).all())
    if what.startswith("page"):  # its sixteen positions are left out
        k, v = pool.rows(1, 90)
        keep = [t for t in range(90) if t // ps != 2]
        ref, a, s = attend64(q[1].double()[:, None], k[:, keep], v[:, keep], d ** -0.5)
        assert bool(((out[1].double()[:, None] - ref).abs() <= attend_tol(ref, a, s, 74, d, "f32", 2.0 ** -20)).all())
    else:
        assert bool((out[1] == 0).all())


def test_large_pool_offsets_pass_32_bits():
    """Pages behind the first 4 GiB of the pool, written and read."""
    h, hkv, d, ps = 32, 8, 128, 128
    n_pages = 33000  # 128 KiB of codes each: 4.3 GB
    pool = Pool([300], hkv, d, ps, 35, extra=1)
    pool.n_pages = n_pages
    pool.k = torch.full((n_pages, hkv, ps, d), 0x7F, dtype=torch.uint8, device="cuda")
    pool.v = torch.full((n_pages, hkv, ps, d), 0x7F, dtype=torch.uint8, device="cuda")
    pool.ks, pool.vs = torch.full((2, n_pages, hkv), math.nan, device="cuda").unbind(0)
    pool.table = ints([[n_pages - 1, n_pages - 3, n_pages - 2]])
    x = (torch.randn(300, (h + 2 * hkv) * d, generator=gen(36), device="cuda") * 1.28).bfloat16()
    q_out = torch.empty(300, h, d, dtype=torch.bfloat16, device="cuda")
    run_append(pool, x, q_out, h, [300], [300], freqs(d), "half", "bf16")
    k = rotate64(x.double().view(300, h + 2 * hkv, d)[:, h:h + hkv], torch.arange(300, device="cuda"), freqs(d), "half", 1.0)
    got, _ = pool.rows(0, 300)
    smax = pool.ks[pool.table[0].long()].double().amax()
    assert bool(((got.transpose(0, 1) - k).abs() <= 2.0 ** -4 * k.abs() + 2.0 ** -10 * smax + 1e-4).all())
    out = torch.empty(1, h, d, dtype=torch.bfloat16, device="cuda")
    run_paged(pool, q_out[299:], out, [300], "bf16")
    check_paged(pool, q_out[299:], out, [300], "bf16")
    del pool, got
    torch.cuda.empty_cache()


# ------------------------------------------------------------------------------------------------ prefill
def run_prefill(q, k, v, out, lq, lk, dtype, causal=True, scale=None, status=None, max_q=None, n_q=None, n_k=None):
    cu_q = lq if isinstance(lq, torch.Tensor) else ints(offsets(lq))
    cu_k = lk if isinstance(lk, torch.Tensor) else ints(offsets(lk))
    pkg.attention_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
                          n_seqs=cu_q.numel() - 1, n_q=q.shape[0] if n_q is None else n_q,
                          n_k=k.shape[0] if n_k is None else n_k, max_q=max(lq) if max_q is None else max_q,
                          n_heads=q.shape[1], n_kv_heads=k.shape[1], head_dim=q.shape[2], dtype=DT[dtype][1],
                          causal=causal, strides=(q.stride(0), k.stride(0), v.stride(0), out.stride(0)), scale=scale,
                          status=None if status is None else status.data_ptr(), stream=stream())


def check_prefill(q, k, v, out, lq, lk, dtype, causal=True, scale=None):
    d = q.shape[2]
    scale = d ** -0.5 if scale is None else scale
    q0 = k0 = 0
    for b, (m, n) in enumerate(zip(lq, lk)):
        if m:
            qs, ks, vs = (t.double().transpose(0, 1) for t in (q[q0:q0 + m], k[k0:k0 + n], v[k0:k0 + n]))
            seen = None
            if causal:
                seen = torch.arange(n, device="cuda")[None, :] <= torch.arange(m, device="cuda")[:, None] + n - m
            ref, a, s = attend64(qs, ks, vs, scale, seen)
            tol = attend_tol(ref, a, s, n, d, dtype, 2.0 ** -8 if dtype == "bf16" else 0.0)
            err = (out[q0:q0 + m].double().transpose(0, 1) - ref).abs()
            assert bool((err <= tol).all()), (b, m, n, float((err / tol).max()))
        q0, k0 = q0 + m, k0 + n


def prefill_inputs(h, hkv, d, nq, nk, dtype, seed, std=1.28):
    g = gen(seed)
    t = DT[dtype][0]
    return tuple((torch.randn(n, hh, d, generator=g, device="cuda") * std).to(t)
                 for n, hh in ((nq, h), (nk, hkv), (nk, hkv)))


PREFILL = [
    # h, hkv, d, lq, lk (None: as lq)
    (6, 2, 64, [1], None),
    (6, 2, 64, [77], None),
    (32, 8, 128, [128, 1, 0, 129, 127, 255, 256, 257], None),
    (16, 2, 128, [513, 64, 300], None),
    (8, 1, 64, [63, 64, 65, 2], None),
    (4, 4, 64, [1000, 17], None),
    (4, 2, 128, [5, 130, 0, 1], [900, 131, 10, 1025]),
    (7, 1, 64, [300, 10], [20, 4]),          # queries before the first key see nothing
    (2, 2, 128, [3, 2], [0, 5]),
    (8, 2, 64, [1700], None),
    (4, 2, 64, [1, 0, 3, 5, 2] * 60, None),  # many tiny prompts
    (3, 1, 64, [200, 70], None),             # three heads of one kv head: none to pair with
    (6, 2, 128, [140, 300], None),           # the same, heads of 128
    (2, 2, 64, [4, 2], [0, 0]),              # no keys at all
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [True, False], ids=["causal", "full"])
@pytest.mark.parametrize("case", PREFILL, ids=lambda c: "h%d_%d_d%d_n%d_max%d" % (*c[:3], len(c[3]), max(c[3])))
def test_prefill(case, causal, dtype):
    h, hkv, d, lq, lk = case
    lk = lq if lk is None else lk
    q, k, v = prefill_inputs(h, hkv, d, sum(lq), max(1, sum(lk)), dtype, 40)
    out = torch.full((sum(lq) + 2, h, d), 7.0, dtype=q.dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    run_prefill(q, k, v, out, lq, lk, dtype, causal, status=status, n_q=sum(lq), n_k=sum(lk))
    torch.cuda.synchronize()
    assert int(status) == 0
    check_prefill(q, k, v, out, lq, lk, dtype, causal)
    assert bool((out[sum(lq):] == 7.0).all())
    again = out.clone()
    run_prefill(q, k, v, again, lq, lk, dtype, causal, n_q=sum(lq), n_k=sum(lk), max_q=max(lq) + 1000)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_fused_rows(dtype):
    """q, k and v as slices of one fused projection's rows, out inside a wider buffer."""
    h, hkv, d, lens = 6, 2, 64, [150, 33]
    n = sum(lens)
    x = (torch.randn(n, (h + 2 * hkv) * d, generator=gen(41), device="cuda")).to(DT[dtype][0])
    q, k, v = (t.unflatten(1, (-1, d)) for t in (x[:, :h * d], x[:, h * d:(h + hkv) * d], x[:, (h + hkv) * d:]))
    wide = torch.full((n, h * d + 32), 7.0, dtype=x.dtype, device="cuda")
    out = wide[:, :h * d].unflatten(1, (h, d))
    run_prefill(q, k, v, out, lens, lens, dtype)
    check_prefill(q, k, v, out, lens, lens, dtype)
    assert bool((wide[:, h * d:] == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_unseen_keys_may_hold_anything(d, dtype):
    """NaN and infinities in later keys and values of the same prompt, in another prompt and behind the last."""
    h, hkv, lens, bad = 4, 2, [200, 90, 140], 150
    q, k, v = prefill_inputs(h, hkv, d, sum(lens), sum(lens) + 50, dtype, 42)
    clean = torch.empty_like(q)
    run_prefill(q, k, v, clean, lens, lens, dtype, n_k=sum(lens))
    for t in (k, v):
        t[bad:200, 0] = math.nan
        t[bad + 7, 1] = math.inf
        t[200:290, 1, ::2] = -math.inf
        t[sum(lens):] = math.nan
    out = torch.empty_like(q)
    run_prefill(q, k, v, out, lens, lens, dtype, n_k=sum(lens))
    check_prefill(q[:bad], k[:bad], v[:bad], out, [bad], [bad], dtype)
    check_prefill(q[290:], k[290:], v[290:], out[290:], lens[2:], lens[2:], dtype)
    assert bool(torch.isnan(out[bad:200, :2]).all())  # these do see them
    assert bool(torch.isfinite(out[:bad + 7, 2:]).all())
    assert torch.isnan(out[bad + 7:200, 2:]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,hkv,d", [(4, 2, 64), (3, 1, 128), (8, 2, 128)])
def test_prefill_one_long_among_many_short(h, hkv, d, dtype):
    """Tiles of the whole batch, not as many for each as the longest has; rows before the first sequence; empty ones."""
    lens = [(3 * i) % 7 for i in range(250)] + [1500] + [129, 0, 128] + [(5 * i) % 4 for i in range(250)]
    before = 300
    n = before + sum(lens)
    q, k, v = prefill_inputs(h, hkv, d, n, n, dtype, 48)
    out = torch.full((n + 1, h, d), 7.0, dtype=q.dtype, device="cuda")
    cu, status = ints([before + a for a in offsets(lens)]), torch.zeros(1, dtype=torch.int32, device="cuda")
    run_prefill(q, k, v, out, cu, cu, dtype, max_q=1500, status=status)
    check_prefill(q[before:], k[before:], v[before:], out[before:], lens, lens, dtype)
    assert int(status) == 0 and bool((out[:before] == 7.0).all()) and bool((out[n:] == 7.0).all())
    # an offset out of order leaves such a batch out whole
    bad = cu.clone()
    bad[100] = before - 1
    out.fill_(7.0)
    run_prefill(q, k, v, out, bad, cu, dtype, max_q=1500, status=status)
    torch.cuda.synchronize()
    assert int(status) == D_.DEC_SEQ_BAD_RANGE and bool((out == 7.0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_infinity(d, dtype):
    """A query whose every score is -infinity, or any is +infinity, has no softmax: NaN, in its own row and head alone."""
    h, hkv, n = 4, 2, 150
    q, k, v = prefill_inputs(h, hkv, d, n, n, dtype, 45)
    k = k.abs() + 0.5
    q[40, 1], q[149, 3] = -math.inf, math.inf
    out = torch.empty_like(q)
    run_prefill(q, k, v, out, [n], [n], dtype)
    bad = torch.isnan(out)
    assert bool(bad[40, 1].all()) and bool(bad[149, 3].all()) and int(bad.sum()) == 2 * d
    lens, ps = [90, 20], 32
    pool = Pool(lens, hkv, d, ps, 46).fill(lens, 47)
    pool.k &= 0x7F  # no negative keys
    pool.k[pool.k == 0] = 0x20
    x = q[:2].clone()
    x[0, 1], x[1, 3] = -math.inf, math.inf
    out = torch.empty_like(x)
    run_paged(pool, x, out, lens, dtype)
    bad = torch.isnan(out)
    assert bool(bad[0, 1].all()) and bool(bad[1, 3].all()) and int(bad.sum()) == 2 * d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_large_scores(dtype):
    h, hkv, d, lens = 4, 2, 64, [300]
    for std, scale in ((12.0, None), (1e-3, None), (1.0, 0.5)):
        q, k, v = prefill_inputs(h, hkv, d, 300, 300, dtype, 43, std)
        out = torch.empty_like(q)
        run_prefill(q, k, v, out, lens, lens, dtype, scale=scale)
        check_prefill(q, k, v, out, lens, lens, dtype, scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["keys_past", "queries_past", "decreasing", "above_max"])
def test_prefill_inconsistent_sequences(what, dtype):
    h, hkv, d, lens = 4, 2, 64, [70, 40, 60]
    q, k, v = prefill_inputs(h, hkv, d, 170, 170, dtype, 44)
    out, status = torch.full_like(q, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
    cu_q, cu_k, max_q, good = offsets(lens), offsets(lens), 70, [0, 1]
    if what == "keys_past":
        cu_k[3] = 171
    elif what == "queries_past":
        cu_q[3] = 2 ** 31 - 1
    elif what == "decreasing":
        cu_k[3] = 100
    else:
        max_q, good = 64, [1, 2]
    run_prefill(q, k, v, out, ints(cu_q), ints(cu_k), dtype, status=status, max_q=max_q)
    torch.cuda.synchronize()
    assert int(status) == D_.DEC_SEQ_BAD_RANGE
    at = offsets(lens)
    for b in good:
        s = slice(at[b], at[b + 1])
        check_prefill(q[s], k[s], v[s], out[s], [lens[b]], [lens[b]], dtype)
    bad = out[110:] if what != "above_max" else out[:64]
    assert bool((bad == (7.0 if what == "queries_past" else 0.0)).all())


# ------------------------------------------------------------------------------------------------ together
def test_empty_calls_do_nothing():
    pool = Pool([5], 2, 64, 16, 50)
    c = pool.cache()
    c.append(None, None, None, None, None, None, None, table_stride=0, n_seqs=0, n_tokens=0, max_new=0, n_heads=4)
    c.attention(None, None, None, None, table_stride=0, n_seqs=0, n_heads=4, workspace=None, workspace_bytes=0)
    pkg.attention_prefill(None, None, None, None, None, None, n_seqs=0, n_q=0, n_k=0, max_q=0, n_heads=4, n_kv_heads=2,
                          head_dim=64)


def test_host_pointers_and_pending_work_are_refused():
    """A host address would fault in a kernel: refused before a launch."""
    h, hkv, d, ps = 4, 2, 64, 16
    pool = Pool([20], hkv, d, ps, 51).fill([20], 52)
    q = torch.randn(1, h, d, device="cuda")
    out = torch.empty_like(q)
    host = torch.empty(4096, pin_memory=True)
    with pytest.raises(pkg.DecError) as e:
        pool.cache().attention(q.data_ptr(), host.data_ptr(), ints([20]).data_ptr(), pool.table.data_ptr(),
                               table_stride=pool.width, n_seqs=1, n_heads=h, dtype=D_.DEC_F32,
                               workspace=torch.empty(1 << 24, device="cuda").data_ptr(), workspace_bytes=1 << 26)
    assert e.value.code == D_.DEC_ERR_INVALID_ARG
    with pytest.raises(pkg.DecError) as e:
        pkg.attention_prefill(q.data_ptr(), q.data_ptr(), torch.zeros(h * d).data_ptr() & ~15, out.data_ptr(),
                              ints([0, 1]).data_ptr(), ints([0, 1]).data_ptr(), n_seqs=1, n_q=1, n_k=1, max_q=1,
                              n_heads=h, n_kv_heads=h, head_dim=d, dtype=D_.DEC_F32)
    assert e.value.code == D_.DEC_ERR_INVALID_ARG


def chain(dtype, h, hkv, d, ps, prompts, steps, capture):
    """Prompts through the three operators, then decode steps for the whole batch, on a stream of its own."""
    n = len(prompts)
    total = [p + steps for p in prompts]
    pool = Pool(total, hkv, d, ps, 60)
    t = DT[dtype][0]
    fr = freqs(d)
    x = (torch.randn(sum(prompts), (h + 2 * hkv) * d, generator=gen(61), device="cuda") * 1.28).to(t)
    xs = (torch.randn(steps, n, (h + 2 * hkv) * d, generator=gen(62), device="cuda") * 1.28).to(t)
    q0 = torch.empty(sum(prompts), h, d, dtype=t, device="cuda")
    c = pool.cache()
    work = torch.cuda.Stream()
    work.wait_stream(torch.cuda.current_stream())
    e = x.element_size()
    row = x.stride(0)
    outs = []
    with torch.cuda.stream(work):
        st = work.cuda_stream
        cu, lens = ints(offsets(prompts)), ints(prompts)
        kr = torch.empty(sum(prompts), hkv, d, dtype=t, device="cuda")
        c.append(x.data_ptr(), x.data_ptr() + h * d * e, x.data_ptr() + (h + hkv) * d * e, q0.data_ptr(), cu.data_ptr(),
                 lens.data_ptr(), pool.table.data_ptr(), table_stride=pool.width, n_seqs=n, n_tokens=sum(prompts),
                 max_new=max(prompts), n_heads=h, dtype=DT[dtype][1], strides=(row, row, row, h * d),
                 inv_freq=fr.data_ptr(), rot_dim=d, k_out=kr.data_ptr(), stream=st)
        o0 = torch.empty_like(q0)
        v = x.view(-1, h + 2 * hkv, d)[:, h + hkv:]
        pkg.attention_prefill(q0.data_ptr(), kr.data_ptr(), v.data_ptr(), o0.data_ptr(), cu.data_ptr(), cu.data_ptr(),
                              n_seqs=n, n_q=sum(prompts), n_k=sum(prompts), max_q=max(prompts), n_heads=h, n_kv_heads=hkv,
                              head_dim=d, dtype=DT[dtype][1], strides=(h * d, hkv * d, row, h * d), stream=st)
        one = ints(list(range(n + 1)))
        xin, q1, o1 = torch.empty_like(xs[0]), torch.empty(n, h, d, dtype=t, device="cuda"), torch.empty(n, h, d, dtype=t, device="cuda")
        space = torch.empty(c.workspace_bytes(n, h), dtype=torch.uint8, device="cuda")

        def step(st):
            lens.add_(1)
            c.append(xin.data_ptr(), xin.data_ptr() + h * d * e, xin.data_ptr() + (h + hkv) * d * e, q1.data_ptr(),
                     one.data_ptr(), lens.data_ptr(), pool.table.data_ptr(), table_stride=pool.width, n_seqs=n, n_tokens=n,
                     max_new=1, n_heads=h, dtype=DT[dtype][1], strides=(row, row, row, h * d), inv_freq=fr.data_ptr(),
                     rot_dim=d, stream=st)
            c.attention(q1.data_ptr(), o1.data_ptr(), lens.data_ptr(), pool.table.data_ptr(), table_stride=pool.width,
                        n_seqs=n, n_heads=h, dtype=DT[dtype][1], workspace=space.data_ptr(),
                        workspace_bytes=space.numel(), stream=st)

        graph = None
        if capture:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=work):
                step(torch.cuda.current_stream().cuda_stream)
        for i in range(steps):
            xin.copy_(xs[i])
            if graph is not None:
                graph.replay()
            else:
                step(st)
            outs.append((q1.clone(), o1.clone()))
    work.synchronize()
    return pool, x, xs, q0, kr, o0, outs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_decode(dtype):
    """Prompt append and attention, then decode steps, eager and from one captured graph: equal bits; against float64 over
    the cache's own codes, which append's tests hold to the inputs."""
    h, hkv, d, ps, prompts, steps = 8, 2, 64, 16, [30, 1, 47], 20
    eager = chain(dtype, h, hkv, d, ps, prompts, steps, False)
    graph = chain(dtype, h, hkv, d, ps, prompts, steps, True)
    for a, b in zip(eager[6], graph[6]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(eager[0].k, graph[0].k) and torch.equal(eager[0].v, graph[0].v)
    pool, x, xs, q0, kr, o0, outs = eager
    check_prefill(q0, kr, x.view(-1, h + 2 * hkv, d)[:, h + hkv:], o0, prompts, prompts, dtype)
    q1, o1 = outs[-1]
    check_paged(pool, q1, o1, [p + steps for p in prompts], dtype)
    # against attention over the unrounded keys and values: E4M3 is off by 2^-4 of a value at most, so a score by 2^-4 S,
    # a weight by a factor of e^(2 * 2^-4 S), and the result by (that - 1 + 2^-4) A; typical errors are far smaller
    for b, p in enumerate(prompts):
        at = offsets(prompts)[b]
        rows = torch.cat([x[at:at + p], xs[:, b]]).double().view(p + steps, h + 2 * hkv, d)
        k = rotate64(rows[:, h:h + hkv], torch.arange(p + steps, device="cuda"), freqs(d), "half", 1.0).transpose(0, 1)
        ref, a, s = attend64(q1[b].double()[:, None], k, rows[:, h + hkv:].transpose(0, 1), d ** -0.5)
        err = (o1[b].double()[:, None] - ref).abs()
        assert bool((err <= a * (math.expm1(2.0 ** -3 * s) + 2.0 ** -4) + 2.0 ** -6).all())
        assert float(err.norm() / ref.norm()) < 2.0 ** -3  # errors of single roundings average out; a wrong rotation gives order 1


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn."""
    h, hkv, d, ps = 8, 2, 128, 64
    pools = [Pool(lens, hkv, d, ps, 70 + i).fill(lens, 72 + i) for i, lens in enumerate(([3000, 5], [700, 2000]))]
    q = torch.randn(2, 2, h, d, generator=gen(74), device="cuda")
    out = torch.empty_like(q)
    space = torch.empty(pools[0].cache().workspace_bytes(2, h), dtype=torch.uint8, device="cuda")
    lens = [ints(p.lens) for p in pools]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run_paged(pools[i], q[i], out[i], lens[i], "f32", space=space)
        graphs.append(g)
    for _ in range(3):
        out.fill_(7.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            check_paged(pools[i], q[i], out[i], pools[i].lens, "f32")
    lens[0].copy_(ints([11, 1234 % 300]))  # a replay reads the lengths that are there
    graphs[0].replay()
    torch.cuda.synchronize()
    check_paged(pools[0], q[0][:1], out[0][:1], [11], "f32")
