"""The stand-alone attention operators, measured: appending to the 8-bit paged cache with the position rotation,
single-token attention over that cache, and attention over packed prompts.

`own = False` computes each in plain float32 torch operations; `own = True` makes the library's calls.  The head
layouts are those of the repository's dense workloads (synth/workloads.py); keys, values and queries have the
spread of a projection of a unit-RMS vector by N(0, 0.02^2) weights.
"""
import math
import random

import torch

own = False

HEADS = [(32, 8, 128), (32, 8, 64), (16, 2, 128), (6, 2, 64), (4, 2, 128), (8, 1, 64), (4, 4, 64)]
STD = 1.28  # 0.02 * sqrt(4096)
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding: a single token into a page that already holds others; latency
        dict(name="append_1_token", op="append", n_seqs=1, old=1024, new=1, ragged=0, heads=32, kv_heads=8, dim=128,
             page=64, rot=128, pairs="half", dtype="bf16", mix=1),
        # a decode batch: one token for each of 256 sequences of different lengths
        dict(name="append_256_tokens", op="append", n_seqs=256, old=2000, new=1, ragged=1, heads=32, kv_heads=8,
             dim=128, page=64, rot=128, pairs="half", dtype="bf16", mix=2),
        # ragged chunks of prompts behind what is cached, fp32 activations, part of the head rotated in neighbour pairs
        dict(name="append_chunks_f32", op="append", n_seqs=11, old=333, new=301, ragged=1, heads=6, kv_heads=2, dim=64,
             page=16, rot=32, pairs="neighbour", dtype="f32", mix=3),
        # four whole prompts of 8k
        dict(name="append_4_prompts_8k", op="append", n_seqs=4, old=0, new=8192, ragged=0, heads=32, kv_heads=8,
             dim=128, page=64, rot=128, pairs="half", dtype="bf16", mix=4),
        # one short sequence, the small workload's heads; latency
        dict(name="paged_1x77", op="paged", n_seqs=1, len=77, ragged=0, heads=6, kv_heads=2, dim=64, page=16,
             dtype="bf16", mix=5),
        # one sequence at the 8k workload's context: split over the GPU
        dict(name="paged_1x8k", op="paged", n_seqs=1, len=8193, ragged=0, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", mix=6),
        # fp32 queries, eight heads a kv head, a ragged batch with an empty sequence
        dict(name="paged_33_f32", op="paged", n_seqs=33, len=5000, ragged=1, heads=16, kv_heads=2, dim=128, page=32,
             dtype="f32", mix=7),
        # a serving batch: 128 sequences of up to 8k
        dict(name="paged_128x8k", op="paged", n_seqs=128, len=8192, ragged=1, heads=32, kv_heads=8, dim=128, page=64,
             dtype="bf16", mix=8),
        # one short prompt; latency
        dict(name="prefill_77", op="prefill", n_seqs=1, len=77, ragged=0, before=0, causal=True, heads=6, kv_heads=2,
             dim=64, dtype="bf16", mix=9),
        # packed prompts of different lengths, fp32
        dict(name="prefill_ragged_f32", op="prefill", n_seqs=5, len=700, ragged=1, before=0, causal=True, heads=4,
             kv_heads=4, dim=64, dtype="f32", mix=10),
        # packed prompts of different lengths, some behind keys that are there already (a later chunk of a prompt)
        dict(name="prefill_ragged_6x1k", op="prefill", n_seqs=6, len=1500, ragged=1, before=500, causal=True, heads=32,
             kv_heads=8, dim=64, dtype="bf16", mix=11),
        # the 8k workload's whole prompt
        dict(name="prefill_8k", op="prefill", n_seqs=1, len=8192, ragged=0, before=0, causal=True, heads=32,
             kv_heads=8, dim=128, dtype="bf16", mix=12),
    ]


def draw(rng):
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    h, hkv, d = rng.choice(HEADS)
    op = rng.choice(["append", "paged", "prefill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    case = dict(op=op, heads=h, kv_heads=hkv, dim=d, dtype=dtype, ragged=rng.choice([0, 1, 1]), mix=rng.randrange(1 << 20))
    if op == "append":
        n = log_int(1, 256)
        case.update(n_seqs=n, old=rng.choice([0, log_int(1, 4000)]), new=log_int(1, max(1, 16384 // n)),
                    page=rng.choice([16, 32, 64, 128]), rot=rng.choice([d, d, d // 2, 0]),
                    pairs=rng.choice(["half", "neighbour"]))
    elif op == "paged":
        n = log_int(1, 128)
        case.update(n_seqs=n, len=log_int(1, min(16384, 524288 // n)), page=rng.choice([16, 32, 64, 128]))
    else:
        n = log_int(1, 16)
        top = 4096 if dtype == "bf16" else 1024
        case.update(n_seqs=n, len=log_int(1, max(1, top // n)), before=rng.choice([0, 0, log_int(1, max(1, 2000 // n))]),
                    causal=rng.random() < 0.8)
    return case


def _ragged(case, top, salt):
    """One length for each sequence, from the case alone: all `top`, or spread over 0..top with the first at `top`."""
    n = case["n_seqs"]
    if not case["ragged"]:
        return [top] * n
    r = random.Random(case["mix"] * 7 + salt)
    return [top] + [int(top * r.random() ** 0.7) for _ in range(n - 1)]


def _append_lens(case):
    new = _ragged(case, case["new"], 1) if case["new"] > 1 else [1] * case["n_seqs"]
    return _ragged(case, case["old"], 2), new


def _prefill_lens(case):
    lq = _ragged(case, case["len"], 1)
    return lq, [a + b for a, b in zip(lq, _ragged(case, case["before"], 2))]


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    h, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        old, new = _append_lens(case)
        t = sum(new)
        pages = sum(-(-(a + b) // case["page"]) - a // case["page"] for a, b in zip(old, new) if b)
        return dict(bytes=t * ((2 * h + 2 * hkv) * d * e + 2 * hkv * d) + pages * hkv * 8, flops=t * (h + hkv) * d * 3)
    if case["op"] == "paged":
        lens = _ragged(case, case["len"], 1)
        t = sum(lens)
        pages = sum(-(-n // case["page"]) for n in lens)
        return dict(bytes=t * 2 * hkv * d + pages * (hkv * 8 + 4) + 2 * case["n_seqs"] * h * d * e, flops=4 * t * h * d)
    lq, lk = _prefill_lens(case)
    pairs = sum(a * b - (a * (a - 1) // 2 if case["causal"] else 0) for a, b in zip(lq, lk))
    return dict(bytes=e * d * (2 * h * sum(lq) + 2 * hkv * sum(lk)), flops=4 * pairs * h * d)


# ------------------------------------------------------------------------------------------------ inputs
def _normal(g, shape, dtype):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * STD
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def _pool(case, g, lens):
    """A pool of pages in random order with every sequence's pages filled: codes, power-of-two scales, page table."""
    hkv, d, ps = case["kv_heads"], case["dim"], case["page"]
    need = [-(-n // ps) for n in lens]
    n_pages, width = sum(need) + 3, max(1, max(need))
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(len(lens), width, dtype=torch.int32, device="cuda")
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    codes, scales = [], []
    for _ in range(2):
        x = torch.randn(n_pages, hkv, ps, d, generator=g, device="cuda") * STD
        m, e = torch.frexp(x.abs().amax((2, 3)))
        s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int())
        codes.append((x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8))
        scales.append(s)
        del x
    return codes[0], codes[1], scales[0], scales[1], table


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h, hkv, d, dt = case["heads"], case["kv_heads"], case["dim"], case["dtype"]
    s = dict(case=case)
    if case["op"] == "append":
        old, new = _append_lens(case)
        lens = [a + b for a, b in zip(old, new)]
        s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"] = _pool(case, g, lens)
        s["qkv"] = _normal(g, (max(1, sum(new)), (h + 2 * hkv) * d), dt)  # one fused projection's output
        s["q_out"] = torch.empty(max(1, sum(new)), h, d, dtype=s["qkv"].dtype, device="cuda")
        s["cu"], s["lens"] = _ints(_offsets(new)), _ints(lens)
        s["n_tokens"], s["max_new"] = sum(new), max(new)
        r = case["rot"]
        s["inv_freq"] = 10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / max(1, r))
    elif case["op"] == "paged":
        lens = _ragged(case, case["len"], 1)
        s["k_pages"], s["v_pages"], s["k_scales"], s["v_scales"], s["table"] = _pool(case, g, lens)
        s["q"] = _normal(g, (case["n_seqs"], h, d), dt)
        s["out"] = torch.empty_like(s["q"])
        s["lens"] = _ints(lens)
    else:
        lq, lk = _prefill_lens(case)
        s["q"] = _normal(g, (max(1, sum(lq)), h, d), dt)
        s["k"] = _normal(g, (max(1, sum(lk)), hkv, d), dt)
        s["v"] = _normal(g, (max(1, sum(lk)), hkv, d), dt)
        s["out"] = torch.empty_like(s["q"])
        s["cu_q"], s["cu_k"] = _ints(_offsets(lq)), _ints(_offsets(lk))
        s["n_q"], s["n_k"], s["max_q"] = sum(lq), sum(lk), max(lq)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, pairs):
    """x [T, heads, D] float32; cos, sin [T, R/2]."""
    r = 2 * cos.shape[1]
    y = x.clone()
    c, s = cos[:, None], sin[:, None]
    if pairs == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * s, a * s + b * c
    return y


def _plain_append(s):
    case = s["case"]
    h, hkv, d, ps, t = case["heads"], case["kv_heads"], case["dim"], case["page"], s["n_tokens"]
    x = s["qkv"][:t].float().view(t, h + 2 * hkv, d)
    cu, lens = s["cu"].long(), s["lens"].long()
    i = torch.arange(t, device="cuda")
    seq = torch.searchsorted(cu, i, right=True) - 1
    pos = lens[seq] - cu[seq + 1] + i
    angle = pos.double()[:, None] * s["inv_freq"]  # 64 bits: far positions turn many times
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s["q_out"][:t] = _rotate(x[:, :h], cos, sin, case["pairs"]).to(s["q_out"].dtype)
    page, slot = s["table"][seq, pos // ps].long(), pos % ps
    start, count = lens - cu[1:] + cu[:-1], cu[1:] - cu[:-1]
    part = ((start % ps > 0) & (count > 0))[:, None]  # sequences whose first new token joins a page in use
    first = s["table"].gather(1, (start // ps).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0].long()
    for x_, pages, scales in ((_rotate(x[:, h:h + hkv], cos, sin, case["pairs"]), s["k_pages"], s["k_scales"]),
                              (x[:, h + hkv:], s["v_pages"], s["v_scales"])):
        amax = torch.zeros_like(scales).index_reduce_(0, page, x_.abs().amax(-1), "amax")
        m, e = torch.frexp(amax.clamp(min=2.0 ** -120))
        need = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int()).clamp(-120, 120))
        was = scales[first]
        now = torch.where(part, torch.maximum(was, need[first]), was)
        fresh = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page[slot == 0], True)
        scales.copy_(torch.where(fresh[:, None], need, scales))
        rows = torch.where(part[:, 0])[0]
        scales[first[rows]] = now[rows]
        before = pages[first[rows]]
        again = (before.view(torch.float8_e4m3fn).float() * (was / now)[rows][:, :, None, None])
        again = again.to(torch.float8_e4m3fn).view(torch.uint8)
        keep = torch.arange(ps, device="cuda")[None, :] < (start % ps)[rows][:, None]
        pages[first[rows]] = torch.where(keep[:, None, :, None], again, before)
        code = (x_ / scales[page][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        pages[page, :, slot] = code.view(torch.uint8)


def _plain_paged(s):
    case = s["case"]
    n, h, hkv, d = case["n_seqs"], case["heads"], case["kv_heads"], case["dim"]
    table = s["table"].long()
    top = table.shape[1] * case["page"]
    kv = []
    for pages, scales in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])):
        x = pages.view(torch.float8_e4m3fn).float() * scales[:, :, None, None]
        kv.append(x[table].permute(0, 2, 1, 3, 4).reshape(n, hkv, top, d))
    q = s["q"].float().view(n, hkv, h // hkv, d)
    score = (q @ kv[0].transpose(-1, -2)) / math.sqrt(d)
    seen = (torch.arange(top, device="cuda")[None, :] < s["lens"][:, None])[:, None, None]
    score = score.masked_fill(~seen, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38)).masked_fill(~seen, 0.0)
    o = (p @ kv[1]) / p.sum(-1, keepdim=True).clamp(min=1e-38)
    s["out"].copy_(o.view(n, h, d))


def _plain_prefill(s):
    case = s["case"]
    h, hkv, d, nq, nk = case["heads"], case["kv_heads"], case["dim"], s["n_q"], s["n_k"]
    q = s["q"][:nq].float().view(nq, hkv, h // hkv, d).permute(1, 2, 0, 3)
    k, v = (s[c][:nk].float().permute(1, 0, 2)[:, None] for c in "kv")
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    i, t = torch.arange(nq, device="cuda"), torch.arange(nk, device="cuda")
    qs, ks = torch.searchsorted(cu_q, i, right=True) - 1, torch.searchsorted(cu_k, t, right=True) - 1
    seen = qs[:, None] == ks[None, :]
    if case["causal"]:  # the last query sees the last key
        seen &= (t[None, :] - cu_k[qs + 1][:, None]) <= (i - cu_q[qs + 1])[:, None]
    score = (q @ k.transpose(-1, -2)).div_(math.sqrt(d)).masked_fill_(~seen, -math.inf)
    score.sub_(score.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    o = (score @ v) / score.sum(-1, keepdim=True).clamp(min=1e-38)
    s["out"][:nq] = o.permute(2, 0, 1, 3).reshape(nq, h, d).to(s["out"].dtype)


# ------------------------------------------------------------------------------------------------ the library's calls
def _own(s):
    import persistent_sm_decode_02_b200 as pkg

    case = s["case"]
    h, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    dtype = pkg.dec.DEC_BF16 if case["dtype"] == "bf16" else pkg.dec.DEC_F32
    stream = torch.cuda.current_stream().cuda_stream
    if case["op"] == "prefill":
        pkg.attention_prefill(s["q"].data_ptr(), s["k"].data_ptr(), s["v"].data_ptr(), s["out"].data_ptr(),
                              s["cu_q"].data_ptr(), s["cu_k"].data_ptr(), n_seqs=case["n_seqs"], n_q=s["n_q"],
                              n_k=s["n_k"], max_q=s["max_q"], n_heads=h, n_kv_heads=hkv, head_dim=d, dtype=dtype,
                              causal=case["causal"], stream=stream)
        return
    cache = s.get("cache")
    if cache is None:  # a user's program keeps the cache's description, and the workspace, for its whole life
        cache = s["cache"] = pkg.PagedCache(s["k_pages"].data_ptr(), s["v_pages"].data_ptr(), s["k_scales"].data_ptr(),
                                            s["v_scales"].data_ptr(), n_pages=s["k_pages"].shape[0],
                                            page_size=case["page"], n_kv_heads=hkv, head_dim=d)
    table, width = s["table"].data_ptr(), s["table"].shape[1]
    if case["op"] == "append":
        x, size = s["qkv"].data_ptr(), s["qkv"].element_size()
        row = s["qkv"].shape[1]
        cache.append(x, x + h * d * size, x + (h + hkv) * d * size, s["q_out"].data_ptr(), s["cu"].data_ptr(),
                     s["lens"].data_ptr(), table, table_stride=width, n_seqs=case["n_seqs"], n_tokens=s["n_tokens"],
                     max_new=s["max_new"], n_heads=h, dtype=dtype, strides=(row, row, row, h * d),
                     inv_freq=s["inv_freq"].data_ptr(), rot_dim=case["rot"], neighbour_pairs=case["pairs"] == "neighbour",
                     stream=stream)
    else:
        space = s.get("space")
        if space is None:
            space = s["space"] = torch.empty(cache.workspace_bytes(case["n_seqs"], h), dtype=torch.uint8, device="cuda")
        cache.attention(s["q"].data_ptr(), s["out"].data_ptr(), s["lens"].data_ptr(), table, table_stride=width,
                        n_seqs=case["n_seqs"], n_heads=h, dtype=dtype, workspace=space.data_ptr(),
                        workspace_bytes=space.numel(), stream=stream)


def run(state):
    op = state["case"]["op"]
    if own:
        _own(state)
    elif op == "append":
        _plain_append(state)
    elif op == "paged":
        _plain_paged(state)
    else:
        _plain_prefill(state)
    if op == "append":  # the codes as the numbers they are, and what each page's and head's are multiplied by
        return dict(q=state["q_out"][:state["n_tokens"]], k=state["k_pages"].view(torch.float8_e4m3fn),
                    v=state["v_pages"].view(torch.float8_e4m3fn), k_scales=state["k_scales"],
                    v_scales=state["v_scales"])
    return state["out"] if op == "paged" else state["out"][:state["n_q"]]


# ------------------------------------------------------------------------------------------------ in 64 bits
def _e4m3_64(x):
    """Nearest E4M3 value of float64 x, ties to even, saturating."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    h, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        old, new = _append_lens(case)
        ps, r = case["page"], case["rot"]
        x = s["qkv"].double().view(-1, h + 2 * hkv, d)
        cache = [s[c].view(torch.float8_e4m3fn).double() for c in ("k_pages", "v_pages")]
        scale = [s[c].double() for c in ("k_scales", "v_scales")]
        half = case["pairs"] == "half"
        first = torch.arange(r // 2, device="cuda") * (1 if half else 2)
        second = first + (r // 2 if half else 1)
        table, q = s["table"].tolist(), []
        at = 0
        for b, (o, n) in enumerate(zip(old, new)):
            if n == 0:
                continue
            angle = torch.arange(o, o + n, device="cuda", dtype=torch.float64)[:, None, None] * s["inv_freq"]
            rows = x[at:at + n].clone()
            at += n
            u, w = rows[:, :h + hkv, first], rows[:, :h + hkv, second]
            rows[:, :h + hkv, first] = u * torch.cos(angle) - w * torch.sin(angle)
            rows[:, :h + hkv, second] = u * torch.sin(angle) + w * torch.cos(angle)
            q.append(rows[:, :h])
            for p in range(o // ps, -(-(o + n) // ps)):
                lo, hi = max(o, p * ps), min(o + n, (p + 1) * ps)
                page = table[b][p]
                for c in range(2):
                    piece = rows[lo - o:hi - o, h + c * hkv:h + (c + 1) * hkv]
                    m, e = torch.frexp(piece.abs().amax((0, 2)).clamp(min=2.0 ** -120))
                    now = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int()).clamp(-120, 120))
                    if lo > p * ps:
                        now = torch.maximum(now, scale[c][page])
                        cache[c][page, :, :lo - p * ps] = _e4m3_64(cache[c][page, :, :lo - p * ps] * (
                            scale[c][page] / now)[:, None, None])
                    scale[c][page] = now
                    cache[c][page, :, lo - p * ps:hi - p * ps] = _e4m3_64(piece / now[:, None]).transpose(0, 1)
        return dict(q=torch.cat(q), k=cache[0], v=cache[1], k_scales=scale[0], v_scales=scale[1])
    if case["op"] == "paged":
        out = torch.zeros(case["n_seqs"], h, d, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_ragged(case, case["len"], 1)):
            if n == 0:
                continue
            ids = s["table"][b, :-(-n // case["page"])].long()
            k, v = ((s[c + "_pages"][ids].view(torch.float8_e4m3fn).double() * s[c + "_scales"][ids].double()[
                :, :, None, None]).transpose(0, 1).reshape(hkv, -1, d)[:, :n] for c in "kv")
            q = s["q"][b].double().view(hkv, h // hkv, d)
            out[b] = (torch.softmax(torch.einsum("gid,gtd->git", q, k) / math.sqrt(d), -1) @ v).reshape(h, d)
        return out
    lq, lk = _prefill_lens(case)
    out = torch.zeros(s["n_q"], h, d, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        for i in range(h if a else 0):
            q = s["q"][q0:q0 + a, i].double()
            k, v = (s[c][k0:k0 + b, i // (h // hkv)].double() for c in "kv")
            score = q @ k.T / math.sqrt(d)
            if case["causal"]:
                score += torch.full((a, b), -math.inf, device="cuda", dtype=torch.float64).triu(b - a + 1)
            out[q0:q0 + a, i] = torch.softmax(score, -1) @ v
        q0, k0 = q0 + a, k0 + b
    return out
