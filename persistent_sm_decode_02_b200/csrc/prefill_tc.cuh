// Attention of packed bf16 prompts on tcgen05 tensor cores.
//
// A block takes two tiles of 128 queries that read the same keys (two heads of one kv head, or neighbouring queries
// of one head), and walks their keys in steps of kN:
//   S = Q K^T (128 x kN, fp32 in TMEM), P = 2^(scale log2(e) S - m) rounded to bf16 over S, O += P V.
// Warps 0-3 and 4-7 are the tiles' softmax, a thread a row; warp 8 issues every MMA; warp 9 every TMA load; warp 10 finds work.
//   TMEM: S0 | S1 (kN columns each, P in the first kN / 2) | O0 | O1 (D columns each)
//   shared memory: Q, and a ring of K and V tiles, rows of 128 bytes in the 128-byte swizzle
// A score is taken off its row's maximum by one fma, which is off by half an ulp of the maximum: from 2^26 on (kHuge) that is
// no longer small beside the weights' range, and a warp that met such a maximum computes its rows once more (redo_row).
// The tiles alternate: while one tile's softmax runs, the tensor cores do the other's P V and next Q K^T.
// One thread's MMAs complete in the order they were issued.  So S_i(j + 1), issued behind P V_i(j), may overwrite P_i(j),
// and once it has arrived O_i is at rest until the tile's next P: a softmax thread may rescale its row of O there.  It
// does only when the row's maximum has grown by more than 2^8 (P up to 2^8 and its sum lose nothing).
//
// P is rounded to bf16 (by up to 2^-8 of each weight, as much as V's own rounding and the result's: the two operands of an MMA
// have one type, and V in two parts would double the P V); its sum is of the unrounded weights, in fp32.
//
// An unseen value meets a weight of zero, and zero times NaN or infinity is NaN.  Values behind a sequence's last key (another
// sequence's, or nobody's) are zeroed in shared memory before P V of the step that holds it.  (To cut that P V short at the
// 16 keys that hold it and zero up to 15 rows instead: 2-4 % slower, for the branch in every step.)  Among a sequence's own
// keys such values are rare and rows that have met one show it, so it is looked for only in the results (mend_rows): where a
// result is not finite although every value that the row sees in that dim is, the row is computed once more with the keys it
// sees alone.  That takes a warp long where keys are many; the block's other warps wait for it as long as it gets on.
//
// What it measures: a causal 8k prompt, 32 heads of 128 on 8, 437-497 us, 1.11-1.26 PFLOP/s (67-77 % of cuBLAS's burst
// rate), and 512 us in calls among others for seconds, under the power cap (78 % of its sustained rate); of heads of 64
// 320-343.  With the softmax left out the MMAs, loads and hand-overs of heads of 128 take 395 us: the tensor cores wait for
// hand-overs (about 800 cycles from S to P and on, two tiles to hide them) and for shared memory (Q K^T reads both operands
// there at its full 128 bytes a cycle).  Tried and slower: two threads a row (115 against 100 us for six ragged prompts of up
// to 1500, heads of 64; spills at 128), steps of 64 keys with two S buffers for heads of 128 (543).
#pragma once
#include <cuda.h>

#include <type_traits>

#include "op_common.cuh"
#include "ptx.cuh"

namespace dec_op {

struct PrefillArgs {
  const void *q, *k, *v;
  void* out;
  int64_t qs, ks, vs, os;
  int heads, gs, n_q, n_k, max_q, causal;
  const int32_t *cu_q, *cu_k;
  float scale_log2;
  int32_t* status;
};

struct Range {
  int64_t q0, k0;
  int lq, lk;
  bool ok;
};
__device__ __forceinline__ Range range_of(const PrefillArgs& a, int s) {
  const int64_t q0 = a.cu_q[s], q1 = a.cu_q[s + 1], k0 = a.cu_k[s], k1 = a.cu_k[s + 1];
  const bool q_ok = q0 >= 0 && q1 >= q0 && q1 <= a.n_q, k_ok = k0 >= 0 && k1 >= k0 && k1 <= a.n_k;
  Range r;
  r.q0 = q0;
  r.k0 = k_ok ? k0 : 0;
  r.lq = q_ok ? (int)(q1 - q0) : 0;
  r.lk = k_ok ? (int)(k1 - k0) : 0;
  r.ok = q_ok && k_ok && r.lq <= a.max_q;
  return r;
}

// How queries are cut into tiles of `rows`.  Sequences of about one length: as many tiles for each as the longest has, the
// late ones of all sequences first.  Where that would leave most of them empty: tile t of the whole batch, sequence s
// owning those from cu_q[s] / rows + s on (never fewer than it needs), late sequences first.
struct Tiling {
  int tiles, packed;  // tiles of a sequence, or of the batch
};
inline Tiling tiling(int n_seqs, int n_q, int max_q, int rows) {
  const int64_t each = ((int64_t)max_q + rows - 1) / rows, batch = (int64_t)n_q / rows + n_seqs;
  // 8 prompts of 4096 among 500 of up to 100, 32 heads of 128: 1.35 ms packed, 1.63 with 32 tiles for each; of 64: 1.28, 2.85.
  // Of about one length, the plain cut's order (longest rows of all sequences first) ends more evenly.
  return n_seqs * each > 4 * batch ? Tiling{(int)batch, 1} : Tiling{(int)each, 0};
}
// Tile `at` of the launch (on a whole warp): its sequence and first query.  packed: -1 where an offset is out of order,
// as every later one would be off.
template <bool kPacked>
__device__ __forceinline__ int tile_at(const PrefillArgs& a, int n_seqs, int tiles, int rows, int at, int& m0) {
  if (!kPacked) {
    m0 = (tiles - 1 - at / n_seqs) * rows;
    return at % n_seqs;
  }
  const int t = tiles - 1 - at, lane = threadIdx.x & 31;
  int s = -1, first = 0;
  bool sound = true;
#pragma unroll 1
  for (int i = lane; i - lane < n_seqs; i += 32) {
    const int q0 = i < n_seqs ? a.cu_q[i] : 0, q1 = i < n_seqs ? a.cu_q[i + 1] : 0;
    sound &= q0 >= 0 && q1 >= q0 && q1 <= a.n_q;
    const uint32_t own = __ballot_sync(0xffffffffu, i < n_seqs && q0 / rows + i <= t);
    if (own) {
      s = i - lane + 31 - __clz(own);
      first = __shfl_sync(0xffffffffu, q0 / rows + i, 31 - __clz(own));
    }
  }
  m0 = s < 0 ? 1 << 30 : (t - first) * rows;  // before the first sequence: past its end
  return __all_sync(0xffffffffu, sound) ? max(s, 0) : -1;
}

namespace tc {

using dec::mbar_arrive;
using dec::mbar_arrive_expect_tx;
using dec::smem_u32;

constexpr int kM = 128;
// Of every 8 pairs of a row's exponentials, those that the polynomial does.  8k causal prompt, 32 heads, us for 0 / 2 / 3 / 4:
// heads of 128 491 / 461 / 502 / 507, of 64 351 / 335 / 333 / 362.
constexpr int kPoly = 2;
constexpr float kC0 = 0x1.fff692p-1f, kC1 = 0x1.62f31ap-1f, kC2 = 0x1.f0de1ap-3f, kC3 = 0x1.c3f75ep-5f;

constexpr float kHuge = 0x1p26f;

// Heads of 128: S and O of two tiles with steps of 128 keys fill an SM's TMEM, one block has the SM to itself, and its
// softmax threads keep a row of S in registers that they take over from the last warpgroup.  The block stays: warp 10 asks
// for the work of blocks that have not begun, and while the softmax warps write one pair of tiles the next one's loads and
// Q K^T are under way (with a block for each pair 16 ragged prompts of up to 512 took 23 % longer, one of 8192 2 %).
// Heads of 64: with steps of 64 keys they fill half of it, and two blocks share an SM (shared memory lets no third in):
// four tiles whose waits overlap, as do one block's first loads and last stores with the other's steps.
template <int D>
struct Shape {
  static constexpr int kN = D;                // keys of a step
  static constexpr int kBlocks = 128 / D;     // on an SM
  static constexpr bool kStay = D == 128;     // a block takes work until there is none
  static constexpr int kColumns = 4 * D;      // of TMEM
  static constexpr int kThreads = D == 128 ? 384 : 320;
  static constexpr int kRegs = 168, kRegsSoftmax = 208, kRegsRest = 88;  // heads of 128: at launch, and handed over
  static_assert(D != 128 || 256 * kRegsSoftmax + 128 * kRegsRest <= kThreads * kRegs, "those at launch");
  static constexpr int kQ = kM * D * 2, kTile = kN * D * 2;  // bytes of a query tile, of a step's keys or values
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kSmem = 2 * kQ + kStages * kTile + 512;  // Bars behind the tiles
  static_assert(kSmem <= 227 * 1024 / kBlocks - 1024 && kSmem > 227 * 1024 / (kBlocks + 1), "blocks on an SM");
};

// What a block works on: two tiles of queries and the keys they see.
struct Item {
  int q0, k0, lq, lk, m0, head0, n[2], sound;  // n: steps of each tile; sound: the sequence's ranges are
};

struct Life {
  int dead;               // a wait has run out
  unsigned int progress;  // of rows that are computed once more
};

struct Bars {  // at most 512 bytes
  uint64_t q_full, q_empty, kv_full[8], kv_empty[8], s_full[2], p_full[2], o_full[2], item_full[2], item_empty[2], next, drained;
  Item item[2];
  uint4 answer;  // of the request for more work
  uint32_t tmem;
  Life life;
  int huge[8];  // of a softmax warp: a maximum of an item's rows was
};
constexpr int kTakers = 10;  // warps that read an item

// One lane of a converged warp.  What an MMA is issued with must be the same for the warp in the compiler's eyes too: the
// issuing warp's loops run in all lanes, over values from shuffles and votes.  Under `lane == 0`, or with loop bounds
// straight from memory, an MMA took about 145 cycles to issue; so it takes its 64.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ uint64_t now_ns() { return dec::globaltimer(); }

// Waits for a phase of an mbarrier, a second without progress at most (another warp's failure ends it too, where `life` is
// given).
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile Life* life) {
  uint64_t t0 = now_ns();
  unsigned int progress = life ? life->progress : 0;
  for (;;) {
    if (dec::mbar_try_wait(bar, parity)) return true;
    if (life && life->dead) return false;
    if (now_ns() - t0 > 1000000000ull) {
      if (!life) return false;
      if (life->progress == progress) {
        life->dead = 1;
        return false;
      }
      t0 = now_ns(), progress = life->progress;
    }
  }
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Life* life) {
  for (int i = 0; i < 16; ++i)
    if (dec::mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, life);
}
// The same for a whole warp, whose lanes stay together.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Life* life) {
  for (int i = 0; i < 16; ++i)
    if (__all_sync(0xffffffffu, dec::mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_slow(bar, parity, life));
}

// More work: the number of a block of this launch that has not begun and now never will, in place of which this block
// does its work; none left: -1.  The answer arrives in shared memory.
__device__ __forceinline__ void ask(uint4* answer, uint64_t* bar) {
  mbar_arrive_expect_tx(bar, 16);
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ int answer_of(const uint4* answer) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tselp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? (int)x : -1;
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
      : "memory");
}

// Operand in rows of 128 bytes under the 128-byte swizzle; `group` = bytes between groups of 8 rows, `slab` = bytes
// between slabs of 64 elements (used where the 64 elements run along N: V).
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t slab) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((slab >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// D[tmem] (+)= A[tmem] B
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 values in a register pair.
using F2 = uint64_t;
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 un2(F2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// (2^x, 2^y) without the special function unit: x = n + f with n the nearest integer (adding 1.5 * 2^23 leaves n in
// the low bits), 2^f on +-1/2 by the cubic of least relative error (7.5e-5, a 50th of P's rounding to bf16), and n
// added to the exponent.  Below 2^-126 the result stays there.  A NaN gives a number above bf16's range.
__device__ __forceinline__ F2 exp2_poly(F2 v) {
  const float2 u = un2(v);
  const F2 x = f2(max_nan(u.x, -126.f), max_nan(u.y, -126.f));
  const F2 t = add2(x, f2(12582912.f, 12582912.f));
  const F2 f = fma2(add2(t, f2(-12582912.f, -12582912.f)), f2(-1.f, -1.f), x);
  F2 p = fma2(f, f2(kC3, kC3), f2(kC2, kC2));
  p = fma2(p, f, f2(kC1, kC1));
  p = fma2(p, f, f2(kC0, kC0));
  const float2 a = un2(t), b = un2(p);
  return f2(__int_as_float(__float_as_int(b.x) + (__float_as_int(a.x) << 23)),
            __int_as_float(__float_as_int(b.y) + (__float_as_int(a.y) << 23)));
}

// One row over the `n` keys it sees, on a warp: lanes take keys for the scores and dims for the values.
template <int D>
__device__ __forceinline__ void redo_row(const PrefillArgs& a, Life* life, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                         const __nv_bfloat16* v, __nv_bfloat16* out, int n) {
  constexpr int kD = D / 32;
  using Values = std::conditional_t<D == 128, uint2, uint32_t>;  // a lane's dims
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f, o[kD] = {};
  for (int t0 = 0; t0 < n; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY;
    if (t < n) {
      s = 0.f;
#pragma unroll 1
      for (int d = 0; d < D; d += 32) {
        Vec8<__nv_bfloat16> x[4], y[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) y[c].load(k + t * a.ks + d + 8 * c), x[c].load(q + d + 8 * c);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float u[8], w[8];
          x[c].get(u);
          y[c].get(w);
#pragma unroll
          for (int i = 0; i < 8; ++i) s = fmaf(u[i], w[i], s);
        }
      }
      s *= a.scale_log2;
    }
    const float mn = fmaxf(m, warp_max(s)), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m - base);
    const float p = t < n ? exp2f(s - base) : 0.f;
    l = l * f + warp_sum(p);
#pragma unroll
    for (int i = 0; i < kD; ++i) o[i] *= f;
#pragma unroll 1
    for (int j0 = 0; j0 < 32 && t0 + j0 < n; j0 += 8) {
      Values x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (t0 + j0 + j < n) x[j] = *reinterpret_cast<const Values*>(v + (t0 + j0 + j) * a.vs + lane * kD);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float pj = __shfl_sync(0xffffffffu, p, j0 + j);
        if (t0 + j0 + j < n) {
          const __nv_bfloat16* y = reinterpret_cast<const __nv_bfloat16*>(&x[j]);
#pragma unroll
          for (int i = 0; i < kD; ++i) o[i] = fmaf(pj, __bfloat162float(y[i]), o[i]);
        }
      }
    }
    m = mn;
    if (lane == 0) atomicAdd(&life->progress, 1u);
  }
#pragma unroll
  for (int i = 0; i < kD; ++i) out[lane * kD + i] = __float2bfloat16_rn(o[i] / l);
}

// Which of eight values are not finite.
__device__ __forceinline__ uint32_t not_finite(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r |= (w[i] & 0x7F80u) == 0x7F80u ? 1u << 2 * i : 0u;
    r |= (w[i] & 0x7F800000u) == 0x7F800000u ? 2u << 2 * i : 0u;
  }
  return r;
}

// Results of a warp's rows (lane's row: `end` keys are seen) that are not finite, in the rows of `rows`: they stand where the
// row sees a value in that dim that is not finite either; else the row is computed once more (`all`: in any case).  q and
// out: the first lane's row.
template <int D>
__device__ __forceinline__ void mend_rows(const PrefillArgs& a, Life* life, uint32_t rows, bool all, int end, const __nv_bfloat16* q,
                                          const __nv_bfloat16* k, const __nv_bfloat16* v, __nv_bfloat16* out) {
  constexpr int kLanes = D / 8, kKeys = 32 / kLanes, kAhead = 8;  // of a key; keys of a load; loads under way
  const int lane = threadIdx.x & 31, dim = lane % kLanes * 8, sub = lane / kLanes;
  const int top = __shfl_sync(0xffffffffu, end, 31 - __clz(rows));  // (later rows see no fewer)
  uint32_t open = 0;  // dims in question for which no such value is found yet
  for (uint32_t left = all ? 0 : rows; left; left &= left - 1)
    open |= not_finite(*reinterpret_cast<const uint4*>(out + (__ffs(left) - 1) * a.os + dim));
  int first[8];  // the first key with such a value
#pragma unroll
  for (int i = 0; i < 8; ++i) first[i] = 0x7FFFFFFF;
  for (int t0 = 0; t0 < top && __any_sync(0xffffffffu, open != 0); t0 += kKeys * kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = t0 + u * kKeys + sub;
      x[u] = t < top ? *reinterpret_cast<const uint4*>(v + t * a.vs + dim) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const uint32_t found = not_finite(x[u]) & open;
      if (found) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (found >> i & 1) first[i] = t0 + u * kKeys + sub;
        open &= ~found;
      }
    }
#pragma unroll
    for (int w = kLanes; w < 32; w <<= 1) open &= __shfl_xor_sync(0xffffffffu, open, w);
    if (lane == 0) atomicAdd(&life->progress, 1u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int w = kLanes; w < 32; w <<= 1) first[i] = min(first[i], __shfl_xor_sync(0xffffffffu, first[i], w));
  for (uint32_t left = rows; left; left &= left - 1) {
    const int r = __ffs(left) - 1, n = __shfl_sync(0xffffffffu, end, r);
    const uint32_t bad = not_finite(*reinterpret_cast<const uint4*>(out + r * a.os + dim));
    bool again = all;
#pragma unroll
    for (int i = 0; i < 8; ++i) again |= (bad >> i & 1) && first[i] >= n;
    if (__any_sync(0xffffffffu, again)) redo_row<D>(a, life, q + r * a.qs, k, v, out + r * a.os, n);
  }
}

template <int D, bool kPacked>
__global__ void __launch_bounds__(Shape<D>::kThreads, Shape<D>::kBlocks)
    prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const PrefillArgs a, const int n_seqs, const int tiles,
                   const int pair) {
  using Sh = Shape<D>;
  using bf16 = __nv_bfloat16;
  constexpr int kN = Sh::kN, kSlabs = D / 64, kRow = 128, kSlabQ = kM * kRow, kSlab = kN * kRow;  // slabs of 64 elements: rows of 128 bytes
  constexpr uint32_t kIdS = dec::umma_idesc_bf16(kM, kN, false), kIdO = dec::umma_idesc_bf16(kM, D, true);
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars& b = *reinterpret_cast<Bars*>(sm + 2 * Sh::kQ + Sh::kStages * Sh::kTile);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int columns = pair ? a.heads / 2 : a.heads, mstep = pair ? 0 : kM;
  // Work `at` of the launch.  pair: the tiles are heads 2x and 2x + 1; else queries m0 and m0 + 128.  Late queries, with
  // most keys, first.  false: the sequence ends before it.
  auto item_at = [&](int at, Item& w) {
    const int s = tile_at<kPacked>(a, n_seqs, tiles, pair ? kM : 2 * kM, at / columns, w.m0);
    if (kPacked && s < 0) {
      if (lane == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
      return false;
    }
    const Range r = range_of(a, s);
    w.q0 = (int)r.q0, w.k0 = (int)r.k0, w.lq = r.lq, w.lk = r.lk, w.sound = r.ok;
    w.head0 = (pair ? 2 : 1) * (at % columns);
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // steps of a tile, up to the last key its last row sees
      const int mi = w.m0 + i * mstep;
      const int keys = !r.ok || mi >= r.lq ? 0 : a.causal ? min(r.lk, min(mi + kM, r.lq) + r.lk - r.lq) : r.lk;
      w.n[i] = keys > 0 ? (keys + kN - 1) / kN : 0;
    }
    if (!r.ok && lane == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
    return w.m0 < r.lq;
  };
  Item only;  // where a block has one
  if (!Sh::kStay && !item_at(blockIdx.x, only)) return;

  uint8_t* ring = sm + 2 * Sh::kQ;
  if (tid == 0) {
    dec::mbar_init(&b.q_full, 1);
    dec::mbar_init(&b.q_empty, 1);
    for (int i = 0; i < Sh::kStages; ++i) dec::mbar_init(&b.kv_full[i], 1), dec::mbar_init(&b.kv_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      dec::mbar_init(&b.s_full[i], 1);
      dec::mbar_init(&b.p_full[i], kM);
      dec::mbar_init(&b.o_full[i], 1);
      dec::mbar_init(&b.item_full[i], 1);
      dec::mbar_init(&b.item_empty[i], kTakers);
    }
    dec::mbar_init(&b.next, 1);
    dec::mbar_init(&b.drained, 1);
    b.life.dead = 0, b.life.progress = 0;
    for (int i = 0; i < 8; ++i) b.huge[i] = 0;
    dec::fence_mbar_init();
  }
  if (warp == 8) {
    dec::tmem_alloc(&b.tmem, Sh::kColumns);
    dec::tmem_relinquish();
  }
  dec::tc_fence_before();
  __syncthreads();
  dec::tc_fence_after();
  const uint32_t tm = Sh::kColumns == 512 ? 0 : __shfl_sync(0xffffffffu, b.tmem, 0);  // (all columns begin at 0)
  auto tS = [&](int i) { return tm + i * kN; };
  auto tO = [&](int i) { return tm + 2 * kN + i * D; };
  bool ok = true;
  // The round-th item; the caller's warp has done with it at leave().  false: there is none.
  auto take = [&](uint32_t round, Item& w) {
    if (!Sh::kStay) {
      w = only;
      return round == 0;
    }
    ok = ok && wait_warp(&b.item_full[round & 1], round >> 1 & 1, &b.life);
    if (!ok) return false;
    w = b.item[round & 1];
    return w.m0 >= 0;
  };
  auto leave = [&](uint32_t round) {
    __syncwarp();
    if (Sh::kStay && lane == 0) mbar_arrive(&b.item_empty[round & 1]);
  };

  if (warp < 8) {
    if (Sh::kStay) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Sh::kRegsSoftmax));
    // ---- softmax of tile i, one row a thread
    const int i = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const float sl = a.scale_log2;
    uint32_t step = 0, written = 0;  // of all items: the barriers' phases
    for (uint32_t round = 0;; ++round) {
      int n, end, warp_end;  // steps, keys the row sees, and the fewest in the warp
      {
        Item w;
        if (!take(round, w)) break;
        n = i ? w.n[1] : w.n[0];
        end = !w.sound ? 0 : a.causal ? min(w.lk, w.m0 + i * mstep + (tid & 127) + w.lk - w.lq + 1) : w.lk;
        warp_end = __shfl_sync(0xffffffffu, end, 0);
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j, ++step) {
        ok = wait_warp(&b.s_full[i], step & 1, &b.life);
        if (!ok) break;
        dec::tc_fence_after();
        uint32_t x[kN / 32][32];
#pragma unroll
        for (int c = 0; c < kN / 32; ++c) dec::tmem_ld32(tS(i) + lanes + c * 32, x[c]);
        dec::tmem_wait_ld();
        const bool masked = j * kN + kN > warp_end;
        if (masked) {
          const int lim = end - j * kN;
#pragma unroll
          for (int e = 0; e < kN; ++e)
            if (e >= lim) x[e / 32][e % 32] = 0xFF800000u;
        }
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kN; e += 2)
          mx4[e / 2 % 4] =
              fmaxf(mx4[e / 2 % 4], fmaxf(__uint_as_float(x[e / 32][e % 32]), __uint_as_float(x[e / 32][e % 32 + 1])));
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        const bool grow = (mx - m) * sl > 8.f || (m == -INFINITY && mx > m);
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? mx : m;
          const float f = grow ? dec::ex2_approx((m - mn) * sl) : 1.f;
          l *= f;
          m = mn;
          if (grow && fabsf(m) * sl >= kHuge && m < INFINITY) b.huge[warp] = 1;
          if (j > 0) {
            // S(j) was issued behind P V of the step before: O is at rest until this step's P
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {  // few at a time: the scores are in registers
              uint32_t o[16];
              tmem_ld16(tO(i) + lanes + c, o);
              dec::tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(tO(i) + lanes + c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m * sl;
        const F2 sl2 = f2(sl, sl), base2 = f2(-base, -base);
        F2 sum[2] = {f2(0.f, 0.f), f2(0.f, 0.f)};
        auto weights = [&](auto poly) {
#pragma unroll
          for (int c = 0; c < kN / 32; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              F2 y = fma2(f2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), sl2, base2);
              if (e % 8 < decltype(poly)::value) {
                y = exp2_poly(y);
              } else {
                const float2 u = un2(y);
                y = f2(dec::ex2_approx(u.x), dec::ex2_approx(u.y));
              }
              sum[e & 1] = add2(sum[e & 1], y);
              const float2 u = un2(y);
              const __nv_bfloat162 h = __floats2bfloat162_rn(u.x, u.y);
              p[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            tmem_st16(tS(i) + lanes + c * 16, p);
          }
        };
        if (masked)  // an unseen key's weight is exactly zero
          weights(std::integral_constant<int, 0>());
        else
          weights(std::integral_constant<int, kPoly>());
        const float2 sums = un2(add2(sum[0], sum[1]));
        l += sums.x + sums.y;
        tmem_wait_st();
        dec::tc_fence_before();
        mbar_arrive(&b.p_full[i]);
      }
      if (!ok) break;
      // ---- results
      if (n > 0) {
        ok = wait_warp(&b.o_full[i], written++ & 1, &b.life);
        if (!ok) break;
        dec::tc_fence_after();
      }
      Item w;  // read again: the loop above needs the registers
      if (Sh::kStay) w = b.item[round & 1]; else w = only;
      leave(round);
      const int row = w.m0 + i * mstep + (tid & 127), head = w.head0 + (pair ? i : 0);
      const bool live = row < w.lq;
      __syncwarp();
      const bool huge = *static_cast<volatile int*>(&b.huge[warp]);
      // No softmax, hence NaN: every score is -infinity (the maximum tells; the polynomial gives such a score 2^-126), or
      // one is +infinity or NaN (the sum of sound weights is below 2^12 a key; the polynomial gives a NaN 2^127)
      const bool none = end <= 0, lost = fabsf(m) == INFINITY || (!huge && !(l > 0.f && l < 1e30f));
      const float inv = lost ? NAN : 1.f / l;
      bf16* op = static_cast<bf16*>(a.out) + ((int64_t)w.q0 + row) * a.os + (int64_t)head * D;
      bool bad = false;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (n > 0) {
          dec::tmem_ld32(tO(i) + lanes + c * 32, o);
          dec::tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[k] = none ? 0.f : __uint_as_float(o[e + k]) * inv;
            bad |= !(fabsf(y[k]) <= 3.38953139e38f);  // bf16's largest: not finite, or rounding to infinity
          }
          if (live) Vec8<bf16>::store(op + c * 32 + e, y);
        }
      }
      dec::tc_fence_before();  // O is read: the next item's first P lets it be written
      const uint32_t again = __ballot_sync(0xffffffffu, (bad || huge) && live && !none && !lost);
      if (huge && lane == 0) b.huge[warp] = 0;
      if (again) {
        __syncwarp();  // the rows' first results are written
        const int64_t r0 = (int64_t)w.q0 + w.m0 + i * mstep + (tid & 96);  // the first lane's row
        mend_rows<D>(a, &b.life, again, huge, end, static_cast<const bf16*>(a.q) + r0 * a.qs + (int64_t)head * D,
                     static_cast<const bf16*>(a.k) + (int64_t)w.k0 * a.ks + (int64_t)(head / a.gs) * D,
                     static_cast<const bf16*>(a.v) + (int64_t)w.k0 * a.vs + (int64_t)(head / a.gs) * D,
                     static_cast<bf16*>(a.out) + r0 * a.os + (int64_t)head * D);
      }
    }
    if (!ok && lane == 0) flag(a.status, DEC_SEQ_TIMEOUT);
    dec::tc_fence_before();
  } else {
    if (Sh::kStay) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Sh::kRegsRest));
    if (warp == 9) {
      // ---- loads: an item's Q, then its K0 V0 K1 V1 ... round the ring
      int issued = 0, n_q = 0;
      for (uint32_t round = 0;; ++round) {
        Item w;
        if (!take(round, w)) break;
        leave(round);
        const int n_max = max(w.n[0], w.n[1]);
        if (n_max > 0 && elect()) {
          ok = n_q == 0 || wait(&b.q_empty, (n_q - 1) & 1, &b.life);
          if (ok) {
            const int tiles_q = w.n[1] > 0 ? 2 : 1;
            mbar_arrive_expect_tx(&b.q_full, tiles_q * Sh::kQ);
            for (int i = 0; i < tiles_q; ++i)
              for (int c = 0; c < kSlabs; ++c)
                tma_load(sm + i * Sh::kQ + c * kSlabQ, &q_map, c * 64, w.head0 + (pair ? i : 0), w.q0 + w.m0 + i * mstep,
                         &b.q_full);
            ++n_q;
          }
          for (int j = 0; j < 2 * n_max && ok; ++j) {
            const int slot = issued % Sh::kStages, turn = issued / Sh::kStages;
            ok = turn == 0 || wait(&b.kv_empty[slot], (turn - 1) & 1, &b.life);
            if (!ok) break;
            mbar_arrive_expect_tx(&b.kv_full[slot], Sh::kTile);
            for (int c = 0; c < kSlabs; ++c)
              tma_load(ring + slot * Sh::kTile + c * kSlab, j & 1 ? &v_map : &k_map, c * 64, w.head0 / a.gs,
                       w.k0 + (j >> 1) * kN, &b.kv_full[slot]);
            ++issued;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      if (!ok) {  // no copy may be in flight when the block ends
        if (n_q > 0) wait_slow(&b.q_full, (n_q - 1) & 1, nullptr);
        for (int x = max(0, issued - Sh::kStages); x < issued; ++x)
          wait_slow(&b.kv_full[x % Sh::kStages], (x / Sh::kStages) & 1, nullptr);
      }
    } else if (warp == 8) {
      // ---- MMAs
      const uint64_t q_desc = desc(smem_u32(sm), 16), k_desc = desc(smem_u32(ring), 16), v_desc = desc(smem_u32(ring), kSlab);
      uint32_t n_q = 0, taken = 0, step[2] = {0, 0};
      for (uint32_t round = 0;; ++round) {
        Item w;
        if (!take(round, w)) break;
        leave(round);
        const int n0 = __shfl_sync(0xffffffffu, w.n[0], 0), n1 = __shfl_sync(0xffffffffu, w.n[1], 0), n_max = max(n0, n1);
        const int lk = __shfl_sync(0xffffffffu, w.lk, 0);
        if (n_max == 0) continue;
        const int last = lk < n_max * kN ? n_max - 1 : -1;  // the step that holds the last key and others behind it
        ok = wait_warp(&b.q_full, n_q++ & 1, &b.life);
        auto full = [&](uint32_t x) {  // the x-th load's place in the ring, in units of 16 bytes
          ok = ok && wait_warp(&b.kv_full[x % Sh::kStages], (x / Sh::kStages) & 1, &b.life);
          return x % Sh::kStages * (Sh::kTile >> 4);
        };
        auto release = [&](int x) {  // the item's x-th load's slot, if it will be filled again
          if ((Sh::kStay || x + Sh::kStages < 2 * n_max) && elect()) dec::tc_commit(&b.kv_empty[(taken + x) % Sh::kStages]);
          __syncwarp();
        };
        auto q_read = [&]() {
          if (Sh::kStay && elect()) dec::tc_commit(&b.q_empty);
          __syncwarp();
        };
        auto scores = [&](int i, uint32_t kt) {
          if (elect()) {
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
              dec::tc_mma(tS(i), q_desc + ((i * Sh::kQ + (ks / 4) * kSlabQ + (ks % 4) * 32) >> 4),
                          k_desc + kt + (((ks / 4) * kSlab + (ks % 4) * 32) >> 4), kIdS, ks != 0);
            dec::tc_commit(&b.s_full[i]);
          }
          __syncwarp();
        };
        auto values = [&](int i, int j, int n, uint32_t vt) {
          if (elect()) {
#pragma unroll
            for (int ks = 0; ks < kN / 16; ++ks)
              mma_ts(tO(i), tS(i) + ks * 8, v_desc + vt + ((ks * 16 * kRow) >> 4), kIdO, ks != 0 ? 1 : j != 0);
            if (j + 1 == n) dec::tc_commit(&b.o_full[i]);
          }
          __syncwarp();
        };
        uint32_t kt = full(taken);
        if (!ok) break;
        dec::tc_fence_after();
        if (n0 > 0) scores(0, kt);
        if (n1 > 0) scores(1, kt);
        release(0);
        if (n_max == 1) q_read();
        for (int j = 0; j < n_max && ok; ++j) {
          const uint32_t vt = full(taken + 2 * j + 1);
          if (j + 1 < n_max) kt = full(taken + 2 * j + 2);
          if (j == last && ok) {
            const int keys = lk - j * kN, rows = kN - keys;
            uint8_t* to = ring + (taken + 2 * j + 1) % Sh::kStages * Sh::kTile + keys * kRow;
#pragma unroll 4
            for (int e = lane * 16; e < rows * kRow; e += 512)
#pragma unroll
              for (int c = 0; c < kSlabs; ++c) *reinterpret_cast<uint4*>(to + c * kSlab + e) = make_uint4(0, 0, 0, 0);
            dec::fence_async_smem();
            __syncwarp();
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int n = i ? n1 : n0;
            if (j >= n) continue;
            ok = ok && wait_warp(&b.p_full[i], step[i]++ & 1, &b.life);
            if (!ok) break;
            dec::tc_fence_after();
            values(i, j, n, vt);
            if (j + 1 < n) scores(i, kt);
          }
          release(2 * j + 1);
          if (j + 1 < n_max) release(2 * j + 2);
          if (j + 2 == n_max) q_read();
        }
        if (!ok) break;
        taken += 2 * n_max;
      }
      if (Sh::kStay || !ok) {  // no MMA, and no arrival of one, may be under way when the block ends
        if (elect()) dec::tc_commit(&b.drained);
        __syncwarp();
        wait_slow(&b.drained, 0, nullptr);
      }
    } else if (Sh::kStay && warp == 10) {
      // ---- work: this block's own, then that of blocks which have not begun, one ahead of the other warps
      int at = blockIdx.x;
      uint32_t round = 0, asked = 0;
      while (ok) {
        if (at >= 0 && elect()) ask(&b.answer, &b.next);
        __syncwarp();
        Item w;
        const bool some = at >= 0 && item_at(at, w);
        if (some || at < 0) {
          if (round > 1) ok = wait_warp(&b.item_empty[round & 1], (round >> 1) - 1 & 1, &b.life);
          if (at < 0) w.m0 = -1;
          if (ok && lane == 0) {
            b.item[round & 1] = w;
            mbar_arrive(&b.item_full[round & 1]);
          }
          ++round;
        }
        if (at < 0) break;
        if (!__all_sync(0xffffffffu, wait_slow(&b.next, asked++ & 1, nullptr))) {  // an answer may not be under way either
          b.life.dead = 1;
          break;
        }
        at = answer_of(&b.answer);
        dec::fence_async_smem();
        __syncwarp();
      }
    }
  }
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    dec::tc_fence_after();
    dec::tmem_dealloc(tm, Sh::kColumns);
  }
}

// A tensor of rows [rows][heads][D] in boxes of `tile` rows and 64 elements.
inline bool make_map(CUtensorMap* m, const void* base, int rows, int heads, int d, int64_t stride, int tile) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult res;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &res) != cudaSuccess) {
      (void)cudaGetLastError();
      return static_cast<Encode>(nullptr);
    }
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)(rows > 0 ? rows : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)tile}, step[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kPacked>
cudaError_t start(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const PrefillArgs& a, int n_seqs,
                  int tiles, int pair, unsigned blocks, cudaStream_t st) {
  using Sh = Shape<D>;
  cudaError_t e =
      cudaFuncSetAttribute(prefill_kernel<D, kPacked>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  if (D == 128) {
    static const int regs = [] {
      cudaFuncAttributes f;
      return cudaFuncGetAttributes(&f, prefill_kernel<D, kPacked>) == cudaSuccess ? f.numRegs : 0;
    }();
    if (regs != Sh::kRegs) return cudaErrorInvalidValue;  // the warps would wait for registers that are not there
  }
  prefill_kernel<D, kPacked><<<blocks, Sh::kThreads, Sh::kSmem, st>>>(q, k, v, a, n_seqs, tiles, pair);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch(const PrefillArgs& a, int n_seqs, cudaStream_t st) {
  using Sh = Shape<D>;
  CUtensorMap q, k, v;
  const bool keys = a.n_k > 0;  // without keys every row is zero and no load is issued
  const void *kp = keys ? a.k : a.q, *vp = keys ? a.v : a.q;
  const int rows = keys ? a.n_k : a.n_q, heads = keys ? a.heads / a.gs : a.heads;
  if (!make_map(&q, a.q, a.n_q, a.heads, D, a.qs, kM) || !make_map(&k, kp, rows, heads, D, keys ? a.ks : a.qs, Sh::kN) ||
      !make_map(&v, vp, rows, heads, D, keys ? a.vs : a.qs, Sh::kN))
    return cudaErrorInvalidValue;
  const int pair = a.gs % 2 == 0, rows_q = pair ? kM : 2 * kM;
  const Tiling tl = tiling(n_seqs, a.n_q, a.max_q, rows_q);
  const int64_t blocks = (int64_t)tl.tiles * (tl.packed ? 1 : n_seqs) * (pair ? a.heads / 2 : a.heads);
  return tl.packed ? start<D, true>(q, k, v, a, n_seqs, tl.tiles, pair, (unsigned)blocks, st)
                   : start<D, false>(q, k, v, a, n_seqs, tl.tiles, pair, (unsigned)blocks, st);
}

}  // namespace tc
}  // namespace dec_op
