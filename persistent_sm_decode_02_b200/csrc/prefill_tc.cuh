// Attention of packed bf16 prompts on tcgen05 tensor cores.
//
// A block takes 256 queries of one head as two tiles of 128, and walks their keys 128 at a time:
//   S = Q K^T (128 x 128, fp32 in TMEM), P = 2^(scale log2(e) S - m) rounded to bf16 over S, O += P V.
// Warps 0-3 and 4-7 are the tiles' softmax, a thread a row; warp 8 issues every MMA; warp 9 every TMA load.  The softmax
// keeps a row of S in registers: it takes them over from the last warpgroup (208 and 88 of the 168 at launch).
// The tiles alternate: while one tile's softmax runs, the tensor cores do the other's P V and next Q K^T.
//   TMEM: S0 | S1 (128 columns each, P in their first 64) | O0 | O1 (D columns each)
//   shared memory: Q, and a ring of K and V tiles, rows of 128 bytes in the 128-byte swizzle
// One thread's MMAs complete in the order they were issued.  So S_i(j + 1), issued behind P V_i(j), may overwrite P_i(j),
// and once it has arrived O_i is at rest until the tile's next P: a softmax thread may rescale its row of O there, with
// no other barrier.  It does only when the row's maximum has grown by more than 2^8 (P up to 2^8 and its sum lose nothing).
//
// P is rounded to bf16 (2^-9 of each weight, of the same size as V's own rounding and the result's); its sum is
// of the unrounded weights, in fp32.
//
// An unseen value meets a weight of zero, and zero times NaN or infinity is NaN.  Such values are rare and rows that have
// met one show it, so it is looked for only in the results: a row that is not finite is computed once more with the keys
// it sees alone (redo_row).
#pragma once
#include <cuda.h>

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

namespace tc {

using dec::mbar_arrive;
using dec::mbar_arrive_expect_tx;
using dec::smem_u32;

constexpr int kThreads = 384, kRegs = 168, kRegsSoftmax = 208, kRegsRest = 88;
static_assert(256 * kRegsSoftmax + 128 * kRegsRest <= kThreads * kRegs, "registers handed over are those at launch");
constexpr int kM = 128, kN = 128;

template <int D>
struct Shape {
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kTile = 128 * D * 2;  // bytes of 128 rows
  static constexpr int kSmem = (2 + kStages) * kTile + 1024;  // more than half an SM's: one block, and its 512 TMEM columns, per SM
};

struct Bars {
  uint64_t q_full, kv_full[8], kv_empty[8], s_full[2], p_full[2], o_full[2], drained;
  uint32_t tmem;
  int dead;
};

__device__ __forceinline__ uint64_t now_ns() { return dec::globaltimer(); }

// Waits for a phase of an mbarrier, a second at most (another warp's failure ends it too, where `dead` is given).
__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* dead) {
  const uint64_t t0 = now_ns();
  for (;;) {
    if (dec::mbar_try_wait(bar, parity)) return true;
    if (dead && *dead) return false;
    if (now_ns() - t0 > 1000000000ull) {
      if (dead) *dead = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* dead) {
  for (int i = 0; i < 16; ++i)
    if (dec::mbar_try_wait(bar, parity)) return true;
  return wait_slow(bar, parity, dead);
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One row over the `n` keys it sees, on a warp: lanes take keys for the scores and dims for the values.
template <int D>
__device__ __forceinline__ void redo_row(const PrefillArgs& a, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                      const __nv_bfloat16* v, __nv_bfloat16* out, int n) {
  constexpr int kD = D / 32;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f, o[kD] = {};
  for (int t0 = 0; t0 < n; t0 += 32) {
    const int t = t0 + lane;
    float s = -INFINITY;
    if (t < n) {
      s = 0.f;
      for (int d = 0; d < D; d += 8) {
        Vec8<__nv_bfloat16> x, y;
        float u[8], w[8];
        x.load(q + d);
        y.load(k + t * a.ks + d);
        x.get(u);
        y.get(w);
        for (int i = 0; i < 8; ++i) s = fmaf(u[i], w[i], s);
      }
      s *= a.scale_log2;
    }
    const float mn = fmaxf(m, warp_max(s)), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m - base);
    const float p = t < n ? exp2f(s - base) : 0.f;
    l = l * f + warp_sum(p);
    for (int i = 0; i < kD; ++i) o[i] *= f;
    for (int j = 0; j < 32 && t0 + j < n; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      for (int i = 0; i < kD; ++i) o[i] = fmaf(pj, __bfloat162float(v[(t0 + j) * a.vs + lane * kD + i]), o[i]);
    }
    m = mn;
  }
  for (int i = 0; i < kD; ++i) out[lane * kD + i] = __float2bfloat16_rn(o[i] / l);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const PrefillArgs a, const int n_seqs) {
  using Sh = Shape<D>;
  using bf16 = __nv_bfloat16;
  constexpr int kSlabs = D / 64, kSlab = 128 * 128;
  constexpr uint32_t kIdS = dec::umma_idesc_bf16(kM, kN, false), kIdO = dec::umma_idesc_bf16(kM, D, true);
  extern __shared__ uint8_t raw[];
  __shared__ Bars b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int head = blockIdx.x % a.heads, s = blockIdx.x / a.heads % n_seqs;
  const int tile = gridDim.x / a.heads / n_seqs - 1 - blockIdx.x / a.heads / n_seqs;  // long rows first
  const Range r = range_of(a, s);
  if (!r.ok && tid == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
  const int m0 = tile * 2 * kM, kvh = head / a.gs, shift = r.lk - r.lq;
  if (m0 >= r.lq) return;
  // 128-key steps of each tile, up to the last key its last row sees
  int n[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int mi = m0 + i * kM;
    const int keys = !r.ok || mi >= r.lq ? 0 : a.causal ? min(r.lk, min(mi + kM, r.lq) + shift) : r.lk;
    n[i] = keys > 0 ? (keys + kN - 1) / kN : 0;
  }
  const int n_max = max(n[0], n[1]);

  uint8_t* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
  if (tid == 0) {
    dec::mbar_init(&b.q_full, 1);
    for (int i = 0; i < Sh::kStages; ++i) dec::mbar_init(&b.kv_full[i], 1), dec::mbar_init(&b.kv_empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      dec::mbar_init(&b.s_full[i], 1);
      dec::mbar_init(&b.p_full[i], kM);
      dec::mbar_init(&b.o_full[i], 1);
    }
    dec::mbar_init(&b.drained, 1);
    b.dead = 0;
    dec::fence_mbar_init();
  }
  if (warp == 8) {
    dec::tmem_alloc(&b.tmem, 512);
    dec::tmem_relinquish();
  }
  dec::tc_fence_before();
  __syncthreads();
  dec::tc_fence_after();
  const uint32_t tm = b.tmem;
  const uint32_t tS[2] = {tm, tm + kN}, tO[2] = {tm + 2 * kN, tm + 2 * kN + D};

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---- softmax of tile i, row m0 + 128 i + (tid & 127)
    const int i = warp >> 2, row = m0 + i * kM + (tid & 127);
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 TMEM lanes
    const int end = !r.ok ? 0 : a.causal ? min(r.lk, row + shift + 1) : r.lk;  // keys the row sees
    const int warp_end = __shfl_sync(0xffffffffu, end, 0);  // the fewest in the warp
    const float sl = a.scale_log2;
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n[i] && ok; ++j) {
      ok = __all_sync(0xffffffffu, wait(&b.s_full[i], j & 1, &b.dead));
      if (!ok) break;
      dec::tc_fence_after();
      uint32_t x[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) dec::tmem_ld32(tS[i] + lanes + c * 32, x[c]);
      dec::tmem_wait_ld();
      float mx = -INFINITY;
      if (j * kN + kN > warp_end) {
        const int lim = end - j * kN;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (c * 32 + e >= lim) x[c][e] = 0xFF800000u;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1])));
      const bool grow = (mx - m) * sl > 8.f || (m == -INFINITY && mx > m);
      if (__any_sync(0xffffffffu, grow)) {
        const float mn = grow ? mx : m;
        const float f = grow ? dec::ex2_approx((m - mn) * sl) : 1.f;
        l *= f;
        m = mn;
        if (j > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            dec::tmem_ld32(tO[i] + lanes + c * 32, o);
            dec::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(tO[i] + lanes + c * 32, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m * sl;
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float p0 = dec::ex2_approx(fmaf(__uint_as_float(x[2 * c + e / 16][2 * (e % 16)]), sl, -base));
          const float p1 = dec::ex2_approx(fmaf(__uint_as_float(x[2 * c + e / 16][2 * (e % 16) + 1]), sl, -base));
          sum0 += p0;
          sum1 += p1;
          const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
          p[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        tmem_st32(tS[i] + lanes + c * 32, p);
      }
      l += sum0 + sum1;
      tmem_wait_st();
      dec::tc_fence_before();
      mbar_arrive(&b.p_full[i]);
    }
    // ---- results
    if (ok && n[i] > 0) {
      ok = __all_sync(0xffffffffu, wait(&b.o_full[i], 0, &b.dead));
      dec::tc_fence_after();
    }
    const bool live = row < r.lq;
    const float inv = l != 0.f ? 1.f / l : 0.f;
    bf16* op = static_cast<bf16*>(a.out) + (r.q0 + row) * a.os + (int64_t)head * D;
    bool bad = false;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      if (ok && n[i] > 0) {
        dec::tmem_ld32(tO[i] + lanes + c * 32, o);
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
          y[k] = l != 0.f ? __uint_as_float(o[e + k]) * inv : 0.f;
          bad |= !(fabsf(y[k]) <= 3.38953139e38f);  // bf16's largest: not finite, or rounding to infinity
        }
        if (live) Vec8<bf16>::store(op + c * 32 + e, y);
      }
    }
    uint32_t again = __ballot_sync(0xffffffffu, bad && live && end > 0 && ok);
    while (again) {
      const int w = __ffs(again) - 1;
      again &= again - 1;
      const int64_t rw = __shfl_sync(0xffffffffu, row, w);
      __syncwarp();  // the row's first result is written
      redo_row<D>(a, static_cast<const bf16*>(a.q) + (r.q0 + rw) * a.qs + (int64_t)head * D,
                  static_cast<const bf16*>(a.k) + r.k0 * a.ks + (int64_t)kvh * D,
                  static_cast<const bf16*>(a.v) + r.k0 * a.vs + (int64_t)kvh * D,
                  static_cast<bf16*>(a.out) + (r.q0 + rw) * a.os + (int64_t)head * D, __shfl_sync(0xffffffffu, end, w));
    }
    if (!ok && lane == 0) flag(a.status, DEC_SEQ_TIMEOUT);
    dec::tc_fence_before();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
    if (warp == 9) {
      // ---- loads: Q once, then K0 V0 K1 V1 ... round the ring
      if (lane == 0 && n_max > 0) {
        const int tiles_q = n[1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(&b.q_full, tiles_q * Sh::kTile);
        for (int i = 0; i < tiles_q; ++i)
          for (int c = 0; c < kSlabs; ++c)
            tma_load(sm + i * Sh::kTile + c * kSlab, &q_map, c * 64, head, (int)r.q0 + m0 + i * kM, &b.q_full);
        int slot = 0, issued = 0;
        uint32_t round = 0;
        for (int j = 0; j < 2 * n_max; ++j) {
          if (round > 0 && !wait(&b.kv_empty[slot], (round - 1) & 1, &b.dead)) break;
          mbar_arrive_expect_tx(&b.kv_full[slot], Sh::kTile);
          uint8_t* dst = sm + (2 + slot) * Sh::kTile;
          for (int c = 0; c < kSlabs; ++c)
            tma_load(dst + c * kSlab, j & 1 ? &v_map : &k_map, c * 64, kvh, (int)r.k0 + (j >> 1) * kN, &b.kv_full[slot]);
          ++issued;
          if (++slot == Sh::kStages) slot = 0, ++round;
        }
        if (b.dead) {  // no copy may be in flight when the block ends
          wait_slow(&b.q_full, 0, nullptr);
          for (int j = max(0, issued - Sh::kStages); j < issued; ++j)
            wait_slow(&b.kv_full[j % Sh::kStages], (j / Sh::kStages) & 1, nullptr);
        }
      }
    } else if (warp == 8) {
      // ---- MMAs
      if (lane == 0 && n_max > 0) {
        bool ok = wait(&b.q_full, 0, &b.dead);
        auto full = [&](int j) {
          ok = ok && wait(&b.kv_full[j % Sh::kStages], (j / Sh::kStages) & 1, &b.dead);
          return smem_u32(sm + (2 + j % Sh::kStages) * Sh::kTile);
        };
        auto scores = [&](int i, uint32_t kt) {
          const uint32_t qt = smem_u32(sm + i * Sh::kTile);
  #pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint32_t at = (ks / 4) * kSlab + (ks % 4) * 32;
            dec::tc_mma(tS[i], desc(qt + at, 16), desc(kt + at, 16), kIdS, ks != 0);
          }
          dec::tc_commit(&b.s_full[i]);
        };
        auto values = [&](int i, int j, uint32_t vt) {
  #pragma unroll
          for (int ks = 0; ks < kN / 16; ++ks)
            mma_ts(tO[i], tS[i] + ks * 8, desc(vt + ks * 16 * 128, kSlab), kIdO, j != 0 || ks != 0);
          if (j == n[i] - 1) dec::tc_commit(&b.o_full[i]);
        };
        uint32_t kt = full(0);
        dec::tc_fence_after();
        for (int i = 0; i < 2; ++i)
          if (ok && n[i] > 0) scores(i, kt);
        auto release = [&](int j) {  // the last loads' slots are not filled again
          if (ok && j + Sh::kStages < 2 * n_max) dec::tc_commit(&b.kv_empty[j % Sh::kStages]);
        };
        release(0);
        for (int j = 0; j < n_max && ok; ++j) {
          const uint32_t vt = full(2 * j + 1);
          if (j + 1 < n_max) kt = full(2 * j + 2);
          for (int i = 0; i < 2 && ok; ++i) {
            if (j >= n[i]) continue;
            ok = wait(&b.p_full[i], j & 1, &b.dead);
            if (!ok) break;
            dec::tc_fence_after();
            values(i, j, vt);
            if (j + 1 < n[i]) scores(i, kt);
          }
          release(2 * j + 1);
          release(2 * j + 2);
        }
        if (!ok) {  // nor any MMA
          dec::tc_commit(&b.drained);
          wait_slow(&b.drained, 0, nullptr);
        }
      }
    }
  }
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    dec::tc_fence_after();
    dec::tmem_dealloc(tm, 512);
  }
}

// The bytes of a tensor of rows [rows][heads][D] as 128-row, 64-element boxes.
inline bool make_map(CUtensorMap* m, const void* base, int rows, int heads, int d, int64_t stride) {
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
  const cuuint32_t box[3] = {64, 1, 128}, step[3] = {1, 1, 1};
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const PrefillArgs& a, int n_seqs, cudaStream_t st) {
  using Sh = Shape<D>;
  CUtensorMap q, k, v;
  const bool keys = a.n_k > 0;  // without keys every row is zero and no load is issued
  if (!make_map(&q, a.q, a.n_q, a.heads, D, a.qs) ||
      !make_map(&k, keys ? a.k : a.q, keys ? a.n_k : a.n_q, keys ? a.heads / a.gs : a.heads, D, keys ? a.ks : a.qs) ||
      !make_map(&v, keys ? a.v : a.q, keys ? a.n_k : a.n_q, keys ? a.heads / a.gs : a.heads, D, keys ? a.vs : a.qs))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  static const int regs = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, prefill_kernel<D>) == cudaSuccess ? f.numRegs : 0;
  }();
  if (regs != kRegs) return cudaErrorInvalidValue;  // the warps would wait for registers that are not there
  const int tiles = (a.max_q + 2 * kM - 1) / (2 * kM);
  prefill_kernel<D><<<(unsigned)((int64_t)n_seqs * tiles * a.heads), kThreads, Sh::kSmem, st>>>(q, k, v, a, n_seqs);
  return cudaGetLastError();
}

}  // namespace tc
}  // namespace dec_op
