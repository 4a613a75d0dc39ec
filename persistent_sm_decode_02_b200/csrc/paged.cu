// The paged 8-bit cache: what writes it (dec_kv_append) and what reads it (dec_attention_paged).
#include <cuda_fp16.h>
#include <float.h>

#include "op_common.cuh"

namespace {

using namespace dec_op;

struct Cache {
  uint8_t *k, *v;
  float *ks, *vs;
  int n_pages, ps, hkv;
};

// ------------------------------------------------------------------ append
enum { kKeysValues = 1, kQueries = 2, kBoth = 3 };  // what a launch does

struct AppendArgs {
  Cache c;
  const double* inv_freq;
  int rot, neighbour;
  float factor;
  const void *q, *k, *v;
  void* q_out;
  int64_t qs, ks, vs, qos;
  int heads, n_tokens, max_new, pieces;  // heads: of q (0: no q)
  int kv_blocks, q_blocks;               // of one (sequence, page): they share its kv heads, and its query heads, evenly
  const int32_t *cu, *lens, *table;
  int table_stride;
  int32_t* status;
};

// E of the smallest 2^E, -120 <= E <= 120, with amax <= 448 * 2^E.  448 = 1.75 * 2^8, so for amax = 1.f * 2^x
// that is x - 8, plus one where 1.f > 1.75; subnormal amax ends at the lower bound.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u);
  return min(120, max(-120, e));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return __half22float2(*reinterpret_cast<__half2*>(&r));
}

// Largest finite magnitude (an infinity or NaN leaves `m`).
__device__ __forceinline__ float amax_finite(float m, float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? fmaxf(m, a) : m;
}

// sin and cos of an angle in turns, to about half an ulp of fp32.  Quarter turns are taken off in fp64 (a far
// position makes many); on the +-pi/4 left, as a pair of floats, the Taylor series with the leading terms kept exact.
__device__ __forceinline__ void sincos_turns(double turns, float& sn, float& cs) {
  const double q = turns * 4.0, k = rint(q), x = (q - k) * 1.5707963267948966;
  const float h = (float)x, l = (float)(x - (double)h), z = h * h;
  const float ps = fmaf(fmaf(fmaf(1.f / 362880.f, z, -1.f / 5040.f), z, 1.f / 120.f), z, -1.f / 6.f);
  const float s = h + fmaf(h * z, ps, l);
  const float pc = fmaf(fmaf(fmaf(-1.f / 3628800.f, z, 1.f / 40320.f), z, -1.f / 720.f), z, 1.f / 24.f);
  const float w = fmaf(-0.5f, z, 1.f);
  // 1 - z / 2 is w + (1 - w - z / 2), and h * h is z + fma(h, h, -z)
  const float c = w + fmaf(z * z, pc, fmaf(-0.5f, z, 1.f - w) - fmaf(0.5f, fmaf(h, h, -z), h * l));
  const int quarter = (int)(long long)k & 3;
  sn = quarter & 1 ? c : s;
  cs = quarter & 1 ? s : c;
  if (quarter & 2) sn = -sn;
  if ((quarter + 1) & 2) cs = -cs;
}

// Sixteen values of one row, in the two 8-element chunks a thread holds, turned by their eight angles.
__device__ __forceinline__ void rotate16(float* x, const float* cs, const float* sn, bool neighbour) {
  if (neighbour) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * cs[i] - b * sn[i];
      x[2 * i + 1] = a * sn[i] + b * cs[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = a * cs[i] - b * sn[i];
      x[8 + i] = a * sn[i] + b * cs[i];
    }
  }
}

__device__ __forceinline__ void store_codes(uint8_t* p, const float* x, float inv) {
  uint2 o;
  o.x = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
  o.y = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
  *reinterpret_cast<uint2*>(p) = o;
}

// The block's maxima, in every thread.
__device__ __forceinline__ void block_max(float (*red)[16], float& x, float& y) {
  x = warp_max(x);
  y = warp_max(y);
  if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = x, red[1][threadIdx.x >> 5] = y;
  __syncthreads();
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    x = fmaxf(x, red[0][w]);
    y = fmaxf(y, red[1][w]);
  }
}

// Rows before the piece, rounded again for a larger scale.
__device__ __forceinline__ void rescale_rows(uint8_t* p, int bytes, float ratio, int thread, int threads) {
#pragma unroll 4
  for (int i = thread * 8; i < bytes; i += threads * 8) {
    uint2 w = *reinterpret_cast<const uint2*>(p + i);
    const float2 a = from_e4m3x2(w.x), b = from_e4m3x2(w.x >> 16), c = from_e4m3x2(w.y), d = from_e4m3x2(w.y >> 16);
    const float x[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    store_codes(p + i, x, ratio);
  }
}

// New tokens of sequence s in one page.
struct Piece {
  int64_t lo, row0;  // first position, its row of q, k and v
  int rows, slot, page;
};
__device__ __forceinline__ bool piece_of(const AppendArgs& a, int s, int piece, Piece& p) {
  const int ps = a.c.ps;
  const int64_t c0 = a.cu[s], c1 = a.cu[s + 1], n = c1 - c0, len = a.lens[s];
  if (n == 0) return false;
  if (n < 0 || c0 < 0 || c1 > a.n_tokens || n > a.max_new || len < n || len > (int64_t)a.table_stride * ps) {
    if (threadIdx.x == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
    return false;
  }
  const int64_t start = len - n, pi = start / ps + piece, hi = min(len, (pi + 1) * ps);
  p.lo = max(start, pi * ps);
  if (p.lo >= hi) return false;
  p.row0 = c0 + (p.lo - start);
  p.rows = (int)(hi - p.lo);
  p.slot = (int)(p.lo - pi * ps);
  p.page = a.table[(int64_t)s * a.table_stride + pi];
  return true;
}

// The eight angles of a thread's dims at position pos.
__device__ __forceinline__ void angles(const AppendArgs& a, int c, int64_t pos, float* sn, float* cs) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sincos_turns((double)pos * a.inv_freq[8 * c + i] * 0.15915494309189535, sn[i], cs[i]);  // 1 / (2 pi)
    sn[i] *= a.factor;
    cs[i] *= a.factor;
  }
}

// Blocks of a (sequence, page it touches): some for its kv heads, some for its query heads.  A thread holds the same 16
// dims of its rows for every head, so it computes their 8 angles once.  Bound by memory where tokens are many (4 x 8192
// tokens, 32 / 8 heads of 128, bf16: 738 MB in 138 us, 5.3 TB/s), by the chain of dependent loads (offsets, page id,
// row) where they are few (one token 3.8 us).  A page's scale needs all of its new values, so its keys and values stay in
// registers between the maximum and the rounding and are read once; the next head's are on their way meanwhile.
template <typename T, int D, int NIT, int ROLE>
__global__ void __launch_bounds__(ROLE == kQueries ? 256 : 512, ROLE == kQueries ? 3 : ROLE == kKeysValues && NIT == 1 ? 2 : 1)
    append_kernel(AppendArgs a) {
  __shared__ float red[2][2][16];
  constexpr int kUnits = D / 16;  // threads a row
  constexpr int kBatch = 4;       // query heads whose loads are under way at once
  asm volatile("griddepcontrol.launch_dependents;");
  const int blocks = (ROLE & kKeysValues ? a.kv_blocks : 0) + (ROLE & kQueries ? a.q_blocks : 0);
  const int part = blockIdx.x % blocks, piece = blockIdx.x / blocks % a.pieces, s = blockIdx.x / blocks / a.pieces;
  const int tid = threadIdx.x, ps = a.c.ps;
  Piece p;
  if (!piece_of(a, s, piece, p)) return;
  const int nr = p.rows, slot0 = p.slot, page = p.page;
  const int64_t row0 = p.row0;
  const bool neighbour = a.neighbour;

  const int c = tid % kUnits;  // blockDim.x is a multiple of kUnits
  const bool turned = c < a.rot / 16;
  const int d0 = turned && !neighbour ? 8 * c : 16 * c, d1 = turned && !neighbour ? a.rot / 2 + 8 * c : 16 * c + 8;
  const int q_part = part - (ROLE & kKeysValues ? a.kv_blocks : 0);
  if ((ROLE & kQueries) && q_part >= 0) {  // ---- query heads
    const int h0 = a.heads * q_part / a.q_blocks, h1 = a.heads * (q_part + 1) / a.q_blocks;
    for (int r = tid / kUnits; r < nr; r += blockDim.x / kUnits) {
      float cs[8], sn[8];
      if (turned) angles(a, c, p.lo + r, sn, cs);
      const T* qp = static_cast<const T*>(a.q) + (row0 + r) * a.qs;
      T* op = static_cast<T*>(a.q_out) + (row0 + r) * a.qos;
      for (int h = h0; h < h1; h += kBatch) {
        Vec8<T> x[kBatch][2];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (h + b < h1) {
            x[b][0].load(qp + (h + b) * D + d0);
            x[b][1].load(qp + (h + b) * D + d1);
          }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          if (h + b < h1) {
            float y[16];
            x[b][0].get(y);
            x[b][1].get(y + 8);
            if (turned) rotate16(y, cs, sn, neighbour);
            Vec8<T>::store(op + (h + b) * D + d0, y);
            Vec8<T>::store(op + (h + b) * D + d1, y + 8);
          }
      }
    }
    return;
  }
  if (!(ROLE & kKeysValues)) return;

  // ---- keys and values
  const bool page_ok = page >= 0 && page < a.c.n_pages;
  if (!page_ok) {
    if (tid == 0) flag(a.status, DEC_SEQ_BAD_PAGE);
    return;
  }
  const int g0 = a.c.hkv * part / a.kv_blocks, g1 = a.c.hkv * (part + 1) / a.kv_blocks;
  float cs[NIT][8], sn[NIT][8];
  int row[NIT];
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    row[it] = (tid + it * blockDim.x) / kUnits;
    if (turned && row[it] < nr) angles(a, c, p.lo + row[it], sn[it], cs[it]);
  }
  Vec8<T> kr[NIT][2], vr[NIT][2];
  auto load = [&](int head) {
#pragma unroll
    for (int it = 0; it < NIT; ++it)
      if (row[it] < nr) {
        const T* kp = static_cast<const T*>(a.k) + (row0 + row[it]) * a.ks + (int64_t)head * D;
        const T* vp = static_cast<const T*>(a.v) + (row0 + row[it]) * a.vs + (int64_t)head * D;
        kr[it][0].load(kp + d0);
        kr[it][1].load(kp + d1);
        vr[it][0].load(vp + d0);
        vr[it][1].load(vp + d1);
      }
  };
  load(g0);
  for (int head = g0; head < g1; ++head) {
    float k[NIT][16], mk = 0.f, mv = 0.f;
    Vec8<T> v[NIT][2];
#pragma unroll
    for (int it = 0; it < NIT; ++it)
      if (row[it] < nr) {
        kr[it][0].get(k[it]);
        kr[it][1].get(k[it] + 8);
        if (turned) rotate16(k[it], cs[it], sn[it], neighbour);
        float y[16];
        v[it][0] = vr[it][0];
        v[it][1] = vr[it][1];
        v[it][0].get(y);
        v[it][1].get(y + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          mk = fmaxf(mk, fabsf(k[it][i]));  // a NaN leaves the maximum as it is
          mv = fmaxf(mv, fabsf(y[i]));
        }
      }
    if (head + 1 < g1) load(head + 1);
    const int64_t si = (int64_t)page * a.c.hkv + head;
    float k_was = 0.f, v_was = 0.f;
    if (slot0 > 0) k_was = a.c.ks[si], v_was = a.c.vs[si];
    block_max(red[0], mk, mv);  // its barrier also orders every read of the old scales before their update
    if (mk == INFINITY || mv == INFINITY) {  // rare: once more without the infinities
      mk = mv = 0.f;
#pragma unroll
      for (int it = 0; it < NIT; ++it)
        if (row[it] < nr) {
          float y[16];
          v[it][0].get(y);
          v[it][1].get(y + 8);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            mk = amax_finite(mk, k[it][i]);
            mv = amax_finite(mv, y[i]);
          }
        }
      block_max(red[1], mk, mv);
    }
    const float k_now = fmaxf(k_was, pow2(scale_exponent(mk))), v_now = fmaxf(v_was, pow2(scale_exponent(mv)));
    if (tid == 0) a.c.ks[si] = k_now, a.c.vs[si] = v_now;
    uint8_t* kp = a.c.k + si * ps * D;
    uint8_t* vp = a.c.v + si * ps * D;
    if (slot0 > 0 && k_now > k_was) rescale_rows(kp, slot0 * D, k_was / k_now, tid, blockDim.x);
    if (slot0 > 0 && v_now > v_was) rescale_rows(vp, slot0 * D, v_was / v_now, tid, blockDim.x);
    const float ik = 1.f / k_now, iv = 1.f / v_now;
#pragma unroll
    for (int it = 0; it < NIT; ++it)
      if (row[it] < nr) {
        const int at = (slot0 + row[it]) * D;
        store_codes(kp + at + d0, k[it], ik);
        store_codes(kp + at + d1, k[it] + 8, ik);
        float y[16];
        v[it][0].get(y);
        v[it][1].get(y + 8);
        store_codes(vp + at + d0, y, iv);
        store_codes(vp + at + d1, y + 8, iv);
      }
    __syncthreads();  // red is used again
  }
  if (ROLE == kKeysValues) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T, int D>
cudaError_t launch_append(const AppendArgs& a, int64_t pages, int units, bool split, cudaStream_t s) {
  const int nit = units > 512 ? 2 : 1;
  const int threads = ((units + nit - 1) / nit + 31) / 32 * 32;
  if (!split) {
    const int blocks = (int)(pages * (a.kv_blocks + a.q_blocks));
    if (nit == 2)
      append_kernel<T, D, 2, kBoth><<<blocks, threads, 0, s>>>(a);
    else
      append_kernel<T, D, 1, kBoth><<<blocks, threads, 0, s>>>(a);
    return cudaGetLastError();
  }
  append_kernel<T, D, 1, kQueries><<<(int)(pages * a.q_blocks), threads < 256 ? threads : 256, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((int)(pages * a.kv_blocks));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return nit == 2 ? cudaLaunchKernelEx(&cfg, append_kernel<T, D, 2, kKeysValues>, a)
                  : cudaLaunchKernelEx(&cfg, append_kernel<T, D, 1, kKeysValues>, a);
}

// ------------------------------------------------------------------ attention
// The batch is one line of tiles: (sequence, kv head, 16 positions), sequences in order.  It is cut into equal
// contiguous pieces, one a warp, so a GPU full of warps is busy whatever the lengths are, and what a warp, a block
// and the grid leave unfinished at their two ends is joined by log-sum-exp: warps of a block in shared memory, blocks
// in a second small kernel.
//
// A warp computes S^T = K q^T (16 positions x 8 query heads) and O^T += V^T P (D x 8) with m16n8k16 fp16 MMAs.
// E4M3 codes are exact in fp16; q is scaled by a power of two into fp16's upper range, where a bf16 q is exact; the
// weights are rounded to fp16 (2^-11, well below a bf16 result's own rounding).  For fp32, q and the weights are
// pairs of fp16 (22 bits) and each product two MMAs.  Positions as M and heads as N waste nothing for a group of 8.
// An MMA's K index may be permuted freely, so a lane's four bytes of a K row are the k pairs (2t, 2t+1) and
// (2t+8, 2t+9) of one MMA, and 16-byte shared-memory reads feed it without a shuffle; V^T pairs positions, one
// byte permute a word.  The weights, in the accumulator's layout, become the second MMA's operand by movmatrix.
//
// Scales: a tile lies in one page, so K's scale multiplies its scores, and V's enters the exponent: weights are
// 2^(s + log2 vs - m'), with a running maximum m' of their own, and the sum uses 2^(s - m).  Either maximum moves
// only when a score is 2^10 above it (weights then reach 2^14, inside fp16), so most tiles need no reduction.
constexpr int kBlocks = 148;  // one block per SM of a B200
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;

struct PagedArgs {
  Cache c;
  const void* q;
  void* out;
  int64_t qs, os;
  int gs, n_seqs, lps;  // lps: log2 of the page size
  const int32_t *lens, *table;
  int table_stride;
  float scale_log2;
  float* part;  // [kBlocks][2] open ends: m[8], m'[8], l[8], O[8][D]
  int4* meta;   // [kBlocks][2] {sequence, head, ends at the sequence's end, in use}
  int32_t* status;
};

__device__ __forceinline__ int tiles_of(const PagedArgs& a, int s) {
  const int len = a.lens[s];
  return len < 0 || len > (int64_t)a.table_stride * a.c.ps ? 0 : (len >> 4) + ((len & 15) != 0);
}

// A place on the line of tiles.
struct Place {
  int s, head, tile, tiles, len;
  __device__ __forceinline__ void enter(const PagedArgs& a) {  // the first sequence from s on that has tiles
    tiles = 0;
    while (s < a.n_seqs && (tiles = tiles_of(a, s)) == 0) ++s;
    len = tiles ? a.lens[s] : 0;
  }
  __device__ __forceinline__ void next(const PagedArgs& a) {
    if (++tile == tiles) {
      tile = 0;
      if (++head == a.c.hkv) {
        head = 0;
        ++s;
        enter(a);
      }
    }
  }
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half_codes(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
__device__ __forceinline__ uint32_t pack_half(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// What rounding (x, y) to the halves in h left over.
__device__ __forceinline__ uint32_t pack_rest(float x, float y, uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_half(x - f.x, y - f.y);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

template <int D>
struct PagedShape {
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kTile = 16 * D;              // bytes of K, or V, of 16 positions
  static constexpr int kStage = 2 * kTile + 16;     // K, V, {ks, vs, rows that count}
  static constexpr int kSlot = (24 + 8 * D) * 4;    // m[8], m'[8], l[8], O[8][D]
  static constexpr int kRing = kStages * kStage;    // also holds a warp's last open end once its copies are done
  static constexpr int kSmem = kWarps * (kRing + kSlot);
  static_assert(kRing >= kSlot && kSmem <= 227 * 1024 - 8192, "shared memory");
};

// Weights of an open end in a join: 2^(m - M), nothing where the end saw no position.
__device__ __forceinline__ float join_weight(float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); }

// O / l in the units of V: O counts 2^(M' - 4), l counts 2^M.
__device__ __forceinline__ float unit(float l, float M, float Mp) {
  return l == 0.f ? 0.f : ex2(Mp - M - 4.f) / l;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(PagedArgs a) {
  using Sh = PagedShape<D>;
  constexpr bool kPair = sizeof(T) == 4;
  constexpr int kSteps = D / 16;            // MMA k steps of S, and M tiles of O
  constexpr int kRow = D / 64;              // 16-byte chunks of a K row a lane reads
  constexpr int kPer = Sh::kTile / 512;     // 16-byte copies a lane issues for K, and for V
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ long long before[kThreads];
  __shared__ long long warp_sum_s[kWarps];
  __shared__ int4 open_meta[kWarps][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- where this warp's piece of the line is
  const int per = (a.n_seqs + kThreads - 1) / kThreads;
  long long mine = 0;
  for (int i = 0; i < per; ++i) {
    const int s = tid * per + i;
    if (s < a.n_seqs) mine += tiles_of(a, s);
  }
  long long scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += y;
  }
  if (lane == 31) warp_sum_s[warp] = scan;
  if (lane < 2) open_meta[warp][lane] = make_int4(-1, 0, 0, 0);
  __syncthreads();
  long long total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) scan += total;
    total += warp_sum_s[w];
  }
  before[tid] = scan - mine;
  __syncthreads();
  const int gw = blockIdx.x * kWarps + warp;
  for (int s = gw; s < a.n_seqs; s += kBlocks * kWarps) {  // sequences without positions
    if (tiles_of(a, s) == 0) {
      if (lane == 0 && a.lens[s] != 0) flag(a.status, DEC_SEQ_BAD_RANGE);
      for (int e = lane * 8; e < a.gs * a.c.hkv * D; e += 256) {
        const float z[8] = {};
        Vec8<T>::store(static_cast<T*>(a.out) + s * a.os + e, z);
      }
    }
  }
  total *= a.c.hkv;
  const long long begin = total * gw / (kBlocks * kWarps), end = total * (gw + 1) / (kBlocks * kWarps);
  int left = (int)(end - begin);
  Place get;
  if (left > 0) {
    int lo = 0, hi = kThreads - 1;  // the last thread whose sequences begin at or before `begin`
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before[mid] * a.c.hkv <= begin) lo = mid; else hi = mid - 1;
    }
    long long at = before[lo] * a.c.hkv;
    get.s = lo * per;
    get.enter(a);
    while (get.s < a.n_seqs && at + (long long)get.tiles * a.c.hkv <= begin) {
      at += (long long)get.tiles * a.c.hkv;
      ++get.s;
      get.enter(a);
    }
    if (get.s < a.n_seqs) {
      get.head = (int)((begin - at) / get.tiles);
      get.tile = (int)((begin - at) % get.tiles);
    } else {
      left = 0;  // the lengths changed under the call
    }
  }
  Place use = get;

  // ---- ring of copies in flight
  uint8_t* ring = sm + warp * Sh::kRing;
  float* slot = reinterpret_cast<float*>(sm + kWarps * Sh::kRing + warp * Sh::kSlot);
  const uint32_t ring_a = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  int to_get = left, get_stage = 0, page = 0;
  auto look_up = [&]() {
    page = to_get > 0 ? a.table[(int64_t)get.s * a.table_stride + ((get.tile << 4) >> a.lps)] : 0;
  };
  auto fetch = [&]() {
    if (to_get > 0) {
      const uint32_t st = ring_a + get_stage * Sh::kStage;
      const bool ok = page >= 0 && page < a.c.n_pages;
      const int rows = ok ? min(16, get.len - (get.tile << 4)) : 0;
      const int64_t si = ok ? (int64_t)page * a.c.hkv + get.head : 0;
      const int64_t at = ((si << a.lps) + ((get.tile << 4) & (a.c.ps - 1))) * D;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int idx = lane + 32 * i, r = idx / (D / 16), ch = idx % (D / 16);
        const int kx = D == 128 ? (r & 1) << 2 : 0, vx = D == 128 ? r & 6 : r & 2;
        const bool live = r < rows;
        const int64_t off = live ? at + idx * 16 : 0;
        copy16(st + r * D + ((ch ^ kx) << 4), a.c.k + off, live);
        copy16(st + Sh::kTile + r * D + ((ch ^ vx) << 4), a.c.v + off, live);
      }
      if (lane == 0) {
        copy4(st + 2 * Sh::kTile, a.c.ks + si);
        copy4(st + 2 * Sh::kTile + 4, a.c.vs + si);
        *reinterpret_cast<int*>(ring + get_stage * Sh::kStage + 2 * Sh::kTile + 8) = rows;
        if (!ok) flag(a.status, DEC_SEQ_BAD_PAGE);
      }
      --to_get;
      get_stage = get_stage + 1 == Sh::kStages ? 0 : get_stage + 1;
      if (to_get > 0) get.next(a);
      if (get.s >= a.n_seqs) to_get = 0;
      look_up();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  look_up();
  for (int i = 0; i < Sh::kStages - 1; ++i) fetch();

  // ---- one (sequence, kv head) after another
  int stage = 0;
  while (left > 0) {
    uint32_t qh[kSteps][2], ql[kPair ? kSteps : 1][2];
    float f0, f1;  // score factors of this lane's two heads, 2t and 2t + 1
    {
      const T* qp = static_cast<const T*>(a.q) + use.s * a.qs + ((int64_t)use.head * a.gs + g) * D;
      float x[kRow][16], mx = 0.f;
#pragma unroll
      for (int c = 0; c < kRow; ++c) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[c][i] = 0.f;
        if (g < a.gs) {
          Vec8<T> w;
          w.load(qp + 64 * c + 16 * t);
          w.get(x[c]);
          w.load(qp + 64 * c + 16 * t + 8);
          w.get(x[c] + 8);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = amax_finite(mx, x[c][i]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // largest magnitude to [2^14, 2^15)
      const int e = max(-110, (int)(__float_as_uint(mx) >> 23) - 127);
      const float up = pow2(14 - e);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const float* y = x[j / 4] + 4 * (j % 4);
        qh[j][0] = pack_half(y[0] * up, y[1] * up);
        qh[j][1] = pack_half(y[2] * up, y[3] * up);
        if (kPair) {
          ql[j][0] = pack_rest(y[0] * up, y[1] * up, qh[j][0]);
          ql[j][1] = pack_rest(y[2] * up, y[3] * up, qh[j][1]);
        }
      }
      const float f = pow2(e - 14) * a.scale_log2;
      f0 = __shfl_sync(0xffffffffu, f, 8 * t);
      f1 = __shfl_sync(0xffffffffu, f, 8 * t + 4);
    }
    const int s = use.s, head = use.head, tile0 = use.tile, tiles = use.tiles;
    float o[kSteps][4] = {}, m0 = -INFINITY, m1 = -INFINITY, n0 = -INFINITY, n1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    int count = min(left, tiles - tile0);
    const bool whole_end = tile0 + count == tiles;
    left -= count;
    for (; count > 0; --count) {
      asm volatile("cp.async.wait_group %0;" ::"n"(Sh::kStages - 2) : "memory");
      __syncwarp();
      fetch();  // into the stage read in the round before
      const uint8_t* st = ring + stage * Sh::kStage;
      stage = stage + 1 == Sh::kStages ? 0 : stage + 1;
      const float ks = *reinterpret_cast<const float*>(st + 2 * Sh::kTile);
      const float vs = *reinterpret_cast<const float*>(st + 2 * Sh::kTile + 4);
      const int rows = *reinterpret_cast<const int*>(st + 2 * Sh::kTile + 8);
      float c[2][4] = {};
#pragma unroll
      for (int r = 0; r < kRow; ++r) {
        const int ch = (4 * r + t) ^ (D == 128 ? (g & 1) << 2 : 0);
        const uint4 u = *reinterpret_cast<const uint4*>(st + g * D + ch * 16);
        const uint4 w = *reinterpret_cast<const uint4*>(st + (g + 8) * D + ch * 16);
        const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = half_codes(x[j]), a1 = half_codes(y[j]), a2 = half_codes(x[j] >> 16),
                         a3 = half_codes(y[j] >> 16);
          mma16816(c[j & 1], a0, a1, a2, a3, qh[4 * r + j][0], qh[4 * r + j][1]);
          if (kPair) mma16816(c[j & 1], a0, a1, a2, a3, ql[4 * r + j][0], ql[4 * r + j][1]);
        }
      }
      const float k0 = f0 * ks, k1 = f1 * ks, lv = __log2f(vs);
      const bool in0 = g < rows, in1 = g + 8 < rows;
      const float s0 = (c[0][0] + c[1][0]) * k0, s1 = (c[0][1] + c[1][1]) * k1;
      const float s2 = (c[0][2] + c[1][2]) * k0, s3 = (c[0][3] + c[1][3]) * k1;
      const float x0 = fmaxf(in0 ? s0 : -INFINITY, in1 ? s2 : -INFINITY);
      const float x1 = fmaxf(in0 ? s1 : -INFINITY, in1 ? s3 : -INFINITY);
      if (__any_sync(0xffffffffu, x0 > m0 + 10.f || x0 + lv > n0 + 10.f || x1 > m1 + 10.f || x1 + lv > n1 + 10.f)) {
        float y0 = x0, y1 = x1;
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, w));
          y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, w));
        }
        const float a0 = fmaxf(m0, y0), a1 = fmaxf(m1, y1), b0 = fmaxf(n0, y0 + lv), b1 = fmaxf(n1, y1 + lv);
        l0 *= join_weight(m0, a0);
        l1 *= join_weight(m1, a1);
        const float w0 = join_weight(n0, b0), w1 = join_weight(n1, b1);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) o[i][0] *= w0, o[i][1] *= w1, o[i][2] *= w0, o[i][3] *= w1;
        m0 = a0, m1 = a1, n0 = b0, n1 = b1;
      }
      const float b0 = lv + 4.f - (n0 == -INFINITY ? 0.f : n0), b1 = lv + 4.f - (n1 == -INFINITY ? 0.f : n1);
      const float p0 = in0 ? ex2(s0 + b0) : 0.f, p1 = in0 ? ex2(s1 + b1) : 0.f;
      const float p2 = in1 ? ex2(s2 + b0) : 0.f, p3 = in1 ? ex2(s3 + b1) : 0.f;
      l0 += (in0 ? ex2(s0 - m0) : 0.f) + (in1 ? ex2(s2 - m0) : 0.f);
      l1 += (in0 ? ex2(s1 - m1) : 0.f) + (in1 ? ex2(s3 - m1) : 0.f);
      const uint32_t h0 = pack_half(p0, p1), h1 = pack_half(p2, p3);
      const uint32_t ph0 = transpose8x8(h0), ph1 = transpose8x8(h1);
      uint32_t pl0 = 0, pl1 = 0;
      if (kPair) pl0 = transpose8x8(pack_rest(p0, p1, h0)), pl1 = transpose8x8(pack_rest(p2, p3, h1));
      // V: this lane's D / 8 dims of positions 2t, 2t + 1, 2t + 8, 2t + 9
      uint32_t v[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * t + (i & 1) + (i >> 1) * 8;
        if (D == 128) {
          const uint4 u = *reinterpret_cast<const uint4*>(st + Sh::kTile + r * D + ((g ^ (r & 6)) << 4));
          v[i][0] = u.x, v[i][1] = u.y, v[i][D / 32 - 2] = u.z, v[i][D / 32 - 1] = u.w;
        } else {
          const uint2 u =
              *reinterpret_cast<const uint2*>(st + Sh::kTile + r * D + (((g >> 1) ^ (r & 2)) << 4) + (g & 1) * 8);
          v[i][0] = u.x, v[i][1] = u.y;
        }
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const uint32_t sel = i & 1 ? 0x7362 : 0x5140;  // bytes 0, 1 or 2, 3 of both positions, paired
        const uint32_t u = __byte_perm(v[0][i / 2], v[1][i / 2], sel), w = __byte_perm(v[2][i / 2], v[3][i / 2], sel);
        const uint32_t a0 = half_codes(u), a1 = half_codes(u >> 16), a2 = half_codes(w), a3 = half_codes(w >> 16);
        mma16816(o[i], a0, a1, a2, a3, ph0, ph1);
        if (kPair) mma16816(o[i], a0, a1, a2, a3, pl0, pl1);
      }
    }
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, w);
      l1 += __shfl_xor_sync(0xffffffffu, l1, w);
    }
    if (tile0 == 0 && whole_end) {  // all of it: the result
      const float u0 = unit(l0, m0, n0), u1 = unit(l1, m1, n1);
      T* op = static_cast<T*>(a.out) + s * a.os + ((int64_t)head * a.gs + 2 * t) * D + g * (D / 8);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        float y0[8], y1[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y0[2 * i] = o[4 * c + i][0] * u0, y0[2 * i + 1] = o[4 * c + i][2] * u0;
          y1[2 * i] = o[4 * c + i][1] * u1, y1[2 * i + 1] = o[4 * c + i][3] * u1;
        }
        if (2 * t < a.gs) Vec8<T>::store(op + 8 * c, y0);
        if (2 * t + 1 < a.gs) Vec8<T>::store(op + D + 8 * c, y1);
      }
    } else {  // an open end: the first in this warp's slot, the last in its ring, which has nothing in flight then
      const int which = tile0 == 0 && !whole_end;
      float* to = slot;
      if (which) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        to = reinterpret_cast<float*>(ring);
      }
      if (lane == 0) open_meta[warp][which] = make_int4(s, head, (tile0 == 0) | (whole_end ? 2 : 0), 1);
      if (g == 0) {
        to[2 * t] = m0, to[2 * t + 1] = m1, to[8 + 2 * t] = n0, to[8 + 2 * t + 1] = n1;
        to[16 + 2 * t] = l0, to[16 + 2 * t + 1] = l1;
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int d = g * (D / 8) + 2 * i;
        *reinterpret_cast<float2*>(to + 24 + (2 * t) * D + d) = make_float2(o[i][0], o[i][2]);
        *reinterpret_cast<float2*>(to + 24 + (2 * t + 1) * D + d) = make_float2(o[i][1], o[i][3]);
      }
    }
    // on to the next (sequence, head); `use` is at this one's first tile here
    use.tile = tiles - 1;
    if (left > 0) use.next(a);
    if (use.s >= a.n_seqs) left = 0;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // ---- join what the warps left open; what stays open goes to the second kernel
  int4* meta = a.meta + 2 * blockIdx.x;
  bool used[2] = {false, false};
  for (int i = 0; i < 2 * kWarps;) {
    const int4 mi = open_meta[i >> 1][i & 1];
    if (!mi.w) {
      ++i;
      continue;
    }
    int j = i, flags = mi.z;
    bool closed = flags & 2;
    int n = i + 1;
    for (; n < 2 * kWarps && !closed; ++n) {
      const int4 mn = open_meta[n >> 1][n & 1];
      if (!mn.w) continue;
      if (mn.x != mi.x || mn.y != mi.y) break;
      closed = mn.z & 2;
    }
    const bool whole = (flags & 1) && closed;
    const int which = flags & 1;
    float* part = a.part + (size_t)(2 * blockIdx.x + which) * (24 + 8 * D);
    for (int e = tid; e < 8 * (D / 4); e += kThreads) {
      const int h = e / (D / 4), d = e % (D / 4) * 4;
      float M = -INFINITY, Mp = -INFINITY;
      for (int k = j; k < n; ++k)
        if (open_meta[k >> 1][k & 1].w) {
          const float* p = k & 1 ? reinterpret_cast<float*>(sm + (k >> 1) * Sh::kRing)
                                 : reinterpret_cast<float*>(sm + kWarps * Sh::kRing + (k >> 1) * Sh::kSlot);
          M = fmaxf(M, p[h]);
          Mp = fmaxf(Mp, p[8 + h]);
        }
      float l = 0.f, x[4] = {};
      for (int k = j; k < n; ++k)
        if (open_meta[k >> 1][k & 1].w) {
          const float* p = k & 1 ? reinterpret_cast<float*>(sm + (k >> 1) * Sh::kRing)
                                 : reinterpret_cast<float*>(sm + kWarps * Sh::kRing + (k >> 1) * Sh::kSlot);
          l = fmaf(p[16 + h], join_weight(p[h], M), l);
          const float w = join_weight(p[8 + h], Mp);
          const float4 y = *reinterpret_cast<const float4*>(p + 24 + h * D + d);
          x[0] = fmaf(y.x, w, x[0]), x[1] = fmaf(y.y, w, x[1]), x[2] = fmaf(y.z, w, x[2]), x[3] = fmaf(y.w, w, x[3]);
        }
      if (whole) {
        if (h < a.gs) {
          const float u = unit(l, M, Mp);
          T* op = static_cast<T*>(a.out) + mi.x * a.os + ((int64_t)mi.y * a.gs + h) * D + d;
          for (int k = 0; k < 4; ++k) op[k] = (T)(x[k] * u);
        }
      } else {
        if (d == 0) part[h] = M, part[8 + h] = Mp, part[16 + h] = l;
        *reinterpret_cast<float4*>(part + 24 + h * D + d) = make_float4(x[0], x[1], x[2], x[3]);
      }
    }
    if (!whole) {
      used[which] = true;
      if (tid == 0) meta[which] = make_int4(mi.x, mi.y, closed, 1);
    }
    i = n;
  }
  if (tid < 2 && !used[tid]) meta[tid] = make_int4(-1, 0, 0, 0);
}

// Block b joins the (sequence, head) that begins in block b of the first kernel and goes on behind it: its slot 1
// and the slots 0 of the blocks that follow, up to the one that ends it.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_join(PagedArgs a) {
  __shared__ int last_s, used_s[kBlocks];
  __shared__ float M_s[8], Mp_s[8], u_s[8];
  const int tid = threadIdx.x, b = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 me = a.meta[2 * b + 1];
  if (!me.w) return;
  if (tid == 0) last_s = kBlocks - 1;
  __syncthreads();
  if (tid >= b && tid < kBlocks) {
    const int4 m = tid == b ? me : a.meta[2 * tid];
    used_s[tid] = m.w;
    if (m.w && m.z) atomicMin(&last_s, tid);  // the first end behind b is ours
  }
  __syncthreads();
  const int last = last_s;
  auto part = [&](int i) { return a.part + (size_t)(i == b ? 2 * b + 1 : 2 * i) * (24 + 8 * D); };
  const int warp = tid >> 5, lane = tid & 31;
  {  // warp h: head h's maxima and sum
    float M = -INFINITY, Mp = -INFINITY, l = 0.f;
    for (int i = b + lane; i <= last; i += 32)
      if (used_s[i]) M = fmaxf(M, part(i)[warp]), Mp = fmaxf(Mp, part(i)[8 + warp]);
    M = warp_max(M), Mp = warp_max(Mp);
    for (int i = b + lane; i <= last; i += 32)
      if (used_s[i]) l = fmaf(part(i)[16 + warp], join_weight(part(i)[warp], M), l);
    l = warp_sum(l);
    if (lane == 0) Mp_s[warp] = Mp, u_s[warp] = unit(l, M, Mp);
  }
  __syncthreads();
  for (int e = tid; e < a.gs * (D / 4); e += 256) {
    const int h = e / (D / 4), d = e % (D / 4) * 4;
    const float Mp = Mp_s[h];
    float x[4] = {};
#pragma unroll 4
    for (int i = b; i <= last; ++i) {
      if (!used_s[i]) continue;
      const float w = join_weight(part(i)[8 + h], Mp);
      const float4 y = *reinterpret_cast<const float4*>(part(i) + 24 + h * D + d);
      x[0] = fmaf(y.x, w, x[0]), x[1] = fmaf(y.y, w, x[1]), x[2] = fmaf(y.z, w, x[2]), x[3] = fmaf(y.w, w, x[3]);
    }
    T* op = static_cast<T*>(a.out) + me.x * a.os + ((int64_t)me.y * a.gs + h) * D + d;
    for (int j = 0; j < 4; ++j) op[j] = (T)(x[j] * u_s[h]);
  }
}

template <typename T, int D>
cudaError_t launch_paged(const PagedArgs& a, cudaStream_t s) {
  using Sh = PagedShape<D>;
  cudaError_t e =
      cudaFuncSetAttribute(paged_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  paged_kernel<T, D><<<kBlocks, kThreads, Sh::kSmem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kBlocks);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at;  // the join's blocks wait on the GPU for the first kernel's end, not in the queue
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_join<T, D>, a);
}

int check_cache(const dec_paged_cache* c) {
  if (!c || !c->k_pages || !c->v_pages || !c->k_scales || !c->v_scales) return DEC_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->page_size < 1) return DEC_ERR_INVALID_ARG;
  if (!aligned16(c->k_pages) || !aligned16(c->v_pages) || !aligned4(c->k_scales) || !aligned4(c->v_scales))
    return DEC_ERR_INVALID_ARG;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return DEC_ERR_UNSUPPORTED;
  return DEC_OK;
}

Cache device_cache(const dec_paged_cache* c) {
  return Cache{static_cast<uint8_t*>(c->k_pages), static_cast<uint8_t*>(c->v_pages), c->k_scales, c->v_scales,
               c->n_pages, c->page_size, c->n_kv_heads};
}

bool cache_on_device(const dec_paged_cache* c, int dev) {
  return on_device(c->k_pages, dev) && on_device(c->v_pages, dev) && on_device(c->k_scales, dev) &&
         on_device(c->v_scales, dev);
}

}  // namespace

extern "C" int dec_kv_append(const dec_paged_cache* cache, const dec_rope* rope, int32_t dtype, const void* q,
                             const void* k, const void* v, void* q_out, int64_t q_stride, int64_t k_stride,
                             int64_t v_stride, int64_t q_out_stride, int32_t n_heads, int32_t n_seqs,
                             int32_t n_tokens, int32_t max_new, const int32_t* cu_new, const int32_t* seq_lens,
                             const int32_t* page_table, int32_t table_stride, int32_t* status, void* stream) {
  int rc = check_cache(cache);
  if (rc) return rc;
  if (!rope || (dtype != DEC_BF16 && dtype != DEC_F32)) return DEC_ERR_INVALID_ARG;
  const int hkv = cache->n_kv_heads, D = cache->head_dim, esz = dtype == DEC_BF16 ? 2 : 4;
  rc = head_layout(q ? n_heads : hkv, hkv, D);
  if (rc) return rc;
  if (rope->rot_dim < 0 || rope->rot_dim > D || (rope->pairs != DEC_ROPE_HALF && rope->pairs != DEC_ROPE_NEIGHBOUR))
    return DEC_ERR_INVALID_ARG;
  if (rope->rot_dim % 16) return DEC_ERR_UNSUPPORTED;
  if (rope->rot_dim && (!rope->inv_freq || (reinterpret_cast<uintptr_t>(rope->inv_freq) & 7) || !isfinite(rope->factor)))
    return DEC_ERR_INVALID_ARG;
  if (n_seqs < 0 || n_tokens < 0 || max_new < 0 || table_stride < 0 || !q != !q_out) return DEC_ERR_INVALID_ARG;
  if (n_seqs == 0 || n_tokens == 0 || max_new == 0) return DEC_OK;
  if (!k || !v || !cu_new || !seq_lens || !page_table) return DEC_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v) || !aligned4(cu_new) || !aligned4(seq_lens) || !aligned4(page_table) ||
      !aligned4(status))
    return DEC_ERR_INVALID_ARG;
  if (!stride_ok(k_stride, (int64_t)hkv * D, esz) || !stride_ok(v_stride, (int64_t)hkv * D, esz))
    return DEC_ERR_INVALID_ARG;
  if (q && (!aligned16(q) || !aligned16(q_out) || !stride_ok(q_stride, (int64_t)n_heads * D, esz) ||
            !stride_ok(q_out_stride, (int64_t)n_heads * D, esz)))
    return DEC_ERR_INVALID_ARG;
  if (cudaPeekAtLastError() != cudaSuccess) return DEC_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DEC_ERR_CUDA;
  if (!cache_on_device(cache, dev) || !on_device(k, dev) || !on_device(v, dev) || !on_device(cu_new, dev) ||
      !on_device(seq_lens, dev) || !on_device(page_table, dev) || (q && (!on_device(q, dev) || !on_device(q_out, dev))) ||
      (rope->rot_dim && !on_device(rope->inv_freq, dev)) || (status && !on_device(status, dev)))
    return DEC_ERR_INVALID_ARG;

  const int ps = cache->page_size;
  if (max_new > n_tokens) max_new = n_tokens;  // no valid sequence has more
  const int64_t pieces = ((int64_t)max_new + ps - 2) / ps + 1, pages = n_seqs * pieces;
  const int units = (max_new < ps ? max_new : ps) * (D / 16);
  AppendArgs a{device_cache(cache), rope->inv_freq, rope->rot_dim, rope->pairs == DEC_ROPE_NEIGHBOUR, rope->factor, q, k,
               v, q_out, q_stride, k_stride, v_stride, q_out_stride, q ? n_heads : 0, n_tokens, max_new, (int)pieces,
               hkv, q ? hkv : 0, cu_new, seq_lens, page_table, table_stride, status};
  // A block a kv head, and one for its query heads, is the shortest path for few tokens; more blocks than fill the GPU
  // compute the angles over and over.  With blocks that a page fills (256 threads or more) twice the SMs are enough
  // and queries and keys are launches of their own, each with the registers it needs; with little in each, 8 an SM.  B200,
  // 32 / 8 heads of 128, us, one way and the other: 256 single tokens 7.1 (8 an SM) / 9.9 (2), 8 x 1000 tokens 50.3 / 41.6,
  // 4 x 8192 154 (one launch) / 138 (two), 64 x 4 tokens 5.0 / 9.8.
  const bool split = q && units >= 256;
  const int64_t enough = split ? 2 * 148 : 8 * 148;
  while (a.kv_blocks > 1 && pages * a.kv_blocks > enough) a.kv_blocks = (a.kv_blocks + 1) / 2;
  while (a.q_blocks > 1 && pages * a.q_blocks > enough) a.q_blocks = (a.q_blocks + 1) / 2;
  const int64_t blocks = pages * (a.kv_blocks + a.q_blocks);
  if (pages > INT32_MAX || blocks > INT32_MAX) return DEC_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DEC_BF16)
    e = D == 64 ? launch_append<__nv_bfloat16, 64>(a, pages, units, split, st)
                : launch_append<__nv_bfloat16, 128>(a, pages, units, split, st);
  else
    e = D == 64 ? launch_append<float, 64>(a, pages, units, split, st)
                : launch_append<float, 128>(a, pages, units, split, st);
  return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA;
}

extern "C" int dec_attention_paged_workspace(const dec_paged_cache* cache, int32_t n_seqs, int32_t n_heads,
                                             size_t* out_bytes) {
  if (!out_bytes || n_seqs < 0) return DEC_ERR_INVALID_ARG;
  int rc = check_cache(cache);
  if (rc) return rc;
  rc = head_layout(n_heads, cache->n_kv_heads, cache->head_dim);
  if (rc) return rc;
  *out_bytes = kBlocks * 2 * (sizeof(int4) + (24 + 8 * (size_t)cache->head_dim) * sizeof(float));
  return DEC_OK;
}

extern "C" int dec_attention_paged(const dec_paged_cache* cache, int32_t dtype, const void* q, void* out,
                                   int64_t q_stride, int64_t out_stride, int32_t n_heads, int32_t n_seqs,
                                   const int32_t* seq_lens, const int32_t* page_table, int32_t table_stride,
                                   float scale, void* workspace, size_t workspace_bytes, int32_t* status,
                                   void* stream) {
  size_t need = 0;
  int rc = dec_attention_paged_workspace(cache, n_seqs, n_heads, &need);
  if (rc) return rc;
  if ((dtype != DEC_BF16 && dtype != DEC_F32) || !(scale > 0.f) || !isfinite(scale) || table_stride < 0)
    return DEC_ERR_INVALID_ARG;
  if (n_seqs == 0) return DEC_OK;
  const int hkv = cache->n_kv_heads, D = cache->head_dim, esz = dtype == DEC_BF16 ? 2 : 4;
  if (!q || !out || !seq_lens || !page_table || !workspace || workspace_bytes < need) return DEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || !aligned4(seq_lens) || !aligned4(page_table) ||
      !aligned4(status) || !stride_ok(q_stride, (int64_t)n_heads * D, esz) ||
      !stride_ok(out_stride, (int64_t)n_heads * D, esz))
    return DEC_ERR_INVALID_ARG;
  if (cudaPeekAtLastError() != cudaSuccess) return DEC_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DEC_ERR_CUDA;
  if (!cache_on_device(cache, dev) || !on_device(q, dev) || !on_device(out, dev) || !on_device(workspace, dev) ||
      !on_device(seq_lens, dev) || !on_device(page_table, dev) || (status && !on_device(status, dev)))
    return DEC_ERR_INVALID_ARG;
  const size_t meta = kBlocks * 2 * sizeof(int4);
  PagedArgs a{device_cache(cache), q, out, q_stride, out_stride, n_heads / hkv, n_seqs, 31 - __builtin_clz(cache->page_size),
              seq_lens, page_table, table_stride, scale * 1.4426950408889634f,
              reinterpret_cast<float*>(static_cast<char*>(workspace) + meta), static_cast<int4*>(workspace), status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DEC_BF16)
    e = D == 64 ? launch_paged<__nv_bfloat16, 64>(a, st) : launch_paged<__nv_bfloat16, 128>(a, st);
  else
    e = D == 64 ? launch_paged<float, 64>(a, st) : launch_paged<float, 128>(a, st);
  return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA;
}
