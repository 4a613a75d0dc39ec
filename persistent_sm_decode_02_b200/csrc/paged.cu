// The paged 8-bit cache: what writes it (dec_kv_append) and what reads it (dec_attention_paged).
#include <cuda_fp16.h>
#include <float.h>

#include <random>

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
  void *q_out, *k_out;  // k_out: nullable
  int64_t qs, ks, vs, qos, kos;
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

// Whether x, which is up to two units in the last place off where nothing cancels, lies at the middle between two E4M3
// values: the scales are powers of two, so that shows in the 20 bits which a code of normal size does not keep.  (Middles
// between subnormal codes, of values below 2^-15 of the page's largest, are not looked for.)
__device__ __forceinline__ bool at_border(float x) {
  return (__float_as_uint(x) << 12) + ((2u - 0x80000u) << 12) <= (4u << 12);  // at most 2 units from 0x80000
}

// Rotated keys with a value at a border between two codes of normal size (a block of 8 heads of a page of 64 in three has
// any) are noted, a bit for a thread's 16 values, and done again at the block's end from an fp64 rotation: their codes are
// then the exact values' nearest, where fp32's last bit would decide.  Their place in k_out, which may be k, is written
// there too.  Where the angles are 0 and the factor is 1 fp32 is exact, and nothing is noted.
__device__ __forceinline__ bool exact_turn(const float* cs, const float* sn) {
  bool exact = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) exact &= sn[i] == 0.f && fabsf(cs[i]) == 1.f;
  return exact;
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
// tokens, 32 / 8 heads of 128, bf16: 738 MB in 143-148 us, 5.0-5.2 TB/s), by the chain of dependent loads (offsets, page id,
// row) where they are few (one token 4.0 us).  A page's scale needs all of its new values, so its keys and values stay in
// registers between the maximum and the rounding and are read once; the next head's are on their way meanwhile.
template <typename T, int D, int NIT, int ROLE>
__device__ __forceinline__ void append_block(const AppendArgs& a) {
  __shared__ float red[2][2][16];
  extern __shared__ uint32_t border_s[];  // [heads of the block][NIT][warps]: lanes whose key values are at a border
  constexpr int kUnits = D / 16;  // threads a row
  constexpr int kBatch = 4;       // query heads whose loads are under way at once
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
    if (!a.k_out) return;
  }
  const int g0 = a.c.hkv * part / a.kv_blocks, g1 = a.c.hkv * (part + 1) / a.kv_blocks;
  float cs[NIT][8], sn[NIT][8];
  int row[NIT];
  bool watch[NIT];
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    row[it] = (tid + it * blockDim.x) / kUnits;
    watch[it] = false;
    if (turned && row[it] < nr) {
      angles(a, c, p.lo + row[it], sn[it], cs[it]);
      watch[it] = page_ok && !exact_turn(cs[it], sn[it]);
    }
  }
  const int warps = blockDim.x >> 5, warp = tid >> 5, lane = tid & 31;
  uint32_t any = 0;
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
    for (int it = 0; it < NIT; ++it) {
      bool border = false;
      if (row[it] < nr) {
        kr[it][0].get(k[it]);
        kr[it][1].get(k[it] + 8);
        if (turned) {
          rotate16(k[it], cs[it], sn[it], neighbour);
#pragma unroll
          for (int i = 0; i < 16; ++i) border |= at_border(k[it][i]);
          border &= watch[it];
        }
        if (a.k_out && !border) {
          T* op = static_cast<T*>(a.k_out) + (row0 + row[it]) * a.kos + (int64_t)head * D;
          Vec8<T>::store(op + d0, k[it]);
          Vec8<T>::store(op + d1, k[it] + 8);
        }
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
      const uint32_t noted = __ballot_sync(0xffffffffu, border);
      if (lane == 0) border_s[((head - g0) * NIT + it) * warps + warp] = noted;
      any |= noted;
    }
    if (head + 1 < g1) load(head + 1);
    if (!page_ok) continue;
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
  if (!any) return;
  const int words = (g1 - g0) * NIT;  // of this warp
  for (int w0 = 0; w0 < words; w0 += 32) {
    const uint32_t bits = w0 + lane < words ? border_s[(w0 + lane) * warps + warp] : 0;
    for (uint32_t some = __ballot_sync(0xffffffffu, bits != 0); some; some &= some - 1) {
      const int from = __ffs(some) - 1, head = g0 + (w0 + from) / NIT, it = (w0 + from) % NIT;
      // two threads' values at a time, one a lane
      for (uint32_t left = __shfl_sync(0xffffffffu, bits, from); left;) {
        const int b0 = __ffs(left) - 1;
        left &= left - 1;
        const int b1 = left ? __ffs(left) - 1 : b0;
        left &= left - 1;
        const int t = warp * 32 + (lane < 16 ? b0 : b1) + it * blockDim.x, r = t / kUnits, u = t % kUnits;
        const int j = lane & 15, i = neighbour ? j >> 1 : j & 7;
        const bool second = neighbour ? j & 1 : j >> 3;
        const int first = neighbour ? 16 * u + 2 * i : 8 * u + i, apart = neighbour ? 1 : a.rot / 2;
        const T* kp = static_cast<const T*>(a.k) + (row0 + r) * a.ks + (int64_t)head * D + first;
        const double x = (double)(float)kp[0], y = (double)(float)kp[apart];
        const double turns = (double)(p.lo + r) * a.inv_freq[8 * u + i] * 0.15915494309189535;
        double sn64, cs64;
        sincospi(2.0 * (turns - rint(turns)), &sn64, &cs64);
        const double v = (second ? x * sn64 + y * cs64 : x * cs64 - y * sn64) * a.factor;
        const float f = __double2float_rz(v);  // rounded to odd: an inexact result has its last bit set
        const float z = (double)f != v ? __uint_as_float(__float_as_uint(f) | 1u) : f;
        const int64_t si = (int64_t)page * a.c.hkv + head;
        const int dim = first + (second ? apart : 0);
        a.c.k[(si * ps + slot0 + r) * D + dim] = (uint8_t)e4m3x2(z * (1.f / a.c.ks[si]), 0.f);
        __syncwarp();  // k is read: k_out may be k
        if (a.k_out) {
          T* op = static_cast<T*>(a.k_out) + (row0 + r) * a.kos + (int64_t)head * D + dim;
          if (sizeof(T) == 4) *op = (T)__double2float_rn(v); else *op = (T)z;
        }
      }
    }
  }
}

// Where queries and keys are launches of their own, they run side by side: the second begins once the first's blocks have
// all begun, and waits for its end at its own end, so that what follows it in the stream follows both.
template <typename T, int D, int NIT, int ROLE>
__global__ void __launch_bounds__(ROLE == kQueries ? 256 : 512, ROLE == kQueries ? 3 : ROLE == kKeysValues && NIT == 1 ? 2 : 1)
    append_kernel(AppendArgs a) {
  if (ROLE == kQueries) asm volatile("griddepcontrol.launch_dependents;");
  append_block<T, D, NIT, ROLE>(a);
  if (ROLE == kKeysValues) asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T, int D>
cudaError_t launch_append(const AppendArgs& a, int64_t pages, int units, bool split, cudaStream_t s) {
  const int nit = units > 512 ? 2 : 1;
  const int threads = ((units + nit - 1) / nit + 31) / 32 * 32;
  const int notes = (a.c.hkv + a.kv_blocks - 1) / a.kv_blocks * nit * (threads / 32) * 4;
  if (!split) {
    const int blocks = (int)(pages * (a.kv_blocks + a.q_blocks));
    if (nit == 2)
      append_kernel<T, D, 2, kBoth><<<blocks, threads, notes, s>>>(a);
    else
      append_kernel<T, D, 1, kBoth><<<blocks, threads, notes, s>>>(a);
    return cudaGetLastError();
  }
  append_kernel<T, D, 1, kQueries><<<(int)(pages * a.q_blocks), threads < 256 ? threads : 256, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((int)(pages * a.kv_blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = notes;
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
// contiguous pieces, one a warp, so a GPU full of warps is busy whatever the lengths are, and what warps and blocks
// leave unfinished at their two ends is joined by log-sum-exp: a block's warps in shared memory, and blocks by the one in
// which the (sequence, head) ends, which waits for those before it.  (They were dispatched before it and wait for none
// behind them, so it never waits for a block that has no SM.)  Sums are in the order of the line: the same bits every time.
//
// A warp computes S^T = K q^T (16 positions x 8 query heads) and O^T += V^T P (D x 8) with m16n8k16 fp16 MMAs.
// E4M3 codes are exact in fp16; q is scaled by a power of two into fp16's upper range, where a bf16 q is exact (an element
// is off by at most 2^-39 of the largest); the weights are rounded to fp16 (2^-11, well below a bf16 result's own
// rounding).  For fp32, q and the weights are pairs of fp16 and each product two MMAs; a q element has 22 bits or 2^-39 of the
// largest.  The low half of a pair of weights is held 2^12 higher and meets V 2^12 lower, which for E4M3 values is exact in
// fp16 too.  Positions as M and heads as N waste nothing for a group of 8.
// An MMA's K index may be permuted freely, so a lane's four bytes of a K row are the k pairs (2t, 2t+1) and
// (2t+8, 2t+9) of one MMA, and 16-byte shared-memory reads feed it without a shuffle; V^T pairs positions, one
// byte permute a word.  The weights, in the accumulator's layout, become the second MMA's operand by movmatrix.
//
// Scales: a tile lies in one page, so K's scale multiplies its scores, and V's enters the exponent: weights are
// 2^(s - m' + log2 vs + 13), with a running maximum m' of their own, and the sum uses 2^(s - m).  m' moves only when a
// score is 2^2 above it, so most tiles need no reduction, and weights stay below 2^15, inside fp16.  (m' is rounded up, which
// costs a weight nothing but range: for scores of 2^28, 2^16 of it.)  Down to 2^-27 of the largest they have fp16's 11 bits,
// and down to 2^-30 a pair has 20; below, one is off by at most 2^-38 of the largest, a pair by 2^-50.
// A maximum of -infinity means that no position was seen; one of the lowest finite value, that every score seen was
// -infinity (those weigh nothing beside a finite score, and alone they have no softmax).
//
// Bound by memory for large batches: 128 sequences of up to 8192, 32 / 8 heads of 128, 1.26 GB in 222-227 us, 5.5-5.7 TB/s (85 %
// of the measured copy), in a graph's calls in a row, 239 us (5.3 TB/s, 80 %) in calls among others; blocks with equal work end
// between 185 and 230 us, as the SMs' shares of the bandwidth differ.
// Every warp has three tiles' copies under way, which covers the latency without a barrier between warps.  Small calls are
// latency: 7.1 us for one sequence of 77, 16.2 us for one of 8193, of which 2-3 us find the place on the line and as much
// joins; a third of a small call's stalls are first fetches of instructions, so what runs once is kept short.
constexpr int kBlocks = 148;  // one block per SM of a B200
constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
// tiles a warp has at least before another block is taken (1, 2, 4: 77 positions 8.1, 7.0, 7.6 us; 512 12.3, 12.8, 14.3; 8193
// 16.3, 16.2, 17.2)
constexpr int kLeast = 2;

struct PagedArgs {
  Cache c;
  const void* q;
  void* out;
  int64_t qs, os;
  int gs, n_seqs, lps;  // lps: log2 of the page size
  const int32_t *lens, *table;
  int table_stride;
  float scale_log2;
  float* part;     // [kBlocks][2] open ends (0: that began before the block, 1: that begins in it): m[8], m'[8], l[8], O[8][D]
  // [kBlocks][2] `key` once part is written, and its reader clears it; gone(key) where the reader's wait ran out first, and
  // the writer clears it.  So every call leaves none of either behind, and one that was late is not taken for the next call's.
  uint64_t* ready;
  uint64_t key;    // a number of this process: uninitialised memory holds neither it nor gone of it
  uint64_t limit_ns;
  int32_t* status;
};
__device__ __forceinline__ uint64_t gone(uint64_t key) { return ~key; }

__device__ __forceinline__ int tiles_of(const PagedArgs& a, int s) {
  const int len = a.lens[s];
  return len < 0 || len > (int64_t)a.table_stride * a.c.ps ? 0 : (len >> 4) + ((len & 15) != 0);
}

// A place on the line of tiles.
struct Place {
  int s, head, tile, tiles, len;
  __device__ __forceinline__ void enter(const PagedArgs& a) {  // the first sequence from s on that has tiles
    tiles = 0;
#pragma unroll 1
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
// What rounding (x, y) to the halves in h left over, times f.
__device__ __forceinline__ uint32_t pack_rest(float x, float y, uint32_t h, float f = 1.f) {
  const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_half((x - z.x) * f, (y - z.y) * f);
}
// Two halves times 1 / kLow.
__device__ __forceinline__ uint32_t lower(uint32_t x) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x0C000C00u));  // 2^-12
  return y;
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
  static_assert(kThreads >= kBlocks, "a thread for each earlier block's part");
  static_assert(kRing >= kSlot && kSmem <= 227 * 1024 - 24 * 1024, "shared memory");
};

constexpr float kTop = 13.f;   // log2 of the weight of a score at the maximum
constexpr float kGrow = 2.f;   // how far a score may be above it: weights stay below 2^(kTop + kGrow), fp16 ends at 2^16
constexpr float kLow = 4096.f; // what a pair's low half, at most 2^(kTop + kGrow - 12), is multiplied by

// Weights of an open end in a join: 2^(m - M), nothing where the end saw no position.
__device__ __forceinline__ float join_weight(float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); }

// O / l in the units of V: O counts 2^(M' - 13), l counts 2^M.  Without a weight: 0 where no position was seen, else NaN.
__device__ __forceinline__ float unit(float l, float M, float Mp) {
  return l == 0.f ? (M == -INFINITY ? 0.f : NAN) : ex2(Mp - M - kTop) / l;
}

__device__ __forceinline__ uint64_t clock_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint64_t load_acquire(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t exchange(uint64_t* p, uint64_t v) {
  uint64_t old;
  asm volatile("atom.acq_rel.gpu.global.exch.b64 %0, [%1], %2;" : "=l"(old) : "l"(p), "l"(v) : "memory");
  return old;
}

__device__ __forceinline__ void store4(float* p, float x, float y, float z, float w) {
  *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float x, float y, float z, float w) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x, y), b = __floats2bfloat162_rn(z, w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) paged_kernel(PagedArgs a) {
  using Sh = PagedShape<D>;
  constexpr bool kPair = sizeof(T) == 4;
  constexpr int kSteps = D / 16;            // MMA k steps of S, and M tiles of O
  constexpr int kRow = D / 64;              // 16-byte chunks of a K row a lane reads
  constexpr int kPer = Sh::kTile / 512;     // 16-byte copies a lane issues for K, and for V
  extern __shared__ __align__(16) uint8_t sm[];
  __shared__ unsigned before[kThreads], warp_sum_s[kWarps];
  __shared__ int4 open_s[2 * kWarps];
  __shared__ int late_s, list_s[2 * kWarps];
  __shared__ float m_s[kBlocks + 2 * kWarps][8], mp_s[kBlocks + 2 * kWarps][8], l_s[kBlocks + 2 * kWarps][8], tot_s[3][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

  // ---- where this warp's piece of the line is
  if (lane < 2) open_s[2 * warp + lane] = make_int4(-1, -1, 0, 0);
  if (tid == 0) late_s = 0;
  const int gw = blockIdx.x * kWarps + warp;
  const int per = a.n_seqs <= 32 ? 1 : (a.n_seqs + kThreads - 1) / kThreads;  // sequences a lane, or a thread, counts
  const int s0 = (a.n_seqs <= 32 ? lane : tid) * per;
  unsigned mine = 0;  // the host has seen to it that 32 bits are enough
#pragma unroll 1
  for (int i = 0; i < per; ++i)
    if (s0 + i < a.n_seqs) mine += tiles_of(a, s0 + i);
  mine *= a.c.hkv;
  unsigned scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += y;
  }
  unsigned total = __shfl_sync(0xffffffffu, scan, 31);
  if (a.n_seqs > 32) {  // up to 32 every warp counts for itself
    if (lane == 31) warp_sum_s[warp] = scan;
    __syncthreads();
    total = 0;
#pragma unroll 1
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) scan += total;
      total += warp_sum_s[w];
    }
    before[tid] = scan - mine;
    __syncthreads();
  }
#pragma unroll 1
  for (int s = gw; s < a.n_seqs; s += kBlocks * kWarps) {  // sequences without positions
    if (tiles_of(a, s) == 0) {
      if (lane == 0 && a.lens[s] != 0) flag(a.status, DEC_SEQ_BAD_RANGE);
#pragma unroll 1
      for (int e = lane * 8; e < a.gs * a.c.hkv * D; e += 256) {
        const float z[8] = {};
        Vec8<T>::store(static_cast<T*>(a.out) + s * a.os + e, z);
      }
    }
  }
  // the first `more` warps have each + 1 tiles, the others `each`
  const unsigned blocks = min((total + kLeast * kWarps - 1) / (kLeast * kWarps), (unsigned)kBlocks);
  if (blockIdx.x >= blocks) return;
  const unsigned warps = min(blocks * kWarps, (total + kLeast - 1) / kLeast), each = total / warps, more = total - each * warps;
  const unsigned begin = gw * each + min((unsigned)gw, more);
  int left = gw < warps ? (int)(each + (gw < more)) : 0;
  Place get;
  if (left > 0) {
    unsigned at = 0;  // where the sequence begins on the line
    if (a.n_seqs <= 32) {
      get.s = __ffs(__ballot_sync(0xffffffffu, scan > begin)) - 1;
      at = __shfl_sync(0xffffffffu, scan - mine, get.s);
    } else {
      int lo = 0, hi = kThreads - 1;  // the last thread whose sequences begin at or before `begin`
#pragma unroll 1
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (before[mid] <= begin) lo = mid; else hi = mid - 1;
      }
      at = before[lo];
      get.s = lo * per;
    }
    get.enter(a);
#pragma unroll 1
    while (get.s < a.n_seqs && at + (unsigned)(get.tiles * a.c.hkv) <= begin) {
      at += get.tiles * a.c.hkv;
      ++get.s;
      get.enter(a);
    }
    if (get.s < a.n_seqs) {
      get.head = (begin - at) / (unsigned)get.tiles;
      get.tile = (begin - at) - get.head * get.tiles;
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
  // This lane's share of a (sequence, head)'s queries: head g's dims 64 c + 16 t on.  The first is under way with the copies
  // (in fp32 there are no registers to hold it).
  Vec8<T> q_raw[kRow][2];
  auto q_at = [&](int c) { return static_cast<const T*>(a.q) + use.s * a.qs + ((int64_t)use.head * a.gs + g) * D + 64 * c + 16 * t; };
  auto load_q = [&]() {
    if (g < a.gs)
#pragma unroll
      for (int c = 0; c < kRow; ++c) q_raw[c][0].load(q_at(c)), q_raw[c][1].load(q_at(c) + 8);
  };
  look_up();
  if (!kPair && left > 0) load_q();
#pragma unroll 1
  for (int i = 0; i < Sh::kStages - 1; ++i) fetch();

  // ---- one (sequence, kv head) after another
  int stage = 0;
  unsigned at_tile = begin;  // the segment's first tile on the line
  while (left > 0) {
    uint32_t qh[kSteps][2], ql[kPair ? kSteps : 1][2];
    float f0, f1;  // score factors of this lane's two heads, 2t and 2t + 1
    {
      float x[kRow][16], mx = 0.f;
#pragma unroll
      for (int c = 0; c < kRow; ++c) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[c][i] = 0.f;
        if (g < a.gs) {
          if (kPair) q_raw[c][0].load(q_at(c));
          q_raw[c][0].get(x[c]);
          if (kPair) q_raw[c][1].load(q_at(c) + 8);
          q_raw[c][1].get(x[c] + 8);
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
    const int counted = count;
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
      const float least = in0 ? -FLT_MAX : -INFINITY;
      const float x0 = fmaxf(fmaxf(in0 ? s0 : least, in1 ? s2 : least), least);
      const float x1 = fmaxf(fmaxf(in0 ? s1 : least, in1 ? s3 : least), least);
      const float grow = kGrow - lv;
      if (__any_sync(0xffffffffu, x0 > m0 + kGrow || x0 - n0 > grow || x1 > m1 + kGrow || x1 - n1 > grow)) {
        float y0 = x0, y1 = x1;
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          y0 = fmaxf(y0, __shfl_xor_sync(0xffffffffu, y0, w));
          y1 = fmaxf(y1, __shfl_xor_sync(0xffffffffu, y1, w));
        }
        const float a0 = fmaxf(m0, y0), a1 = fmaxf(m1, y1), b0 = fmaxf(n0, __fadd_ru(y0, lv)), b1 = fmaxf(n1, __fadd_ru(y1, lv));
        l0 *= join_weight(m0, a0);
        l1 *= join_weight(m1, a1);
        const float w0 = join_weight(n0, b0), w1 = join_weight(n1, b1);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) o[i][0] *= w0, o[i][1] *= w1, o[i][2] *= w0, o[i][3] *= w1;
        m0 = a0, m1 = a1, n0 = b0, n1 = b1;
      }
      // (differences of scores first: they are exact where they matter)
      const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1, top = lv + kTop;
      const float p0 = in0 ? ex2(s0 - b0 + top) : 0.f, p1 = in0 ? ex2(s1 - b1 + top) : 0.f;
      const float p2 = in1 ? ex2(s2 - b0 + top) : 0.f, p3 = in1 ? ex2(s3 - b1 + top) : 0.f;
      l0 += (in0 ? ex2(s0 - m0) : 0.f) + (in1 ? ex2(s2 - m0) : 0.f);
      l1 += (in0 ? ex2(s1 - m1) : 0.f) + (in1 ? ex2(s3 - m1) : 0.f);
      const uint32_t h0 = pack_half(p0, p1), h1 = pack_half(p2, p3);
      const uint32_t ph0 = transpose8x8(h0), ph1 = transpose8x8(h1);
      uint32_t pl0 = 0, pl1 = 0;
      if (kPair) pl0 = transpose8x8(pack_rest(p0, p1, h0, kLow)), pl1 = transpose8x8(pack_rest(p2, p3, h1, kLow));
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
        if (kPair) mma16816(o[i], lower(a0), lower(a1), lower(a2), lower(a3), pl0, pl1);
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
      if (lane == 0) {
        int first = blockIdx.x;  // the block in which this (sequence, head) begins
        if (tile0 > 0) {
          const unsigned t0 = at_tile - tile0, edge = more * (each + 1);
          first = (int)((t0 < edge ? t0 / (each + 1) : more + (t0 - edge) / each) / kWarps);
        }
        open_s[2 * warp + which] = make_int4(s, head, (tile0 == 0) | (whole_end ? 2 : 0), first);
      }
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
    at_tile += counted;
    use.tile = tiles - 1;
    if (left > 0) use.next(a);
    if (use.s >= a.n_seqs) left = 0;
    if (!kPair && left > 0) load_q();
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();

  // ---- join what the warps left open: runs of slots of one (sequence, head)
  const int4 mine_o = lane < 2 * kWarps ? open_s[lane] : make_int4(-1, -1, 0, 0);
  const uint32_t used = __ballot_sync(0xffffffffu, mine_o.x >= 0);
  const uint32_t below = used & ((1u << lane) - 1);
  const int prev = below ? 31 - __clz(below) : 0;
  const int px = __shfl_sync(0xffffffffu, mine_o.x, prev), py = __shfl_sync(0xffffffffu, mine_o.y, prev);
  const uint32_t starts = __ballot_sync(0xffffffffu, mine_o.x >= 0 && (!below || px != mine_o.x || py != mine_o.y));
  if (!starts) return;
  // lane i, where a run starts at slot i: its slots and kind
  const uint32_t later = starts & ~((2u << lane) - 1);
  const uint32_t slots = used & ~((1u << lane) - 1) & (later ? (1u << (__ffs(later) - 1)) - 1 : 0xFFFFFFFFu);
  const bool ends = __shfl_sync(0xffffffffu, mine_o.z, 31 - __clz(slots | 1)) & 2;
  const bool is_start = starts >> lane & 1, late = ends && !(mine_o.z & 1), few = !late && __popc(slots) <= 4;
  uint32_t shorts = __ballot_sync(0xffffffffu, is_start && few), longs = __ballot_sync(0xffffffffu, is_start && !few && !late),
           waiting = __ballot_sync(0xffffffffu, is_start && late);
  auto slot_at = [&](int k) {
    return k & 1 ? reinterpret_cast<const float*>(sm + (k >> 1) * Sh::kRing)
                 : reinterpret_cast<const float*>(sm + kWarps * Sh::kRing + (k >> 1) * Sh::kSlot);
  };
  constexpr int kItems = 8 * (D / 4);  // (head, four dims)
  // Short runs first, a warp each; then long ones, by all warps; last the one that waits for earlier blocks, so that what
  // a block hands on never waits for what it is handed.
  for (int run = 0; shorts | longs | waiting; ++run) {
    const bool shorter = shorts;
    uint32_t& from = shorts ? shorts : longs ? longs : waiting;
    const int i0 = __ffs(from) - 1;
    from &= from - 1;
    if (shorter && run % kWarps != warp) continue;
    {
      const uint32_t members = __shfl_sync(0xffffffffu, slots, i0);
      const int4 fst = open_s[i0];
      const bool from_start = fst.z & 1, to_end = __shfl_sync(0xffffffffu, ends, i0), waits = to_end && !from_start;
      const int first = waits ? fst.w : blockIdx.x, local = __popc(members);  // blocks first .. this one - 1 have parts of it
      float* part = a.part + (size_t)(2 * blockIdx.x + from_start) * (24 + 8 * D);
      auto put = [&](int h, int d, const float (&x)[4], float M, float Mp, float l) {
        if (to_end) {
          if (h < a.gs) {
            const float u = unit(l, M, Mp);
            T* op = static_cast<T*>(a.out) + fst.x * a.os + ((int64_t)fst.y * a.gs + h) * D + d;
            store4(op, x[0] * u, x[1] * u, x[2] * u, x[3] * u);
          }
        } else {
          if (d == 0) part[h] = M, part[8 + h] = Mp, part[16 + h] = l;
          *reinterpret_cast<float4*>(part + 24 + h * D + d) = make_float4(x[0], x[1], x[2], x[3]);
        }
      };
      if (shorter) {
        const float* at[4];  // an end that is not there weighs nothing
        int own = 0;
        uint32_t left_m = members;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          at[k] = slot_at(left_m ? __ffs(left_m) - 1 : i0);
          left_m &= left_m - 1;
          if (k == lane >> 3) own = k;
        }
        // lane (k, h): end k's weights for head h
        const float* p = own & 2 ? (own & 1 ? at[3] : at[2]) : (own & 1 ? at[1] : at[0]);
        const int hl = lane & 7;
        const bool there = own < local;
        const float m = there ? p[hl] : -INFINITY, mp = there ? p[8 + hl] : -INFINITY;
        float M = m, Mp = mp;
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) {
          M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
          Mp = fmaxf(Mp, __shfl_xor_sync(0xffffffffu, Mp, o));
        }
        const float v = join_weight(mp, Mp);
        float l = there ? p[16 + hl] * join_weight(m, M) : 0.f;
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll 2
        for (int it = 0; it < kItems / 32; ++it) {
          const int h = (lane + 32 * it) / (D / 4), d = (lane + 32 * it) % (D / 4) * 4;
          float x[4] = {};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float vk = __shfl_sync(0xffffffffu, v, 8 * k + h);
            if (k < local) {
              const float4 y = *reinterpret_cast<const float4*>(at[k] + 24 + h * D + d);
              x[0] = fmaf(y.x, vk, x[0]), x[1] = fmaf(y.y, vk, x[1]), x[2] = fmaf(y.z, vk, x[2]), x[3] = fmaf(y.w, vk, x[3]);
            }
          }
          put(h, d, x, __shfl_sync(0xffffffffu, M, h), __shfl_sync(0xffffffffu, Mp, h), __shfl_sync(0xffffffffu, l, h));
        }
        __syncwarp();
      } else {
        const int remote = blockIdx.x - first, n = remote + local;
        auto remote_at = [&](int k) { return a.part + (size_t)(2 * (first + k) + (k == 0)) * (24 + 8 * D); };
        bool came = true;
        if (tid < remote) {  // the earlier blocks' parts have to be there
          uint64_t* r = a.ready + 2 * (first + tid) + (tid == 0);
          const uint64_t t0 = clock_ns();
          while (load_acquire(r) != a.key)
            if (clock_ns() - t0 > a.limit_ns) {
              came = exchange(r, gone(a.key)) == a.key;
              if (!came) late_s = 1;
              break;
            }
        }
        if (warp == 0 && members >> lane & 1) list_s[__popc(members & ((1u << lane) - 1))] = lane;
        __syncthreads();
        for (int e = tid; e < n * 8; e += kThreads) {
          const int k = e >> 3, h = e & 7;
          const float* p = k < remote ? remote_at(k) : slot_at(list_s[k - remote]);
          m_s[k][h] = p[h], mp_s[k][h] = p[8 + h], l_s[k][h] = p[16 + h];
        }
        __syncthreads();
        if (warp < 8) {  // a head's maxima, sum and weights
          const int h = warp;
          float M = -INFINITY, Mp = -INFINITY, l = 0.f;
          for (int k = lane; k < n; k += 32) M = fmaxf(M, m_s[k][h]), Mp = fmaxf(Mp, mp_s[k][h]);
          M = warp_max(M), Mp = warp_max(Mp);
          for (int k = lane; k < n; k += 32) {
            l = fmaf(l_s[k][h], join_weight(m_s[k][h], M), l);
            mp_s[k][h] = join_weight(mp_s[k][h], Mp);
          }
          l = warp_sum(l);
          if (lane == 0) tot_s[0][h] = M, tot_s[1][h] = Mp, tot_s[2][h] = l;
        }
        __syncthreads();
        for (int e = tid; e < kItems; e += kThreads) {
          const int h = e / (D / 4), d = e % (D / 4) * 4;
          float x[4] = {};
#pragma unroll 8
          for (int k = 0; k < remote; ++k) {
            const float4 y = __ldcg(reinterpret_cast<const float4*>(remote_at(k) + 24 + h * D + d));
            const float v = mp_s[k][h];
            x[0] = fmaf(y.x, v, x[0]), x[1] = fmaf(y.y, v, x[1]), x[2] = fmaf(y.z, v, x[2]), x[3] = fmaf(y.w, v, x[3]);
          }
#pragma unroll 2
          for (int k = 0; k < local; ++k) {
            const float4 y = *reinterpret_cast<const float4*>(slot_at(list_s[k]) + 24 + h * D + d);
            const float v = mp_s[remote + k][h];
            x[0] = fmaf(y.x, v, x[0]), x[1] = fmaf(y.y, v, x[1]), x[2] = fmaf(y.z, v, x[2]), x[3] = fmaf(y.w, v, x[3]);
          }
          put(h, d, x, tot_s[0][h], tot_s[1][h], tot_s[2][h]);
        }
        __syncthreads();
        if (tid < remote && came) a.ready[2 * (first + tid) + (tid == 0)] = 0;  // read: for the next call
        if (tid == 0 && late_s) flag(a.status, DEC_SEQ_TIMEOUT);
      }
      if (!to_end && (shorter ? lane == 0 : tid == 0)) {
        uint64_t* r = a.ready + 2 * blockIdx.x + from_start;
        if (exchange(r, a.key) == gone(a.key)) *r = 0;  // behind the barrier above, hence every thread's part
      }
    }
  }
}

template <typename T, int D>
cudaError_t launch_paged(const PagedArgs& a, cudaStream_t s) {
  using Sh = PagedShape<D>;
  cudaError_t e =
      cudaFuncSetAttribute(paged_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
  if (e != cudaSuccess) return e;
  paged_kernel<T, D><<<kBlocks, kThreads, Sh::kSmem, s>>>(a);
  return cudaGetLastError();
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
                             const void* k, const void* v, void* q_out, void* k_out, int64_t q_stride,
                             int64_t k_stride, int64_t v_stride, int64_t q_out_stride, int64_t k_out_stride,
                             int32_t n_heads, int32_t n_seqs, int32_t n_tokens, int32_t max_new, const int32_t* cu_new, const int32_t* seq_lens,
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
  if (k_out && (!aligned16(k_out) || !stride_ok(k_out_stride, (int64_t)hkv * D, esz))) return DEC_ERR_INVALID_ARG;
  const int ps = cache->page_size;
  if (max_new > n_tokens) max_new = n_tokens;  // no valid sequence has more
  const int64_t pieces = ((int64_t)max_new + ps - 2) / ps + 1, pages = n_seqs * pieces;
  if (pages * 2 * hkv > INT32_MAX) return DEC_ERR_UNSUPPORTED;
  if (cudaPeekAtLastError() != cudaSuccess) return DEC_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DEC_ERR_CUDA;
  if (!cache_on_device(cache, dev) || !on_device(k, dev) || !on_device(v, dev) || !on_device(cu_new, dev) ||
      !on_device(seq_lens, dev) || !on_device(page_table, dev) || (q && (!on_device(q, dev) || !on_device(q_out, dev))) ||
      (k_out && !on_device(k_out, dev)) || (rope->rot_dim && !on_device(rope->inv_freq, dev)) || (status && !on_device(status, dev)))
    return DEC_ERR_INVALID_ARG;

  const int units = (max_new < ps ? max_new : ps) * (D / 16);
  AppendArgs a{device_cache(cache), rope->inv_freq, rope->rot_dim, rope->pairs == DEC_ROPE_NEIGHBOUR, rope->factor, q, k,
               v, q_out, k_out, q_stride, k_stride, v_stride, q_out_stride, k_out_stride, q ? n_heads : 0, n_tokens, max_new, (int)pieces,
               hkv, q ? hkv : 0, cu_new, seq_lens, page_table, table_stride, status};
  // A block a kv head, and one for its query heads, is the shortest path for few tokens; more blocks than fill the GPU
  // compute the angles over and over.  With blocks that a page fills (256 threads or more) twice the SMs are enough
  // and queries and keys are launches of their own, each with the registers it needs; with little in each, 8 an SM.  B200,
  // 32 / 8 heads of 128, bf16, us, one way and the other: 256 single tokens 7.4 (8 an SM) / 11.1 (2), 64 x 4 5.5 / 7.0, 8 x 1000
  // 51.8 / 43.2, 4 x 8192 158 (one launch) / 143 (two).
  const bool split = q && units >= 256;
  const int64_t enough = split ? 2 * 148 : 8 * 148;
  // (a block notes borders in shared memory: 128 bytes a head, which is enough for 128 heads)
  while (a.kv_blocks > 1 && pages * a.kv_blocks > enough && hkv <= a.kv_blocks / 2 * 128) a.kv_blocks = (a.kv_blocks + 1) / 2;
  while (a.q_blocks > 1 && pages * a.q_blocks > enough) a.q_blocks = (a.q_blocks + 1) / 2;
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
  *out_bytes = kBlocks * 2 * (sizeof(uint64_t) + (24 + 8 * (size_t)cache->head_dim) * sizeof(float));
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
  if ((dtype != DEC_BF16 && dtype != DEC_F32) || !scale_ok(scale) || table_stride < 0)
    return DEC_ERR_INVALID_ARG;
  if (n_seqs == 0) return DEC_OK;
  const int hkv = cache->n_kv_heads, D = cache->head_dim, esz = dtype == DEC_BF16 ? 2 : 4;
  // tiles of 16 positions are counted in 32 bits
  if ((double)n_seqs * hkv * table_stride * cache->page_size / 16 >= 2147483648.0) return DEC_ERR_UNSUPPORTED;
  if (!q || !out || !seq_lens || !page_table || !workspace || workspace_bytes < need || out == q) return DEC_ERR_INVALID_ARG;
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
  static const uint64_t key = [] {
    std::random_device r;
    return (uint64_t)r() << 32 | r() | 1;
  }();
  const size_t flags = kBlocks * 2 * sizeof(uint64_t);
  PagedArgs a{device_cache(cache), q, out, q_stride, out_stride, n_heads / hkv, n_seqs, 31 - __builtin_clz(cache->page_size),
              seq_lens, page_table, table_stride, scale * 1.4426950408889634f,
              reinterpret_cast<float*>(static_cast<char*>(workspace) + flags), static_cast<uint64_t*>(workspace), key,
              (cache->wait_timeout_us ? cache->wait_timeout_us : 1000000) * 1000ull, status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DEC_BF16)
    e = D == 64 ? launch_paged<__nv_bfloat16, 64>(a, st) : launch_paged<__nv_bfloat16, 128>(a, st);
  else
    e = D == 64 ? launch_paged<float, 64>(a, st) : launch_paged<float, 128>(a, st);
  return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA;
}
