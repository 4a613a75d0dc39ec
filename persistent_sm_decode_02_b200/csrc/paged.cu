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
struct AppendArgs {
  Cache c;
  const double* inv_freq;
  int rot, neighbour;
  float factor;
  const void *q, *k, *v;
  void* q_out;
  int64_t qs, ks, vs, qos;
  int gs, n_tokens, max_new, pieces, hpc;  // gs: query heads per kv head (0: no q); hpc: kv heads per block
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

// Sixteen values of one row, in the two 8-element chunks a thread holds, turned by their eight angles.
__device__ __forceinline__ void rotate16(float* x, const float* cs, const float* sn, bool neighbour) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (neighbour) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * cs[i] - b * sn[i];
      x[2 * i + 1] = a * sn[i] + b * cs[i];
    } else {
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

// Rows before the piece, rounded again for a larger scale.
__device__ __forceinline__ void rescale_rows(uint8_t* p, int bytes, float ratio) {
  for (int i = threadIdx.x * 8; i < bytes; i += blockDim.x * 8) {
    uint2 w = *reinterpret_cast<const uint2*>(p + i);
    const float2 a = from_e4m3x2(w.x), b = from_e4m3x2(w.x >> 16), c = from_e4m3x2(w.y), d = from_e4m3x2(w.y >> 16);
    const float x[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    store_codes(p + i, x, ratio);
  }
}

// One block per (sequence, page it touches, hpc kv heads).  A thread holds the same 16 dims of its rows for
// every head, so it computes their 8 angles once (fp64 turns, reduced to +-1/2, then fp32 sin and cos).
template <typename T, int D, int NIT>
__global__ void __launch_bounds__(512) append_kernel(AppendArgs a) {
  __shared__ float red[2][2][16];
  constexpr int kUnits = D / 16;  // threads a row
  const int groups = a.c.hkv / a.hpc;
  const int hg = blockIdx.x % groups, piece = blockIdx.x / groups % a.pieces, s = blockIdx.x / groups / a.pieces;
  const int tid = threadIdx.x, ps = a.c.ps;
  const int64_t c0 = a.cu[s], c1 = a.cu[s + 1], n = c1 - c0;
  const int64_t len = a.lens[s];
  if (n == 0) return;
  if (n < 0 || c0 < 0 || c1 > a.n_tokens || n > a.max_new || len < n || len > (int64_t)a.table_stride * ps) {
    if (tid == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
    return;
  }
  const int64_t start = len - n, pi = start / ps + piece;
  const int64_t lo = max(start, pi * ps), hi = min(len, (pi + 1) * ps);
  if (lo >= hi) return;
  const int page = a.table[(int64_t)s * a.table_stride + pi];
  const bool page_ok = page >= 0 && page < a.c.n_pages;
  if (!page_ok && tid == 0) flag(a.status, DEC_SEQ_BAD_PAGE);
  const int nr = (int)(hi - lo), slot0 = (int)(lo - pi * ps);
  const int64_t row0 = c0 + (lo - start);
  const bool neighbour = a.neighbour;

  const int c = tid % kUnits;  // blockDim.x is a multiple of kUnits
  const bool turned = c < a.rot / 16;
  const int d0 = turned && !neighbour ? 8 * c : 16 * c, d1 = turned && !neighbour ? a.rot / 2 + 8 * c : 16 * c + 8;
  float cs[NIT][8], sn[NIT][8];
  int row[NIT];
#pragma unroll
  for (int it = 0; it < NIT; ++it) {
    row[it] = (tid + it * blockDim.x) / kUnits;
    if (turned && row[it] < nr) {
      const double pos = (double)(lo + row[it]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double turns = pos * a.inv_freq[8 * c + i] * 0.15915494309189535;  // 1 / (2 pi)
        float co, si;
        sincospif(2.f * (float)(turns - rint(turns)), &si, &co);
        cs[it][i] = co * a.factor;
        sn[it][i] = si * a.factor;
      }
    }
  }

  for (int g = 0; g < a.hpc; ++g) {
    const int head = hg * a.hpc + g;
    float k[NIT][16], mk = 0.f, mv = 0.f;
    Vec8<T> v[NIT][2];
#pragma unroll
    for (int it = 0; it < NIT; ++it)
      if (row[it] < nr) {
        const T* kp = static_cast<const T*>(a.k) + (row0 + row[it]) * a.ks + (int64_t)head * D;
        const T* vp = static_cast<const T*>(a.v) + (row0 + row[it]) * a.vs + (int64_t)head * D;
        Vec8<T> x[2];
        x[0].load(kp + d0);
        x[1].load(kp + d1);
        v[it][0].load(vp + d0);
        v[it][1].load(vp + d1);
        x[0].get(k[it]);
        x[1].get(k[it] + 8);
        if (turned) rotate16(k[it], cs[it], sn[it], neighbour);
        float y[16];
        v[it][0].get(y);
        v[it][1].get(y + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          mk = amax_finite(mk, k[it][i]);
          mv = amax_finite(mv, y[i]);
        }
      }
    const int64_t si = (int64_t)page * a.c.hkv + head;
    float k_was = 0.f, v_was = 0.f;
    if (page_ok && slot0 > 0) k_was = a.c.ks[si], v_was = a.c.vs[si];
    mk = warp_max(mk);
    mv = warp_max(mv);
    if ((tid & 31) == 0) red[g & 1][0][tid >> 5] = mk, red[g & 1][1][tid >> 5] = mv;
    __syncthreads();  // also orders every read of the old scales before their update
    for (int w = 0; w < (int)blockDim.x / 32; ++w) {
      mk = fmaxf(mk, red[g & 1][0][w]);
      mv = fmaxf(mv, red[g & 1][1][w]);
    }
    if (page_ok) {
      const float k_now = fmaxf(k_was, pow2(scale_exponent(mk))), v_now = fmaxf(v_was, pow2(scale_exponent(mv)));
      if (tid == 0) a.c.ks[si] = k_now, a.c.vs[si] = v_now;
      uint8_t* kp = a.c.k + si * ps * D;
      uint8_t* vp = a.c.v + si * ps * D;
      if (slot0 > 0 && k_now > k_was) rescale_rows(kp, slot0 * D, k_was / k_now);
      if (slot0 > 0 && v_now > v_was) rescale_rows(vp, slot0 * D, v_was / v_now);
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
    }
    for (int h = head * a.gs; h < (head + 1) * a.gs; ++h)
#pragma unroll
      for (int it = 0; it < NIT; ++it)
        if (row[it] < nr) {
          const T* qp = static_cast<const T*>(a.q) + (row0 + row[it]) * a.qs + (int64_t)h * D;
          T* op = static_cast<T*>(a.q_out) + (row0 + row[it]) * a.qos + (int64_t)h * D;
          Vec8<T> x[2];
          float y[16];
          x[0].load(qp + d0);
          x[1].load(qp + d1);
          x[0].get(y);
          x[1].get(y + 8);
          if (turned) rotate16(y, cs[it], sn[it], neighbour);
          Vec8<T>::store(op + d0, y);
          Vec8<T>::store(op + d1, y + 8);
        }
  }
}

template <typename T, int D>
cudaError_t launch_append(const AppendArgs& a, int blocks, int units, cudaStream_t s) {
  const int nit = units > 256 ? 2 : 1;
  const int threads = ((units + nit - 1) / nit + 31) / 32 * 32;
  if (nit == 2)
    append_kernel<T, D, 2><<<blocks, threads, 0, s>>>(a);
  else
    append_kernel<T, D, 1><<<blocks, threads, 0, s>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ attention
struct PagedArgs {
  Cache c;
  const void* q;
  void* out;
  int64_t qs, os;
  int gs;
  const int32_t *lens, *table;
  int table_stride;
  float scale_log2;
  int32_t* status;
};

// One block per (sequence, kv head): warps take positions in turn, lanes hold D / 32 dims of every query head.
template <typename T, int D>
__global__ void __launch_bounds__(256) paged_kernel(PagedArgs a) {
  constexpr int kD = D / 32, kW = 8;
  __shared__ float m_s[kW][8], l_s[kW][8], o_s[kW][8][D];
  const int s = blockIdx.x / a.c.hkv, head = blockIdx.x % a.c.hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ps = a.c.ps;
  int64_t len = a.lens[s];
  if (len < 0 || len > (int64_t)a.table_stride * ps) {
    if (tid == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
    len = 0;
  }
  const T* qp = static_cast<const T*>(a.q) + s * a.qs + (int64_t)head * a.gs * D;
  float q[8][kD], o[8][kD], m[8], l[8];
  for (int h = 0; h < 8; ++h) {
    m[h] = -INFINITY, l[h] = 0.f;
    for (int i = 0; i < kD; ++i) q[h][i] = h < a.gs ? (float)qp[h * D + lane * kD + i] * a.scale_log2 : 0.f, o[h][i] = 0.f;
  }
  for (int64_t t = warp; t < len; t += kW) {
    const int page = a.table[(int64_t)s * a.table_stride + t / ps];
    if (page < 0 || page >= a.c.n_pages) {
      if (lane == 0) flag(a.status, DEC_SEQ_BAD_PAGE);
      continue;
    }
    const int64_t si = (int64_t)page * a.c.hkv + head, at = (si * ps + t % ps) * D + lane * kD;
    float k[kD], v[kD];
    for (int i = 0; i < kD; i += 2) {
      const float2 x = from_e4m3x2(*reinterpret_cast<const uint16_t*>(a.c.k + at + i));
      const float2 y = from_e4m3x2(*reinterpret_cast<const uint16_t*>(a.c.v + at + i));
      k[i] = x.x * a.c.ks[si], k[i + 1] = x.y * a.c.ks[si], v[i] = y.x * a.c.vs[si], v[i + 1] = y.y * a.c.vs[si];
    }
    for (int h = 0; h < a.gs; ++h) {
      float d = 0.f;
      for (int i = 0; i < kD; ++i) d = fmaf(q[h][i], k[i], d);
      d = warp_sum(d);
      const float mn = fmaxf(m[h], d), f = exp2f(m[h] - mn), p = exp2f(d - mn);
      m[h] = mn, l[h] = l[h] * f + p;
      for (int i = 0; i < kD; ++i) o[h][i] = fmaf(p, v[i], o[h][i] * f);
    }
  }
  for (int h = 0; h < a.gs; ++h) {
    if (lane == 0) m_s[warp][h] = m[h], l_s[warp][h] = l[h];
    for (int i = 0; i < kD; ++i) o_s[warp][h][lane * kD + i] = o[h][i];
  }
  __syncthreads();
  for (int e = tid; e < a.gs * D; e += blockDim.x) {
    const int h = e / D;
    float M = -INFINITY, L = 0.f, x = 0.f;
    for (int w = 0; w < kW; ++w)
      if (l_s[w][h] != 0.f) M = fmaxf(M, m_s[w][h]);
    for (int w = 0; w < kW; ++w)
      if (l_s[w][h] != 0.f) {
        const float f = exp2f(m_s[w][h] - M);
        L += f * l_s[w][h];
        x += f * o_s[w][h][e % D];
      }
    static_cast<T*>(a.out)[s * a.os + (int64_t)head * a.gs * D + e] = (T)(L != 0.f ? x / L : 0.f);
  }
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
  AppendArgs a{device_cache(cache), rope->inv_freq, rope->rot_dim, rope->pairs == DEC_ROPE_NEIGHBOUR, rope->factor, q, k,
               v, q_out, q_stride, k_stride, v_stride, q_out_stride, q ? n_heads / hkv : 0, n_tokens, max_new,
               (int)(((int64_t)max_new + ps - 2) / ps + 1), 1, cu_new, seq_lens, page_table, table_stride, status};
  const int64_t blocks = (int64_t)n_seqs * a.pieces * (hkv / a.hpc);
  if (blocks > INT32_MAX) return DEC_ERR_UNSUPPORTED;
  const int units = (max_new < ps ? max_new : ps) * (D / 16);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DEC_BF16)
    e = D == 64 ? launch_append<__nv_bfloat16, 64>(a, (int)blocks, units, st)
                : launch_append<__nv_bfloat16, 128>(a, (int)blocks, units, st);
  else
    e = D == 64 ? launch_append<float, 64>(a, (int)blocks, units, st)
                : launch_append<float, 128>(a, (int)blocks, units, st);
  return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA;
}

extern "C" int dec_attention_paged_workspace(const dec_paged_cache* cache, int32_t n_seqs, int32_t n_heads,
                                             size_t* out_bytes) {
  if (!out_bytes || n_seqs < 0) return DEC_ERR_INVALID_ARG;
  int rc = check_cache(cache);
  if (rc) return rc;
  rc = head_layout(n_heads, cache->n_kv_heads, cache->head_dim);
  if (rc) return rc;
  *out_bytes = 16;
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
  if ((int64_t)n_seqs * hkv > INT32_MAX) return DEC_ERR_UNSUPPORTED;
  PagedArgs a{device_cache(cache), q, out, q_stride, out_stride, n_heads / hkv, seq_lens, page_table, table_stride,
              scale * 1.4426950408889634f, status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int blocks = n_seqs * hkv;
  if (dtype == DEC_BF16) {
    if (D == 64)
      paged_kernel<__nv_bfloat16, 64><<<blocks, 256, 0, st>>>(a);
    else
      paged_kernel<__nv_bfloat16, 128><<<blocks, 256, 0, st>>>(a);
  } else {
    if (D == 64)
      paged_kernel<float, 64><<<blocks, 256, 0, st>>>(a);
    else
      paged_kernel<float, 128><<<blocks, 256, 0, st>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? DEC_OK : DEC_ERR_CUDA;
}
