// dec_attention_prefill: attention of packed prompts.
#include "op_common.cuh"
#include "prefill_tc.cuh"

namespace {

using namespace dec_op;

// One block per (64 queries, head): scores and values on the CUDA cores in fp32, 4 x 4 scores and 4 x (D / 16)
// outputs a thread, 64 keys at a time with the running maximum and sum of the softmax.
template <typename T, int D>
__global__ void __launch_bounds__(256) prefill_simt(PrefillArgs a, int tiles) {
  constexpr int kM = 64, kN = 64, kStride = D + 4, kC = D / 64;
  extern __shared__ __align__(16) float sm[];
  float *q_s = sm, *k_s = q_s + kM * kStride, *v_s = k_s + kN * kStride, *p_s = v_s + kN * kStride;
  const int head = blockIdx.x % a.heads, tile = blockIdx.x / a.heads % tiles, s = blockIdx.x / a.heads / tiles;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const Range r = range_of(a, s);
  if (!r.ok && tid == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
  const int m0 = (tiles - 1 - tile) * kM, kvh = head / a.gs;
  if (m0 >= r.lq) return;
  const int rows = min(kM, r.lq - m0), shift = r.lk - r.lq;
  const int n_end = !r.ok ? 0 : a.causal ? min(r.lk, m0 + rows + shift) : r.lk;

  for (int e = tid; e < kM * (D / 8); e += 256) {
    const int i = e / (D / 8), c = e % (D / 8) * 8;
    float x[8] = {};
    if (i < rows) {
      Vec8<T> w;
      w.load(static_cast<const T*>(a.q) + (r.q0 + m0 + i) * a.qs + (int64_t)head * D + c);
      w.get(x);
    }
    for (int j = 0; j < 8; ++j) q_s[i * kStride + c + j] = x[j] * a.scale_log2;
  }
  float o[4][kC * 4] = {}, m[4], l[4];
  for (int i = 0; i < 4; ++i) m[i] = -INFINITY, l[i] = 0.f;
  for (int n0 = 0; n0 < n_end; n0 += kN) {
    __syncthreads();
    for (int e = tid; e < kN * (D / 8); e += 256) {
      const int i = e / (D / 8), c = e % (D / 8) * 8;
      float x[8] = {}, y[8] = {};
      if (n0 + i < n_end) {
        Vec8<T> w;
        w.load(static_cast<const T*>(a.k) + (r.k0 + n0 + i) * a.ks + (int64_t)kvh * D + c);
        w.get(x);
        w.load(static_cast<const T*>(a.v) + (r.k0 + n0 + i) * a.vs + (int64_t)kvh * D + c);
        w.get(y);
      }
      for (int j = 0; j < 8; ++j) k_s[i * kStride + c + j] = x[j], v_s[i * kStride + c + j] = y[j];
    }
    __syncthreads();
    float sc[4][4] = {};
    for (int d = 0; d < D; d += 4) {
      float4 x[4], y[4];
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(q_s + (ty * 4 + i) * kStride + d);
      for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(k_s + (tx + 16 * j) * kStride + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sc[i][j] = fmaf(x[i].x, y[j].x, fmaf(x[i].y, y[j].y, fmaf(x[i].z, y[j].z, fmaf(x[i].w, y[j].w, sc[i][j]))));
    }
    int seen[4];  // keys of this tile that row i sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + ty * 4 + i;
      seen[i] = row < r.lq ? min(kN, (a.causal ? min(n_end, row + shift + 1) : n_end) - n0) : 0;
      float mx = -INFINITY;
      for (int j = 0; j < 4; ++j)
        if (tx + 16 * j < seen[i]) mx = fmaxf(mx, sc[i][j]);
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[i] - base);
      float sum = 0.f;
      for (int j = 0; j < 4; ++j) {
        const float p = tx + 16 * j < seen[i] ? exp2f(sc[i][j] - base) : 0.f;
        p_s[(ty * 4 + i) * kN + tx + 16 * j] = p;
        sum += p;
      }
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      m[i] = mn, l[i] = l[i] * f + sum;
      for (int j = 0; j < kC * 4; ++j) o[i][j] *= f;
    }
    __syncwarp();  // a row's 16 threads are in one warp
    const bool whole = seen[0] == kN && seen[3] == kN;
    for (int t = 0; t < kN; ++t) {
      float4 y[kC];
      for (int c = 0; c < kC; ++c) y[c] = *reinterpret_cast<const float4*>(v_s + t * kStride + c * 64 + tx * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (!whole && t >= seen[i]) continue;  // an unseen value may be anything
        const float p = p_s[(ty * 4 + i) * kN + t];
#pragma unroll
        for (int c = 0; c < kC; ++c) {
          o[i][4 * c] = fmaf(p, y[c].x, o[i][4 * c]);
          o[i][4 * c + 1] = fmaf(p, y[c].y, o[i][4 * c + 1]);
          o[i][4 * c + 2] = fmaf(p, y[c].z, o[i][4 * c + 2]);
          o[i][4 * c + 3] = fmaf(p, y[c].w, o[i][4 * c + 3]);
        }
      }
    }
  }
  for (int i = 0; i < 4; ++i) {
    if (ty * 4 + i >= rows) continue;
    const float inv = l[i] != 0.f ? 1.f / l[i] : 0.f;
    T* op = static_cast<T*>(a.out) + (r.q0 + m0 + ty * 4 + i) * a.os + (int64_t)head * D;
    for (int c = 0; c < kC; ++c)
      for (int j = 0; j < 4; ++j) op[c * 64 + tx * 4 + j] = (T)(o[i][4 * c + j] * inv);
  }
}

template <typename T, int D>
cudaError_t launch_simt(const PrefillArgs& a, int n_seqs, cudaStream_t st) {
  const int tiles = (a.max_q + 63) / 64;
  const int smem = (3 * 64 * (D + 4) + 64 * 64) * 4;
  cudaError_t e = cudaFuncSetAttribute(prefill_simt<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prefill_simt<T, D><<<(unsigned)((int64_t)n_seqs * tiles * a.heads), 256, smem, st>>>(a, tiles);
  return cudaGetLastError();
}

}  // namespace

extern "C" int dec_attention_prefill(int32_t dtype, const void* q, const void* k, const void* v, void* out,
                                     int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t out_stride,
                                     int32_t n_heads, int32_t n_kv_heads, int32_t head_dim, int32_t n_seqs, int32_t n_q,
                                     int32_t n_k, int32_t max_q, const int32_t* cu_q, const int32_t* cu_k,
                                     int32_t causal, float scale, int32_t* status, void* stream) {
  int rc = head_layout(n_heads, n_kv_heads, head_dim);
  if (rc) return rc;
  if ((dtype != DEC_BF16 && dtype != DEC_F32) || !(scale > 0.f) || !isfinite(scale)) return DEC_ERR_INVALID_ARG;
  if (n_seqs < 0 || n_q < 0 || n_k < 0 || max_q < 0) return DEC_ERR_INVALID_ARG;
  if (n_seqs == 0 || n_q == 0 || max_q == 0) return DEC_OK;
  const int D = head_dim, esz = dtype == DEC_BF16 ? 2 : 4;
  if (!q || !out || !cu_q || !cu_k || (n_k > 0 && (!k || !v))) return DEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned4(cu_q) || !aligned4(cu_k) ||
      !aligned4(status) || !stride_ok(q_stride, (int64_t)n_heads * D, esz) ||
      !stride_ok(out_stride, (int64_t)n_heads * D, esz) || !stride_ok(k_stride, (int64_t)n_kv_heads * D, esz) ||
      !stride_ok(v_stride, (int64_t)n_kv_heads * D, esz))
    return DEC_ERR_INVALID_ARG;
  if (cudaPeekAtLastError() != cudaSuccess) return DEC_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DEC_ERR_CUDA;
  if (!on_device(q, dev) || !on_device(out, dev) || !on_device(cu_q, dev) || !on_device(cu_k, dev) ||
      (n_k > 0 && (!on_device(k, dev) || !on_device(v, dev))) || (status && !on_device(status, dev)))
    return DEC_ERR_INVALID_ARG;
  if (max_q > n_q) max_q = n_q;  // no valid sequence has more
  if ((int64_t)n_seqs * n_heads * (((int64_t)max_q + 63) / 64) > INT32_MAX) return DEC_ERR_UNSUPPORTED;
  PrefillArgs a{q, k, v, out, q_stride, k_stride, v_stride, out_stride, n_heads, n_heads / n_kv_heads, n_q, n_k, max_q,
                causal, cu_q, cu_k, scale * 1.4426950408889634f, status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DEC_BF16)
    e = D == 64 ? tc::launch<64>(a, n_seqs, st) : tc::launch<128>(a, n_seqs, st);
  else
    e = D == 64 ? launch_simt<float, 64>(a, n_seqs, st) : launch_simt<float, 128>(a, n_seqs, st);
  return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA;
}
