// dec_attention_prefill: attention of packed prompts.
#include "op_common.cuh"
#include "prefill_tc.cuh"

namespace {

using namespace dec_op;
using tc::F2;

__device__ __forceinline__ void copy16(float* dst, const float* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
// Waits for all copies but those issued last (since the group before).
__device__ __forceinline__ void earlier_copies() { asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 1;" ::: "memory"); }

// fp32 prompts, on the CUDA cores (the tensor cores' fp32 inputs keep 11 bits).  A block takes 32 queries of one head,
// and its groups of 4 warps 64 keys in turn, so that the longest row's chain of steps is short; each keeps the running
// maximum and sum of its softmax, and they are joined at the end.  A block has an SM to itself: short rows then go where
// long ones are done, not beside them.  A thread has 4 x 4 scores and 4 x (D / 16)
// outputs, in pairs for the two-wide FMA.  K of a group's next step is on its way while this one's values are added up,
// V while its scores are worked out.  Five ragged prompts of up to 700, 4 heads of 64: 39 us (two
// groups and two blocks an SM 51, one group and 64 queries 87).
template <int D>
struct Fp32Shape {
  static constexpr int kGroups = D == 64 ? 4 : 2;  // what shared memory holds
  static constexpr int kSmem = (32 * (D + 4) + kGroups * (2 * 64 * (D + 4) + 32 * 64)) * 4;
};

template <int D>
__global__ void __launch_bounds__(Fp32Shape<D>::kGroups * 128) prefill_fp32(PrefillArgs a, Tiling tl, int n_seqs) {
  constexpr int kM = 32, kN = 64, kStride = D + 4, kC = D / 64, kGroups = Fp32Shape<D>::kGroups, kStep = kGroups * kN;
  extern __shared__ __align__(16) float sm[];
  constexpr int kGroup = 2 * kN * kStride + kM * kN;  // floats of a group: K, V, P
  const int group = threadIdx.x >> 7;
  float *q_s = sm, *k_s = q_s + kM * kStride + group * kGroup, *v_s = k_s + kN * kStride, *p_s = v_s + kN * kStride;
  auto sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory"); };
  const int head = blockIdx.x % a.heads;
  int m0;
  const int at = blockIdx.x / a.heads;
  const int s = tl.packed ? tile_at<true>(a, n_seqs, tl.tiles, kM, at, m0) : tile_at<false>(a, n_seqs, tl.tiles, kM, at, m0);
  if (s < 0) {
    if (threadIdx.x == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
    return;
  }
  const int tid = threadIdx.x & 127, tx = tid & 15, ty = tid >> 4;
  const Range r = range_of(a, s);
  if (!r.ok && threadIdx.x == 0) flag(a.status, DEC_SEQ_BAD_RANGE);
  const int kvh = head / a.gs;
  if (m0 >= r.lq) return;
  const int rows = min(kM, r.lq - m0), shift = r.lk - r.lq;
  const int n_end = !r.ok ? 0 : a.causal ? min(r.lk, m0 + rows + shift) : r.lk;

  auto load = [&](float* dst, const void* src, int64_t stride, int n0) {
    const float* p = static_cast<const float*>(src) + (int64_t)kvh * D;
    for (int e = tid; e < kN * (D / 4); e += 128) {
      const int i = e / (D / 4), c = e % (D / 4) * 4;
      const bool live = n0 + i < n_end;
      copy16(dst + i * kStride + c, live ? p + (r.k0 + n0 + i) * stride + c : p, live);
    }
  };
  if (group * kN < n_end) {
    load(k_s, a.k, a.ks, group * kN);
    asm volatile("cp.async.commit_group;" ::: "memory");
    load(v_s, a.v, a.vs, group * kN);
  }
  for (int e = threadIdx.x; e < kM * (D / 4); e += kGroups * 128) {
    const int i = e / (D / 4), c = e % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < rows) x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + (r.q0 + m0 + i) * a.qs + (int64_t)head * D + c);
    *reinterpret_cast<float4*>(q_s + i * kStride + c) =
        make_float4(x.x * a.scale_log2, x.y * a.scale_log2, x.z * a.scale_log2, x.w * a.scale_log2);
  }
  F2 o[4][kC * 2];
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < kC * 2; ++c) o[i][c] = 0;
  }
  __syncthreads();
  for (int n0 = group * kN; n0 < n_end; n0 += kStep) {
    earlier_copies();  // K is here, V may be under way
    sync();
    F2 sc2[4][4];  // sums over even and odd dims
#pragma unroll
    for (int i = 0; i < 16; ++i) sc2[i / 4][i % 4] = 0;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      ulonglong2 x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const ulonglong2*>(q_s + (ty * 4 + i) * kStride + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const ulonglong2*>(k_s + (tx + 16 * j) * kStride + d);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc2[i][j] = tc::fma2(x[i].y, y[j].y, tc::fma2(x[i].x, y[j].x, sc2[i][j]));
    }
    float sc[4][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 u = tc::un2(sc2[i / 4][i % 4]);
      sc[i / 4][i % 4] = u.x + u.y;
    }
    sync();  // K is read
    if (n0 + kStep < n_end) load(k_s, a.k, a.ks, n0 + kStep);
    int seen[4];  // keys of this tile that row i sees
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = m0 + ty * 4 + i;
      seen[i] = row < r.lq ? min(kN, (a.causal ? min(n_end, row + shift + 1) : n_end) - n0) : 0;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (tx + 16 * j < seen[i]) mx = fmaxf(mx, sc[i][j]);
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx), base = mn == -INFINITY ? 0.f : mn, f = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = tx + 16 * j < seen[i] ? exp2f(sc[i][j] - base) : 0.f;
        p_s[(ty * 4 + i) * kN + tx + 16 * j] = p;
        sum += p;
      }
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
      m[i] = mn, l[i] = l[i] * f + sum;
#pragma unroll
      for (int j = 0; j < kC * 2; ++j) o[i][j] = tc::mul2(o[i][j], tc::f2(f, f));
    }
    earlier_copies();  // V is here, the next K may be under way
    sync();            // (a row's weights are its own warp's)
    auto add = [&](int i, float p, const ulonglong2 (&y)[kC]) {
      const F2 pp = tc::f2(p, p);
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        o[i][2 * c] = tc::fma2(pp, y[c].x, o[i][2 * c]);
        o[i][2 * c + 1] = tc::fma2(pp, y[c].y, o[i][2 * c + 1]);
      }
    };
    const int least = max(0, min(min(seen[0], seen[1]), min(seen[2], seen[3]))) & ~3;  // keys that all four rows see
    const int most = max(max(seen[0], seen[1]), max(seen[2], seen[3]));
#pragma unroll 2
    for (int t = 0; t < least; t += 4) {
      float p[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(p_s + (ty * 4 + i) * kN + t);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        ulonglong2 y[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) y[c] = *reinterpret_cast<const ulonglong2*>(v_s + (t + u) * kStride + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) add(i, p[i][u], y);
      }
    }
#pragma unroll 1
    for (int t = least; t < most; ++t) {
      ulonglong2 y[kC];
#pragma unroll
      for (int c = 0; c < kC; ++c) y[c] = *reinterpret_cast<const ulonglong2*>(v_s + t * kStride + c * 64 + tx * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t < seen[i]) add(i, p_s[(ty * 4 + i) * kN + t], y);  // an unseen value may be anything
    }
    sync();  // V is read
    if (n0 + kStep < n_end) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      load(v_s, a.v, a.vs, n0 + kStep);
    }
  }
  // the other groups' sums to the first, through their K and V tiles
  if (group > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int c = 0; c < kC * 2; ++c) reinterpret_cast<F2*>(k_s)[(i * kC * 2 + c) * 128 + tid] = o[i][c];
      k_s[(16 * kC + i) * 128 + tid] = m[i], k_s[(16 * kC + 4 + i) * 128 + tid] = l[i];
    }
  }
  __syncthreads();
  if (group > 0) return;
#pragma unroll 1
  for (int other = 1; other < kGroups; ++other) {
    const float* x_s = k_s + other * kGroup;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m1 = x_s[(16 * kC + i) * 128 + tid], l1 = x_s[(16 * kC + 4 + i) * 128 + tid];
      const float mn = fmaxf(m[i], m1), base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - base), f1 = exp2f(m1 - base);
      m[i] = mn;
      l[i] = l[i] * f + l1 * f1;
#pragma unroll
      for (int c = 0; c < kC * 2; ++c)
        o[i][c] = tc::fma2(reinterpret_cast<const F2*>(x_s)[(i * kC * 2 + c) * 128 + tid], tc::f2(f1, f1),
                           tc::mul2(o[i][c], tc::f2(f, f)));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (ty * 4 + i >= rows) continue;
    // a row that sees nothing gives zeros, one that sees only scores of -infinity 0 / 0
    const bool blind = n_end <= 0 || (a.causal && m0 + ty * 4 + i + shift < 0);
    const float inv = blind ? 0.f : 1.f / l[i];
    float* op = static_cast<float*>(a.out) + (r.q0 + m0 + ty * 4 + i) * a.os + (int64_t)head * D;
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const float2 u = tc::un2(o[i][2 * c]), w = tc::un2(o[i][2 * c + 1]);
      *reinterpret_cast<float4*>(op + c * 64 + tx * 4) = make_float4(u.x * inv, u.y * inv, w.x * inv, w.y * inv);
    }
  }
}

template <int D>
cudaError_t launch_fp32(const PrefillArgs& a, int n_seqs, cudaStream_t st) {
  const Tiling tl = tiling(n_seqs, a.n_q, a.max_q, 32);
  constexpr int smem = Fp32Shape<D>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(prefill_fp32<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  prefill_fp32<D><<<(unsigned)((int64_t)tl.tiles * (tl.packed ? 1 : n_seqs) * a.heads), Fp32Shape<D>::kGroups * 128, smem, st>>>(
      a, tl, n_seqs);
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
  if ((dtype != DEC_BF16 && dtype != DEC_F32) || !scale_ok(scale)) return DEC_ERR_INVALID_ARG;
  if (n_seqs < 0 || n_q < 0 || n_k < 0 || max_q < 0) return DEC_ERR_INVALID_ARG;
  if (n_seqs == 0 || n_q == 0 || max_q == 0) return DEC_OK;
  const int D = head_dim, esz = dtype == DEC_BF16 ? 2 : 4;
  if (!q || !out || !cu_q || !cu_k || (n_k > 0 && (!k || !v))) return DEC_ERR_INVALID_ARG;
  if (out == q || out == k || out == v) return DEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned4(cu_q) || !aligned4(cu_k) ||
      !aligned4(status) || !stride_ok(q_stride, (int64_t)n_heads * D, esz) ||
      !stride_ok(out_stride, (int64_t)n_heads * D, esz) || !stride_ok(k_stride, (int64_t)n_kv_heads * D, esz) ||
      !stride_ok(v_stride, (int64_t)n_kv_heads * D, esz))
    return DEC_ERR_INVALID_ARG;
  if (max_q > n_q) max_q = n_q;  // no valid sequence has more
  if ((int64_t)n_seqs * n_heads * (((int64_t)max_q + 31) / 32) > INT32_MAX) return DEC_ERR_UNSUPPORTED;
  if (cudaPeekAtLastError() != cudaSuccess) return DEC_ERR_CUDA;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return DEC_ERR_CUDA;
  if (!on_device(q, dev) || !on_device(out, dev) || !on_device(cu_q, dev) || !on_device(cu_k, dev) ||
      (n_k > 0 && (!on_device(k, dev) || !on_device(v, dev))) || (status && !on_device(status, dev)))
    return DEC_ERR_INVALID_ARG;
  PrefillArgs a{q, k, v, out, q_stride, k_stride, v_stride, out_stride, n_heads, n_heads / n_kv_heads, n_q, n_k, max_q,
                causal, cu_q, cu_k, scale * 1.4426950408889634f, status};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == DEC_BF16)
    e = D == 64 ? tc::launch<64>(a, n_seqs, st) : tc::launch<128>(a, n_seqs, st);
  else
    e = D == 64 ? launch_fp32<64>(a, n_seqs, st) : launch_fp32<128>(a, n_seqs, st);
  return e == cudaSuccess ? DEC_OK : DEC_ERR_CUDA;
}
