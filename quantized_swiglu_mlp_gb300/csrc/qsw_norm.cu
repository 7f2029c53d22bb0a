// Norms around a block, one pass over the rows (HBM-bound):
//
//   z  = y rsqrt(mean y^2 + eps) w_post           the block's output, normed
//   h' = h + scale gate z                         residual
//   n  = h' rsqrt(mean h'^2 + eps) w_next         the next block's input
//
// Any of the three may be left out (see qsw_post_norm and qsw_rms_norm).  One
// CTA per row holds the row in registers as f32: both means are sums over
// those registers, and n is computed from h' before it is rounded for storing.
#include "qsw_fp4.cuh"
#include "qsw_internal.h"

namespace qsw {
namespace {

struct NormParams {
  const uint16_t *h, *y, *w_post, *gate, *w_next;
  uint16_t *h_out, *n_out;
  int64_t rows_per_gate;   // rows that share a row of the gate
  int H;
  int gate_cols;           // H, or 1: one gate value per gate row
  int norm_y;
  float scale, eps, inv_h;
};

// VEC consecutive 16-bit values as f32.
template <class A, int VEC>
__device__ __forceinline__ void load_vec(const uint16_t *p, float (&v)[VEC]) {
  if constexpr (VEC == 8) {
    const uint4 q = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = A::lo(w[i]);
      v[2 * i + 1] = A::hi(w[i]);
    }
  } else if constexpr (VEC == 2) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    v[0] = A::lo(w);
    v[1] = A::hi(w);
  } else {
    v[0] = A::lo(*p);
  }
}

template <class A, int VEC>
__device__ __forceinline__ void store_vec(uint16_t *p, const float (&v)[VEC]) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4 *>(p) = make_uint4(A::pack2(v[0], v[1]), A::pack2(v[2], v[3]), A::pack2(v[4], v[5]),
                                               A::pack2(v[6], v[7]));
  else if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t *>(p) = A::pack2(v[0], v[1]);
  else
    *p = A::store(v[0]);
}

// Sum over the CTA; `buf` is one of two 32-float buffers, so that a second
// sum needs no barrier before it.
__device__ __forceinline__ float block_sum(float v, float *buf) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  float s = lane < warps ? buf[lane] : 0.0f;
#pragma unroll
  for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

// EPT elements per thread in runs of VEC: run i of thread t starts at
// (t + i blockDim) VEC.  Past the end the values are 0.
template <class A, int VEC, int EPT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
  constexpr int RUNS = EPT / VEC;
  __shared__ float sums[2][32];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const uint16_t *h = p.h + row * p.H;
  float hv[RUNS][VEC];
#pragma unroll
  for (int i = 0; i < RUNS; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * VEC;
    if (c < p.H) {
      load_vec<A, VEC>(h + c, hv[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) hv[i][j] = 0.0f;
    }
  }
  if (p.y) {
    const uint16_t *y = p.y + row * p.H;
    float yv[RUNS][VEC];
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * VEC;
      if (c < p.H) {
        load_vec<A, VEC>(y + c, yv[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) yv[i][j] = 0.0f;
      }
    }
    float r = p.scale;
    if (p.norm_y) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < RUNS; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(yv[i][j], yv[i][j], ss);
      r *= rsqrtf(block_sum(ss, sums[0]) * p.inv_h + p.eps);
    }
    const uint16_t *gate = p.gate ? p.gate + row / p.rows_per_gate * p.gate_cols : nullptr;
    if (gate && p.gate_cols == 1) r *= A::lo(__ldg(gate));
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * VEC;
      if (c >= p.H) continue;
      float f[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = r;
      float q[VEC];
      if (p.w_post) {
        load_vec<A, VEC>(p.w_post + c, q);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] *= q[j];
      }
      if (gate && p.gate_cols != 1) {
        load_vec<A, VEC>(gate + c, q);
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] *= q[j];
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) hv[i][j] = fmaf(f[j], yv[i][j], hv[i][j]);
      if (p.h_out) store_vec<A, VEC>(p.h_out + row * p.H + c, hv[i]);
    }
  }
  if (!p.n_out) return;
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < RUNS; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) ss = fmaf(hv[i][j], hv[i][j], ss);
  const float r = rsqrtf(block_sum(ss, sums[1]) * p.inv_h + p.eps);
#pragma unroll
  for (int i = 0; i < RUNS; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * VEC;
    if (c >= p.H) continue;
    float q[VEC];
    if (p.w_next) {
      load_vec<A, VEC>(p.w_next + c, q);
#pragma unroll
      for (int j = 0; j < VEC; ++j) q[j] = hv[i][j] * r * q[j];
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) q[j] = hv[i][j] * r;
    }
    store_vec<A, VEC>(p.n_out + row * p.H + c, q);
  }
}

template <class A, int VEC>
cudaError_t launch_vec(const NormParams &p, int64_t rows, cudaStream_t stream) {
  // the fewest elements per thread that a CTA of at most 512 threads covers
  const dim3 grid(static_cast<unsigned>(rows));
  const int need8 = (p.H + 7) / 8;
  auto threads = [](int n) { return (n + 31) / 32 * 32; };
  if (need8 <= 256) return launch_on(norm_kernel<A, VEC, 8>, grid, threads(need8), 0, stream, false, p);
  if (need8 <= 1024) return launch_on(norm_kernel<A, VEC, 16>, grid, threads((need8 + 1) / 2), 0, stream, false, p);
  return launch_on(norm_kernel<A, VEC, 32>, grid, threads((need8 + 3) / 4), 0, stream, false, p);
}

template <class A>
cudaError_t launch_act(const NormParams &p, int64_t rows, cudaStream_t stream) {
  // the widest loads that every row's start and every vector allows
  uintptr_t bits = static_cast<uintptr_t>(p.H) * 2;
  for (const void *q : {static_cast<const void *>(p.h), static_cast<const void *>(p.y),
                        static_cast<const void *>(p.w_post), static_cast<const void *>(p.w_next),
                        static_cast<const void *>(p.h_out), static_cast<const void *>(p.n_out),
                        static_cast<const void *>(p.gate)})
    bits |= reinterpret_cast<uintptr_t>(q);
  if (bits % 16 == 0) return launch_vec<A, 8>(p, rows, stream);
  if (bits % 4 == 0) return launch_vec<A, 2>(p, rows, stream);
  return launch_vec<A, 1>(p, rows, stream);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, cudaStream_t stream) {
  NormParams p = {};
  p.h = static_cast<const uint16_t *>(a.h);
  p.y = static_cast<const uint16_t *>(a.y);
  p.w_post = static_cast<const uint16_t *>(a.w_post);
  p.gate = static_cast<const uint16_t *>(a.gate);
  p.w_next = static_cast<const uint16_t *>(a.w_next);
  p.h_out = static_cast<uint16_t *>(a.h_out);
  p.n_out = static_cast<uint16_t *>(a.n_out);
  p.rows_per_gate = a.gate ? a.rows / a.gate_rows : 1;
  p.H = static_cast<int>(a.H);
  p.gate_cols = static_cast<int>(a.gate_cols);
  p.norm_y = a.norm_y;
  p.scale = a.scale;
  p.eps = a.eps;
  p.inv_h = 1.0f / static_cast<float>(a.H);
  return a.act == ActF16::kId ? launch_act<ActF16>(p, a.rows, stream) : launch_act<ActBf16>(p, a.rows, stream);
}

}  // namespace qsw
