// Norms around a block, one pass over the rows (HBM-bound):
//
//   z  = y rsqrt(mean y^2 + eps) w_post           the block's output, normed
//   h' = h + scale gate z                         residual
//   n  = h' rsqrt(mean h'^2 + eps) w_next         the next block's input
//
// Any of the three may be left out (see qsw_post_norm and qsw_rms_norm).  A CTA
// holds a row in registers as f32: both means are sums over those registers, and
// n is computed from h' before it is rounded for storing.
#include "qsw_fp4.cuh"
#include "qsw_internal.h"

namespace qsw {
namespace {

struct NormParams {
  const uint16_t *h, *y, *w_post, *gate, *w_next;
  uint16_t *h_out, *n_out;
  int64_t rows;
  int64_t rows_per_gate;   // rows that share a row of the gate
  int H;
  int gate_cols;           // H, or 1: one gate value per gate row
  int norm_y;
  int stream;              // more rows than stay in L2
  float scale, eps, inv_h;
};

// VEC consecutive 16-bit values as they are stored.
template <int VEC>
struct Raw {
  uint32_t w[(VEC + 1) / 2];
};

// `once`: a row's value, which is not read again (evicted first from L2).
template <int VEC>
__device__ __forceinline__ Raw<VEC> load_raw(const uint16_t *p, bool once = false) {
  Raw<VEC> r;
  if constexpr (VEC == 8) {
    const uint4 q = once ? __ldcs(reinterpret_cast<const uint4 *>(p)) : *reinterpret_cast<const uint4 *>(p);
    r.w[0] = q.x;
    r.w[1] = q.y;
    r.w[2] = q.z;
    r.w[3] = q.w;
  } else if constexpr (VEC == 2) {
    r.w[0] = *reinterpret_cast<const uint32_t *>(p);
  } else {
    r.w[0] = *p;
  }
  return r;
}

template <class A, int VEC>
__device__ __forceinline__ float value(const Raw<VEC> &r, int j) {
  return (j & 1) ? A::hi(r.w[j >> 1]) : A::lo(r.w[j >> 1]);
}

template <class A, int VEC>
__device__ __forceinline__ void store_vec(uint16_t *p, const float (&v)[VEC], bool stream) {
  if constexpr (VEC == 8) {
    const uint4 q = make_uint4(A::pack2(v[0], v[1]), A::pack2(v[2], v[3]), A::pack2(v[4], v[5]), A::pack2(v[6], v[7]));
    if (stream)
      __stcs(reinterpret_cast<uint4 *>(p), q);
    else
      *reinterpret_cast<uint4 *>(p) = q;
  } else if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t *>(p) = A::pack2(v[0], v[1]);
  else
    *p = A::store(v[0]);
}

// Sum over the CTA.  `buf` rotates over the row's parity and sum, so that one
// barrier per sum is enough.
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
// (t + i blockDim) VEC.  Past the end the values are 0.  A CTA walks the rows
// with a stride of the grid; while it works on one, the next one's h and y are on
// their way, and the weights stay in registers.  (With a CTA per row, the row's
// loads, two block sums and stores came one after the other and each row read the
// weights again: 57.4 us for 8192 rows of 4096; a device copy of as many bytes takes
// 47 us.)
template <class A, int VEC, int EPT>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
  constexpr int RUNS = EPT / VEC;
  // The next row and the weights in registers, where 64 hold them or spill little: 16 elements
  // spill up to 100 bytes a thread and still gain over many rows (2048 rows, bf16: H = 16384 58.8 us,
  // without 63.1; 12288 49.7 and 52.4; 8200 44.7 and 42.5), but not as single values, a
  // register each (H = 12001: 329 us and 928 bytes, without 114).
  constexpr bool kAhead = EPT <= 8 || (EPT <= 16 && VEC > 1);
  __shared__ float sums[4][32];
  griddep_wait();
  griddep_launch_dependents();
  const int first = threadIdx.x * VEC, step = blockDim.x * VEC;
  const Raw<VEC> zero = {};
  auto load_row = [&](const uint16_t *base, int64_t row, Raw<VEC>(&r)[RUNS]) {
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      const int c = first + i * step;
      r[i] = c < p.H ? load_raw<VEC>(base + row * p.H + c, p.stream) : zero;
    }
  };
  Raw<VEC> wp[kAhead ? RUNS : 1], wn[kAhead ? RUNS : 1];
  Raw<VEC> h_next[RUNS], y_next[RUNS];
  int64_t row = blockIdx.x;
  if (kAhead) {
    load_row(p.h, row, h_next);
    if (p.y) load_row(p.y, row, y_next);
    if (p.w_post) load_row(p.w_post, 0, reinterpret_cast<Raw<VEC>(&)[RUNS]>(wp));
    if (p.w_next) load_row(p.w_next, 0, reinterpret_cast<Raw<VEC>(&)[RUNS]>(wn));
  }
  int parity = 0;
  for (; row < p.rows; row += gridDim.x, parity ^= 2) {
    float hv[RUNS][VEC];
    Raw<VEC> y[RUNS];
    if (!kAhead) {
      load_row(p.h, row, h_next);
      if (p.y) load_row(p.y, row, y_next);
    }
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      y[i] = y_next[i];
#pragma unroll
      for (int j = 0; j < VEC; ++j) hv[i][j] = value<A, VEC>(h_next[i], j);
    }
    if (kAhead && row + gridDim.x < p.rows) {
      load_row(p.h, row + gridDim.x, h_next);
      if (p.y) load_row(p.y, row + gridDim.x, y_next);
    }
    if (p.y) {
      const uint16_t *gate = p.gate ? p.gate + row / p.rows_per_gate * p.gate_cols : nullptr;
      float r = p.scale;
      if (gate && p.gate_cols == 1) r *= A::lo(__ldg(gate));
      if (p.norm_y) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < RUNS; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) ss = fmaf(value<A, VEC>(y[i], j), value<A, VEC>(y[i], j), ss);
        r *= rsqrtf(block_sum(ss, sums[parity]) * p.inv_h + p.eps);
      }
#pragma unroll
      for (int i = 0; i < RUNS; ++i) {
        const int c = first + i * step;
        if (c >= p.H) continue;
        float f[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) f[j] = r;
        if (p.w_post) {
          const Raw<VEC> w = kAhead ? wp[kAhead ? i : 0] : load_raw<VEC>(p.w_post + c);
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[j] *= value<A, VEC>(w, j);
        }
        if (gate && p.gate_cols != 1) {
          const Raw<VEC> w = load_raw<VEC>(gate + c);
#pragma unroll
          for (int j = 0; j < VEC; ++j) f[j] *= value<A, VEC>(w, j);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) hv[i][j] = fmaf(f[j], value<A, VEC>(y[i], j), hv[i][j]);
        if (p.h_out) store_vec<A, VEC>(p.h_out + row * p.H + c, hv[i], p.stream);
      }
    }
    if (!p.n_out) continue;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < RUNS; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss = fmaf(hv[i][j], hv[i][j], ss);
    const float r = rsqrtf(block_sum(ss, sums[parity + 1]) * p.inv_h + p.eps);
#pragma unroll
    for (int i = 0; i < RUNS; ++i) {
      const int c = first + i * step;
      if (c >= p.H) continue;
      float q[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) q[j] = hv[i][j] * r;
      if (p.w_next) {
        const Raw<VEC> w = kAhead ? wn[kAhead ? i : 0] : load_raw<VEC>(p.w_next + c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) q[j] *= value<A, VEC>(w, j);
      }
      store_vec<A, VEC>(p.n_out + row * p.H + c, q, p.stream);
    }
  }
}

template <class A, int VEC>
cudaError_t launch_vec(const NormParams &p, int num_sms, cudaStream_t stream) {
  // 8 elements per thread, 16 and 32 where 1024 threads need them (rows of 4096:
  // 512 threads of 8 take 51.5 us for 8192 of them, 256 threads of 16 take 53.0);
  // as many CTAs as 64 registers a thread let run at once
  const int need8 = (p.H + 7) / 8;
  const int ept = need8 <= 1024 ? 8 : need8 <= 2048 ? 16 : 32;
  const int threads = ((p.H + ept - 1) / ept + 31) / 32 * 32;
  const int64_t most = static_cast<int64_t>(num_sms) * (1024 / threads);
  const dim3 grid(static_cast<unsigned>(p.rows < most ? p.rows : most));
  if (ept == 8) return launch_on(norm_kernel<A, VEC, 8>, grid, threads, 0, stream, false, p);
  if (ept == 16) return launch_on(norm_kernel<A, VEC, 16>, grid, threads, 0, stream, false, p);
  return launch_on(norm_kernel<A, VEC, 32>, grid, threads, 0, stream, false, p);
}

template <class A>
cudaError_t launch_act(const NormParams &p, int num_sms, cudaStream_t stream) {
  // the widest loads that every row's start and every vector allows
  uintptr_t bits = static_cast<uintptr_t>(p.H) * 2;
  for (const void *q : {static_cast<const void *>(p.h), static_cast<const void *>(p.y),
                        static_cast<const void *>(p.w_post), static_cast<const void *>(p.w_next),
                        static_cast<const void *>(p.h_out), static_cast<const void *>(p.n_out),
                        static_cast<const void *>(p.gate)})
    bits |= reinterpret_cast<uintptr_t>(q);
  if (bits % 16 == 0) return launch_vec<A, 8>(p, num_sms, stream);
  if (bits % 4 == 0) return launch_vec<A, 2>(p, num_sms, stream);
  return launch_vec<A, 1>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_norm(const NormArgs &a, int num_sms, cudaStream_t stream) {
  if (num_sms <= 0) return cudaErrorInvalidDevice;
  NormParams p = {};
  p.h = static_cast<const uint16_t *>(a.h);
  p.y = static_cast<const uint16_t *>(a.y);
  p.w_post = static_cast<const uint16_t *>(a.w_post);
  p.gate = static_cast<const uint16_t *>(a.gate);
  p.w_next = static_cast<const uint16_t *>(a.w_next);
  p.h_out = static_cast<uint16_t *>(a.h_out);
  p.n_out = static_cast<uint16_t *>(a.n_out);
  p.rows = a.rows;
  p.rows_per_gate = a.gate ? a.rows / a.gate_rows : 1;
  p.H = static_cast<int>(a.H);
  p.gate_cols = static_cast<int>(a.gate_cols);
  p.norm_y = a.norm_y;
  p.scale = a.scale;
  p.eps = a.eps;
  p.inv_h = 1.0f / static_cast<float>(a.H);
  // rows, twice in and twice out, against the L2's 129 MB: streaming accesses take 8192
  // rows of 4096 from 53.4 to 51.5 us; what fits stays for its reader
  p.stream = a.rows * a.H * 8 > int64_t(128) << 20;
  return a.act == ActF16::kId ? launch_act<ActF16>(p, num_sms, stream) : launch_act<ActBf16>(p, num_sms, stream);
}

}  // namespace qsw
