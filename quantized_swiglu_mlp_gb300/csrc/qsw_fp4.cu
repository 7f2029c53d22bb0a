// Quantisation of activations and weights to microscaled 4-bit floating point,
// and back.  Both are HBM-bound: 2 + 0.5 + 1/block bytes per element.
//
// The quantiser's unit is one 512-byte scale block, 128 rows by 4 scales.  Lane l
// of warp w holds the scale at byte 32 w + l of the block -- row 2w + l/16 +
// 32 ((l/4) mod 4), scale l mod 4 -- so that a warp's scale bytes are one 32-byte
// sector, four lanes read 4 consecutive blocks of a row (128 or 256
// contiguous bytes) and write 32 or 64 contiguous bytes of codes, and no value
// crosses a lane.
#include "qsw_fp4.cuh"
#include "qsw_internal.h"

namespace qsw {
namespace {

struct QuantSource {
  const void *x;           // [rows, K] activations
  uint8_t *codes;          // [rows, K/2]
  uint8_t *scales;         // scale blocks
  const int *offsets;      // ragged: [groups + 1] first row of each group
  const int *order;        // ragged: row r of the result is row order[r] / fan of x; null: row r
  int fan;
  int64_t rows;            // uniform: rows per group
  int64_t K;
  int64_t k_blocks;        // scale blocks along K
  int groups;
};

template <class A, int FMT>
__device__ __forceinline__ void quantize_block(const uint16_t *src, int64_t k0, int64_t K, uint8_t *codes,
                                               uint8_t *scale, const Fp4Scale &q) {
  constexpr int B = Fp4<FMT>::kBlock;
  if (k0 >= K) {      // padding of the last scale block
    *scale = 0;
    return;
  }
  uint4 v[B / 8];
#pragma unroll
  for (int i = 0; i < B / 8; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(src + k0) + i);
  uint32_t amax = amax_pairs<A>(v[0], v[1]);
  if (B == 32) amax = max(amax, amax_pairs<A>(v[B / 8 - 2], v[B / 8 - 1]));
  float inv;
  *scale = static_cast<uint8_t>(fp4_scale_of<FMT>(amax, q, inv));
  if (B == 16) {
    *reinterpret_cast<uint2 *>(codes + k0 / 2) = make_uint2(fp4_code8<A>(v[0], inv), fp4_code8<A>(v[1], inv));
  } else {
    *reinterpret_cast<uint4 *>(codes + k0 / 2) =
        make_uint4(fp4_code8<A>(v[0], inv), fp4_code8<A>(v[1], inv), fp4_code8<A>(v[B / 8 - 2], inv),
                   fp4_code8<A>(v[B / 8 - 1], inv));
  }
}

constexpr int kQuantThreads = 512;

// Grid: x = row blocks over all groups, y = runs of `run` scale blocks along K.
template <class A, int FMT, bool RAGGED>
__global__ void __launch_bounds__(kQuantThreads) quantize_kernel(const QuantSource s, const Fp4Scale q, int run) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = 2 * warp + (lane >> 4) + 32 * ((lane >> 2) & 3);   // row within the block
  const int64_t block = blockIdx.x;
  int64_t dst;            // row of the result, -1: none
  if (RAGGED) {
    // the group whose padded row blocks hold this one: one thread per group looks
    __shared__ int found;
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    const int rows = static_cast<int>(s.rows);
    int lo, hi;
    for (int e = threadIdx.x; e < s.groups; e += blockDim.x) {
      ragged_range(s.offsets, e, rows, lo, hi);
      const int64_t base = ragged_row_block(lo, e);
      if (base <= block && block < base + (hi - lo + kSfRows - 1) / kSfRows) found = e;
    }
    __syncthreads();
    const int e = found;
    if (e < 0) return;
    ragged_range(s.offsets, e, rows, lo, hi);
    dst = lo + (block - ragged_row_block(lo, e)) * kSfRows + row;
    if (dst >= hi) return;
  } else {
    const int64_t per = (s.rows + kSfRows - 1) / kSfRows;
    const int64_t g = block / per, r = (block - g * per) * kSfRows + row;
    if (r >= s.rows) return;
    dst = g * s.rows + r;
  }
  const int64_t from = RAGGED && s.order ? __ldg(s.order + dst) / s.fan : dst;
  const uint16_t *src = static_cast<const uint16_t *>(s.x) + from * s.K;
  uint8_t *codes = s.codes + dst * (s.K / 2);
  uint8_t *scale = s.scales + block * s.k_blocks * kSfBytes + warp * 32 + lane;
  const int64_t first = static_cast<int64_t>(blockIdx.y) * run;
  const int64_t end = first + run < s.k_blocks ? first + run : s.k_blocks;
#pragma unroll 2
  for (int64_t kb = first; kb < end; ++kb)
    quantize_block<A, FMT>(src, (kb * 4 + (lane & 3)) * Fp4<FMT>::kBlock, s.K, codes, scale + kb * kSfBytes, q);
}

template <class A, int FMT>
__global__ void __launch_bounds__(256) dequantize_kernel(const uint8_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales, int64_t rows, int64_t K,
                                                         int64_t k_blocks, int64_t n, float g, uint16_t *out) {
  griddep_wait();
  griddep_launch_dependents();
  // one thread per 16 elements (one scale of either format)
  const uint32_t per_row = static_cast<uint32_t>(K / 16);
  const int64_t row_blocks = (rows + kSfRows - 1) / kSfRows;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / per_row;
    const int c = static_cast<int>(i - row * per_row);
    const int64_t grp = row / rows;
    const int64_t r = row - grp * rows;
    const int j = c * 16 / Fp4<FMT>::kBlock;
    const int rb = static_cast<int>(r % kSfRows);
    const uint32_t byte = __ldg(scales + ((grp * row_blocks + r / kSfRows) * k_blocks + j / 4) * kSfBytes +
                                (rb & 31) * 16 + (rb >> 5) * 4 + (j & 3));
    const float s = fp4_scale_value<FMT>(byte, g);
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(codes) + i);
    uint32_t h[4];
    uint32_t o[8];
    fp4_unpack8(w.x, h);
#pragma unroll
    for (int t = 0; t < 4; ++t) o[t] = A::pack2(ActF16::lo(h[t]) * s, ActF16::hi(h[t]) * s);
    fp4_unpack8(w.y, h);
#pragma unroll
    for (int t = 0; t < 4; ++t) o[4 + t] = A::pack2(ActF16::lo(h[t]) * s, ActF16::hi(h[t]) * s);
    uint4 *dst = reinterpret_cast<uint4 *>(out + i * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <class A, int FMT, bool RAGGED>
cudaError_t launch_quant(const QuantSource &s, const Fp4Scale &q, int64_t row_blocks, int threads, int num_sms,
                         cudaStream_t stream, bool dependent) {
  // runs long enough that the grid is a few waves of 4 CTAs per SM
  const int64_t want = row_blocks * s.k_blocks / (static_cast<int64_t>(num_sms) * 16);
  const int run = static_cast<int>(want < 1 ? 1 : want > 16 ? 16 : want);
  const dim3 grid(static_cast<unsigned>(row_blocks), static_cast<unsigned>((s.k_blocks + run - 1) / run));
  return launch_on(quantize_kernel<A, FMT, RAGGED>, grid, threads, 0, stream, dependent, s, q, run);
}

template <bool RAGGED>
cudaError_t dispatch_quant(const QuantSource &s, int fmt, int act, float g, int64_t row_blocks, int threads,
                           int num_sms, cudaStream_t stream, bool dependent) {
  const Fp4Scale q = make_fp4_scale(g);
  if (act == ActBf16::kId)
    return fmt == FP4_MX ? launch_quant<ActBf16, FP4_MX, RAGGED>(s, q, row_blocks, threads, num_sms, stream, dependent)
                         : launch_quant<ActBf16, FP4_NV, RAGGED>(s, q, row_blocks, threads, num_sms, stream, dependent);
  return fmt == FP4_MX ? launch_quant<ActF16, FP4_MX, RAGGED>(s, q, row_blocks, threads, num_sms, stream, dependent)
                       : launch_quant<ActF16, FP4_NV, RAGGED>(s, q, row_blocks, threads, num_sms, stream, dependent);
}

}  // namespace

cudaError_t launch_fp4_quantize(const void *x, int64_t groups, int64_t rows, int64_t K, int fmt, int act, float g,
                                uint8_t *codes, uint8_t *scales, int num_sms, cudaStream_t stream) {
  QuantSource s = {};
  s.x = x;
  s.codes = codes;
  s.scales = scales;
  s.rows = rows;
  s.K = K;
  s.k_blocks = fp4_k_blocks(K, fmt);
  s.groups = static_cast<int>(groups);
  // a warp serves rows 2w, 2w + 1 of each 32: fewer rows need fewer warps
  const int threads = rows < 32 ? static_cast<int>((rows + 1) / 2) * 32 : kQuantThreads;
  return dispatch_quant<false>(s, fmt, act, g, groups * ((rows + kSfRows - 1) / kSfRows), threads, num_sms, stream,
                               false);
}

cudaError_t launch_fp4_quantize_ragged(const void *x, int64_t rows, int64_t K, const int *offsets, int groups,
                                       const int *order, int fan, int fmt, int act, float g, uint8_t *codes,
                                       uint8_t *scales, int num_sms, cudaStream_t stream, bool dependent) {
  QuantSource s = {};
  s.x = x;
  s.codes = codes;
  s.scales = scales;
  s.offsets = offsets;
  s.order = order;
  s.fan = fan;
  s.rows = rows;
  s.K = K;
  s.k_blocks = fp4_k_blocks(K, fmt);
  s.groups = groups;
  return dispatch_quant<true>(s, fmt, act, g, ragged_row_block(rows, groups), kQuantThreads, num_sms, stream,
                              dependent);
}

cudaError_t launch_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t groups, int64_t rows,
                                  int64_t K, int fmt, int act, float g, void *out, int num_sms, cudaStream_t stream) {
  const int64_t n = groups * rows * (K / 16);
  int64_t blocks = (n + 255) / 256;
  const int64_t cap = static_cast<int64_t>(num_sms) * 16;
  if (blocks > cap) blocks = cap;
  const int64_t kb = fp4_k_blocks(K, fmt);
  auto *o = static_cast<uint16_t *>(out);
  const dim3 grid(static_cast<unsigned>(blocks));
#define QSW_DEQ(A, F) launch_on(dequantize_kernel<A, F>, grid, 256, 0, stream, false, codes, scales, rows, K, kb, n, g, o)
  if (act == ActBf16::kId) return fmt == FP4_MX ? QSW_DEQ(ActBf16, FP4_MX) : QSW_DEQ(ActBf16, FP4_NV);
  return fmt == FP4_MX ? QSW_DEQ(ActF16, FP4_MX) : QSW_DEQ(ActF16, FP4_NV);
#undef QSW_DEQ
}

}  // namespace qsw
