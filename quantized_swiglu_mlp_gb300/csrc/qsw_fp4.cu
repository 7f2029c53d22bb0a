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
#include "qsw_tiles.h"

namespace qsw {
namespace {

struct QuantSource {
  const void *x;           // [rows, K] activations
  uint8_t *codes;          // [rows, K/2]
  uint8_t *scales;         // scale blocks
  const int *offsets;      // ragged: [groups + 1] first row of each group
  int64_t rows;            // uniform: rows per group
  int64_t K;
  int64_t k_blocks;        // scale blocks along K
  int groups;
  bool stream;             // too much to stay in L2
};

// 16-bit matrices beyond this many bytes are read and written with streaming
// accesses, so that they do not push the codes out of the 129 MB of L2 (4096 x 14336
// there and back: 68.1 -> 61.6 us); a smaller one may still be there for its reader.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

template <class A, int FMT>
__device__ __forceinline__ void quantize_block(const uint16_t *src, int64_t k0, int64_t K, uint8_t *codes,
                                               uint8_t *scale, const Fp4Scale &q, bool stream) {
  constexpr int B = Fp4<FMT>::kBlock;
  if (k0 >= K) {      // padding of the last scale block
    *scale = 0;
    return;
  }
  uint4 v[B / 8];
#pragma unroll
  for (int i = 0; i < B / 8; ++i) {
    const uint4 *p = reinterpret_cast<const uint4 *>(src + k0) + i;
    v[i] = stream ? __ldcs(p) : __ldg(p);
  }
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
    // the group whose padded row blocks hold this one: a thread looks at each.  Its
    // rows are the product's (raised_offset), which in an ascending table are its own
    // two entries'; a thread walks any other table from the start.  (With the walk as
    // a scan in every CTA, for all tables: 8192 rows of 4096 in 32 groups 3 us longer.)
    __shared__ int found, found_lo, found_hi;
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    const int rows = static_cast<int>(s.rows);
    auto look = [&](int e, int top) {
      const int lo = raised_offset(__ldg(s.offsets + e), top, rows);
      const int hi = raised_offset(__ldg(s.offsets + e + 1), lo, rows);
      const int64_t base = ragged_row_block(lo, e);
      if (base <= block && block < base + ceil_div(hi - lo, kSfRows)) {
        found = e;
        found_lo = lo;
        found_hi = hi;
      }
      return lo;
    };
    bool backward = false;
    for (int e = threadIdx.x; e < s.groups; e += blockDim.x)
      backward |= raised_offset(__ldg(s.offsets + e + 1), 0, rows) < look(e, 0);
    if (__syncthreads_or(backward)) {
      if (threadIdx.x == 0) {
        found = -1;
        for (int e = 0, top = 0; e < s.groups; ++e) top = look(e, top);
      }
      __syncthreads();
    }
    const int e = found;
    if (e < 0) return;
    const int lo = found_lo, hi = found_hi;
    dst = lo + (block - ragged_row_block(lo, e)) * kSfRows + row;
    if (dst >= hi) return;
  } else {
    const int64_t per = (s.rows + kSfRows - 1) / kSfRows;
    const int64_t g = block / per, r = (block - g * per) * kSfRows + row;
    if (r >= s.rows) return;
    dst = g * s.rows + r;
  }
  const uint16_t *src = static_cast<const uint16_t *>(s.x) + dst * s.K;
  uint8_t *codes = s.codes + dst * (s.K / 2);
  uint8_t *scale = s.scales + block * s.k_blocks * kSfBytes + warp * 32 + lane;
  const int64_t first = static_cast<int64_t>(blockIdx.y) * run;
  const int64_t end = first + run < s.k_blocks ? first + run : s.k_blocks;
#pragma unroll 2
  for (int64_t kb = first; kb < end; ++kb)
    quantize_block<A, FMT>(src, (kb * 4 + (lane & 3)) * Fp4<FMT>::kBlock, s.K, codes, scale + kb * kSfBytes, q, s.stream);
}

// The same unit and mapping as the quantiser: a warp reads 32 consecutive scale
// bytes, four lanes read and write consecutive blocks of a row.
template <class A, int FMT>
__global__ void __launch_bounds__(kQuantThreads)
    dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows, int64_t K,
                      int64_t k_blocks, float g, int run, bool stream, uint16_t *__restrict__ out) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int B = Fp4<FMT>::kBlock;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = 2 * warp + (lane >> 4) + 32 * ((lane >> 2) & 3);
  const int64_t block = blockIdx.x;
  const int64_t per = (rows + kSfRows - 1) / kSfRows;
  const int64_t grp = block / per, r = (block - grp * per) * kSfRows + row;
  if (r >= rows) return;
  const int64_t at = grp * rows + r;
  const uint8_t *src = codes + at * (K / 2);
  const uint8_t *scale = scales + block * k_blocks * kSfBytes + warp * 32 + lane;
  const int64_t first = static_cast<int64_t>(blockIdx.y) * run;
  const int64_t end = first + run < k_blocks ? first + run : k_blocks;
#pragma unroll 4
  for (int64_t kb = first; kb < end; ++kb) {
    const int64_t k0 = (kb * 4 + (lane & 3)) * B;
    if (k0 >= K) break;
    const float s = fp4_scale_value<FMT>(__ldg(scale + kb * kSfBytes), g);
    uint32_t w[B / 8];
    if (B == 16) {
      const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + k0 / 2));
      w[0] = v.x;
      w[1] = v.y;
    } else {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + k0 / 2));
      w[0] = v.x;
      w[1] = v.y;
      w[B / 8 - 2] = v.z;
      w[B / 8 - 1] = v.w;
    }
    uint4 *dst = reinterpret_cast<uint4 *>(out + at * K + k0);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) {
      uint32_t h[4];
      fp4_unpack8(w[i], h);
      const uint4 o = make_uint4(A::pack2(ActF16::lo(h[0]) * s, ActF16::hi(h[0]) * s),
                                 A::pack2(ActF16::lo(h[1]) * s, ActF16::hi(h[1]) * s),
                                 A::pack2(ActF16::lo(h[2]) * s, ActF16::hi(h[2]) * s),
                                 A::pack2(ActF16::lo(h[3]) * s, ActF16::hi(h[3]) * s));
      if (stream)
        __stcs(dst + i, o);
      else
        dst[i] = o;
    }
  }
}

// Activations of a mixture of experts: each token's row is quantised once and its
// codes and scales written to the rows of all its experts.  One warp per token and
// run of 32 scales; a lane holds one scale's elements, four lanes a scale block's
// four bytes.  (Quantising each expert's row from the gathered token instead read
// and rounded every token k times: 27 us for 4096 tokens of 2048, k = 8.)
struct FanParams {
  const uint16_t *x;         // [T, K]
  const int *ids, *slots;    // [T, k]
  const int *offsets;        // [E + 1]
  uint8_t *codes, *scales;   // [T k, K/2] and ragged scale blocks
  int64_t T, K, k_blocks;
  int k, E, rows, segments;
};

template <class A, int FMT>
__global__ void __launch_bounds__(256) quantize_fan_kernel(const FanParams p, const Fp4Scale q) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int B = Fp4<FMT>::kBlock;
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int64_t t = w / p.segments;
  if (t >= p.T) return;
  const int64_t j0 = (w - t * p.segments) * 32;       // first scale of the run
  const int64_t k0 = (j0 + lane) * B;
  // lane c's destination: the row of the token's expert c
  int slot = -1;
  int64_t sf_row = 0;
  if (lane < p.k) {
    const int e = __ldg(p.ids + t * p.k + lane);
    slot = __ldg(p.slots + t * p.k + lane);
    if (e >= 0 && e < p.E && slot >= 0 && slot < p.rows) {
      int lo, hi;
      ragged_range(p.offsets, e, p.rows, lo, hi);
      const int local = slot - lo;
      if (local >= 0 && slot < hi)
        sf_row = (ragged_row_block(lo, e) + local / kSfRows) * p.k_blocks * kSfBytes + (local & 31) * 16 +
                 ((local >> 5) & 3) * 4;
      else
        slot = -1;
    } else {
      slot = -1;
    }
  }
  uint32_t byte = 0;
  uint32_t code[B / 8];
  const bool in = k0 < p.K;
  if (in) {
    uint4 v[B / 8];
#pragma unroll
    for (int i = 0; i < B / 8; ++i) v[i] = __ldg(reinterpret_cast<const uint4 *>(p.x + t * p.K + k0) + i);
    uint32_t amax = amax_pairs<A>(v[0], v[1]);
    if (B == 32) amax = max(amax, amax_pairs<A>(v[B / 8 - 2], v[B / 8 - 1]));
    float inv;
    byte = fp4_scale_of<FMT>(amax, q, inv);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) code[i] = fp4_code8<A>(v[i], inv);
  }
  // the four scale bytes of a block in its first lane
  uint32_t word = byte << (8 * (lane & 3));
  word |= __shfl_xor_sync(0xffffffffu, word, 1);
  word |= __shfl_xor_sync(0xffffffffu, word, 2);
  const int64_t kb = j0 / 4 + (lane >> 2);
  for (int c = 0; c < p.k; ++c) {
    const int row = __shfl_sync(0xffffffffu, slot, c);
    const int64_t sf = __shfl_sync(0xffffffffu, sf_row, c);
    if (row < 0) continue;
    if (in) {
      uint8_t *dst = p.codes + static_cast<int64_t>(row) * (p.K / 2) + k0 / 2;
      if (B == 16)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(code[0], code[1]);
      else
        *reinterpret_cast<uint4 *>(dst) = make_uint4(code[0], code[1], code[B / 8 - 2], code[B / 8 - 1]);
    }
    if ((lane & 3) == 0 && kb < p.k_blocks) *reinterpret_cast<uint32_t *>(p.scales + sf + kb * kSfBytes) = word;
  }
}

// Scale blocks per CTA: a grid of a few waves of 4 CTAs per SM.  (Longer runs with
// more loads in flight per thread measured the same: the kernels run at the rate
// of a device copy of their sizes.)
int quant_run(int64_t row_blocks, int64_t k_blocks, int num_sms) {
  const int64_t want = row_blocks * k_blocks / (static_cast<int64_t>(num_sms) * 16);
  return static_cast<int>(want < 1 ? 1 : want > 16 ? 16 : want);
}

template <class A, int FMT, bool RAGGED>
cudaError_t launch_quant(const QuantSource &s, const Fp4Scale &q, int64_t row_blocks, int num_sms,
                         cudaStream_t stream) {
  const int run = quant_run(row_blocks, s.k_blocks, num_sms);
  const dim3 grid(static_cast<unsigned>(row_blocks), static_cast<unsigned>((s.k_blocks + run - 1) / run));
  return launch_on(quantize_kernel<A, FMT, RAGGED>, grid, kQuantThreads, 0, stream, false, s, q, run);
}

template <bool RAGGED>
cudaError_t dispatch_quant(const QuantSource &s, int fmt, int act, float g, int64_t row_blocks,
                           int num_sms, cudaStream_t stream) {
  if (num_sms <= 0) return cudaErrorInvalidDevice;
  const Fp4Scale q = make_fp4_scale(g);
  if (act == ActBf16::kId)
    return fmt == FP4_MX ? launch_quant<ActBf16, FP4_MX, RAGGED>(s, q, row_blocks, num_sms, stream)
                         : launch_quant<ActBf16, FP4_NV, RAGGED>(s, q, row_blocks, num_sms, stream);
  return fmt == FP4_MX ? launch_quant<ActF16, FP4_MX, RAGGED>(s, q, row_blocks, num_sms, stream)
                       : launch_quant<ActF16, FP4_NV, RAGGED>(s, q, row_blocks, num_sms, stream);
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
  s.stream = groups * rows * K * 2 > kStreamBytes;
  return dispatch_quant<false>(s, fmt, act, g, groups * ((rows + kSfRows - 1) / kSfRows), num_sms, stream);
}

cudaError_t launch_fp4_quantize_ragged(const void *x, int64_t rows, int64_t K, const int *offsets, int groups,
                                       int fmt, int act, float g, uint8_t *codes, uint8_t *scales, int num_sms,
                                       cudaStream_t stream) {
  QuantSource s = {};
  s.x = x;
  s.codes = codes;
  s.scales = scales;
  s.offsets = offsets;
  s.rows = rows;
  s.K = K;
  s.k_blocks = fp4_k_blocks(K, fmt);
  s.groups = groups;
  return dispatch_quant<true>(s, fmt, act, g, ragged_row_block(rows, groups), num_sms, stream);
}

cudaError_t launch_fp4_quantize_fan(const void *x, int64_t T, int64_t K, int k, const int *ids, const int *slots,
                                    const int *offsets, int groups, int fmt, int act, float g, uint8_t *codes,
                                    uint8_t *scales, cudaStream_t stream) {
  FanParams p = {};
  p.x = static_cast<const uint16_t *>(x);
  p.ids = ids;
  p.slots = slots;
  p.offsets = offsets;
  p.codes = codes;
  p.scales = scales;
  p.T = T;
  p.K = K;
  p.k_blocks = fp4_k_blocks(K, fmt);
  p.k = k;
  p.E = groups;
  p.rows = static_cast<int>(T * k);
  p.segments = static_cast<int>((p.k_blocks * 4 + 31) / 32);
  const Fp4Scale q = make_fp4_scale(g);
  // few warps: one per CTA, on as many SMs (the expert MLP of 12 tokens: 8 experts of
  // 4096 x 1024 19.1 us with CTAs of a warp, 19.7 with 8; of 48 tokens 20.4 and 19.8)
  const int64_t warps = T * p.segments;
  const int threads = warps < 128 ? 32 : 256;
  const dim3 grid(static_cast<unsigned>((warps * 32 + threads - 1) / threads));
#define QSW_FAN(A, F) launch_on(quantize_fan_kernel<A, F>, grid, threads, 0, stream, false, p, q)
  if (act == ActBf16::kId) return fmt == FP4_MX ? QSW_FAN(ActBf16, FP4_MX) : QSW_FAN(ActBf16, FP4_NV);
  return fmt == FP4_MX ? QSW_FAN(ActF16, FP4_MX) : QSW_FAN(ActF16, FP4_NV);
#undef QSW_FAN
}

cudaError_t launch_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t groups, int64_t rows,
                                  int64_t K, int fmt, int act, float g, void *out, int num_sms, cudaStream_t cs) {
  if (num_sms <= 0) return cudaErrorInvalidDevice;
  const bool stream = groups * rows * K * 2 > kStreamBytes;
  const int64_t kb = fp4_k_blocks(K, fmt), row_blocks = groups * ((rows + kSfRows - 1) / kSfRows);
  const int run = quant_run(row_blocks, kb, num_sms);
  auto *o = static_cast<uint16_t *>(out);
  const dim3 grid(static_cast<unsigned>(row_blocks), static_cast<unsigned>((kb + run - 1) / run));
#define QSW_DEQ(A, F) \
  launch_on(dequantize_kernel<A, F>, grid, kQuantThreads, 0, cs, false, codes, scales, rows, K, kb, g, run, stream, o)
  if (act == ActBf16::kId) return fmt == FP4_MX ? QSW_DEQ(ActBf16, FP4_MX) : QSW_DEQ(ActBf16, FP4_NV);
  return fmt == FP4_MX ? QSW_DEQ(ActF16, FP4_MX) : QSW_DEQ(ActF16, FP4_NV);
#undef QSW_DEQ
}

}  // namespace qsw
