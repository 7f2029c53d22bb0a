// Microscaled 4-bit floating point (e2m1 codes with one scale per block of
// consecutive elements), shared by the quantisation and product kernels.
//
//   QSW_FP4_MX  block of 32, scale 2^(floor(log2 amax) - 2) held as E8M0
//               (2 is the exponent of e2m1's largest value, 6)
//   QSW_FP4_NV  block of 16, scale E4M3(amax / (6 g)); g is one f32 per tensor
//
// An element is the e2m1 value nearest to x / scale (ties to even, saturating
// at 6) times the scale.  A block that holds an infinity or a NaN gets the
// scale NaN, so that everything computed from it is NaN.
//
// Scale bytes are stored the way the tensor core takes them: blocks of 128 rows
// by 4 scales, 512 bytes, row blocks outermost; inside a block row r, scale j
// is byte 16 (r mod 32) + 4 (r / 32) + j.  Row counts are padded to 128 per
// matrix (the padding rows' bytes are never looked at), scale counts to 4 (those
// bytes are 0).
#pragma once

#include "qsw_device.cuh"

namespace qsw {

enum : int { FP4_MX = 0, FP4_NV = 1 };

template <int FMT>
struct Fp4 {
  static constexpr int kBlock = FMT == FP4_MX ? 32 : 16;     // elements per scale
  static constexpr int kSfK = 4 * kBlock;                    // elements per 512-byte scale block
  static constexpr uint32_t kNan = FMT == FP4_MX ? 0xFFu : 0x7Fu;
};

constexpr int kSfRows = 128;
constexpr int kSfBytes = 512;

__host__ __device__ inline int fp4_block(int fmt) { return fmt == FP4_MX ? 32 : 16; }
__host__ __device__ inline int64_t fp4_k_blocks(int64_t K, int fmt) {
  return (K + 4 * fp4_block(fmt) - 1) / (4 * fp4_block(fmt));
}

// First row block of group e when rows [off, next off) of a matrix sorted by
// group each start a new row block: non-overlapping for any group sizes,
// without a scan over the groups, and at most rows / 128 + groups in all.
__host__ __device__ __forceinline__ int64_t ragged_row_block(int64_t off, int e) {
  return (off + kSfRows - 1) / kSfRows + e;
}

// Rows [lo, hi) of group e of an ascending table, clamped so that no other one leads
// outside the rows.
__device__ __forceinline__ void ragged_range(const int *offsets, int e, int rows, int &lo, int &hi) {
  lo = min(max(__ldg(offsets + e), 0), rows);
  hi = min(max(__ldg(offsets + e + 1), lo), rows);
}

// The tensor's scale g with the reciprocal that the scale of a block is
// computed with (f32 of 1 / (6 g)).
struct Fp4Scale {
  float g;
  float rcp6g;
};
inline Fp4Scale make_fp4_scale(float g) {
  return Fp4Scale{g, static_cast<float>(1.0 / (6.0 * static_cast<double>(g)))};
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xffffu)));
}

// The scale byte of a block whose largest magnitude has the f32 bits `amax`,
// and the factor its elements are multiplied with before rounding to e2m1.  The
// factor is 0 where the scale is 0 or below the normal range, and in NaN blocks.
template <int FMT>
__device__ __forceinline__ uint32_t fp4_scale_of(uint32_t amax, const Fp4Scale &q, float &inv) {
  inv = 0.0f;
  if (amax >= 0x7F800000u) return Fp4<FMT>::kNan;
  if (FMT == FP4_MX) {
    const uint32_t e = amax >> 23;              // biased exponent; subnormals end at scale 2^-127
    const uint32_t byte = e > 2 ? e - 2 : 0;
    inv = __uint_as_float((254u - byte) << 23);   // 2^(127 - byte), byte <= 252
    return byte;
  }
  uint16_t byte;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(byte) : "f"(0.0f), "f"(__uint_as_float(amax) * q.rcp6g));
  const float s = e4m3_to_f32(byte) * q.g;
  if (s >= 1.17549435e-38f) inv = __frcp_rn(s);
  return byte;
}

// The f32 value of a scale byte (times g).
template <int FMT>
__device__ __forceinline__ float fp4_scale_value(uint32_t byte, float g) {
  if (FMT == FP4_MX) {
    if (byte == 0xFFu) return __uint_as_float(0x7FC00000u);
    return byte ? __uint_as_float(byte << 23) : __uint_as_float(0x00400000u);   // 2^(byte - 127)
  }
  return e4m3_to_f32(byte) * g;
}

// Eight f32 -> eight e2m1 codes, element i at bits 4i.
__device__ __forceinline__ uint32_t fp4_pack8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t3, %8, %7;\n\t"
      "mov.b32 %0, {t0, t1, t2, t3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Four e2m1 pairs of a word -> f16 pairs (exact).
__device__ __forceinline__ void fp4_unpack8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 t0, t1, t2, t3;\n\t"
      "mov.b32 {t0, t1, t2, t3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, t1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, t2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, t3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Largest magnitude of eight 16-bit words of pairs, as f32 bits.  Magnitudes of
// either activation type order like their bits, NaN above infinity.
template <class A>
__device__ __forceinline__ uint32_t amax_pairs(const uint4 &a, const uint4 &b) {
  constexpr uint32_t m = 0x7FFF7FFFu;
  const uint32_t x = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
  const uint32_t y = __vmaxu2(__vmaxu2(b.x & m, b.y & m), __vmaxu2(b.z & m, b.w & m));
  const uint32_t z = __vmaxu2(x, y);
  return __float_as_uint(A::lo(__vmaxu2(z, z >> 16)));
}

// Eight activations (four pairs) times `inv`, as e2m1 codes.
template <class A>
__device__ __forceinline__ uint32_t fp4_code8(const uint4 &w, float inv) {
  const float v[8] = {A::lo(w.x) * inv, A::hi(w.x) * inv, A::lo(w.y) * inv, A::hi(w.y) * inv,
                      A::lo(w.z) * inv, A::hi(w.z) * inv, A::lo(w.w) * inv, A::hi(w.w) * inv};
  return fp4_pack8(v);
}

// Launch on `stream`; `dependent`: as a programmatic dependent of the work
// before it (the kernel waits with griddep_wait before touching its results);
// `cluster`: CTAs per cluster.
template <class... P, class... Q>
inline cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, int cluster, int threads, size_t smem,
                                   cudaStream_t stream, bool dependent, Q... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}
template <class... P, class... Q>
inline cudaError_t launch_on(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                             bool dependent, Q... args) {
  return launch_clusters(kernel, grid, 1, threads, smem, stream, dependent, args...);
}

}  // namespace qsw
