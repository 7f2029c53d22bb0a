// Rotary positions, and appending keys and values to a paged cache with the
// rotation on the way (HBM-bound):
//
//   angle a = position f_i,  f_i the angle per position of pair i < rot / 2
//   y0 = s (x0 cos a - x1 sin a),  y1 = s (x1 cos a + x0 sin a)
//
// with (x0, x1) the elements (i, i + rot/2) of a head or (2i, 2i + 1); elements from
// `rot` on are copied.  Far positions: an angle of 10^5 rad in f32 is off by 0.004.
// Here f_i is held as a fraction of a turn in 64 fractional bits, so that position *
// f_i modulo 2^64 is the fraction of a turn exactly, and its upper 32 bits go through
// sincospif: the angle is within 2^-23 rad of the exact one at any position.
//
// A CTA takes a few tokens, whose units its threads walk: 8 pairs as two 16-byte runs half a
// rotation apart, or two runs of 8 elements.  cos and sin are worked out once per token
// and pair, while the first units are on their way, and all heads find them in shared memory.
// 8192 tokens of 32 heads of 128 (134 MB) take 24 us, 5.6 TB/s; a device copy of as many bytes 21.2.
#include "qsw_fp4.cuh"
#include "qsw_internal.h"

namespace qsw {
namespace {

// n / d for n < 2^31 and 1 <= d < 2^31 as one multiplication: (n m) >> 32 >> shift with
// m = ceil(2^(32 + shift) / d) (Granlund and Montgomery).
struct FastDiv {
  uint32_t d, m, shift;
};
FastDiv make_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;          // 2^s >= d
  // 2^(32 + s - 1) / d fits in 32 bits and serves n < 2^31
  const uint32_t shift = s ? s - 1 : 0;
  const uint64_t m = ((uint64_t(1) << (32 + shift)) + d - 1) / d;
  return FastDiv{d, d == 1 ? 0u : static_cast<uint32_t>(m), shift};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
  return f.d == 1 ? n : __umulhi(n, f.m) >> f.shift;
}

// Heads of one tensor: where they come from and go to.
struct Segment {
  const uint16_t *src;
  uint16_t *dst;
  int64_t src_t, src_h;          // strides in elements
  int64_t dst_t, dst_h;          // strides; of a cache, page (dst_t), head and row strides
  int64_t dst_r;
  int heads;
  int rotate;
  int paged;
  FastDiv per_head;              // units of a head
};

struct RopeParams {
  Segment seg[3];
  int segments;
  int first_unit[4];             // of each segment within a token, and their number
  const int *positions;          // null: all 0
  const int *slots;
  const int64_t *table;
  int T, D, half;                // half: pairs
  int groups, turns;             // of 8 pairs, and 8 for each: of a token in shared memory
  int tokens;                    // per CTA
  int interleaved;
  int skip_negative;             // tokens at negative positions are left out
  int pages;
  float scale;
  FastDiv per_token, page_size, halves;
};

constexpr int kThreads = 256;
constexpr int kAhead = 4;          // units of a thread in flight

// Where the cos and sin of a token's pair lie: one after the other; with runs of 8 elements,
// pairs 2 j and 2 j + 1 of all groups of 8 side by side, so that neighbouring threads, each with a
// group, read neighbouring words (in order, four of them shared a bank: an append of 7363 tokens, 181
// MB, took 42 us, so 36).
template <int VEC>
__device__ __forceinline__ int turn_at(const RopeParams &p, int pair) {
  return VEC == 1 ? pair : (((pair & 7) >> 1) * p.groups + (pair >> 3)) * 2 + (pair & 1);
}

// Two runs of VEC elements.
template <int VEC>
struct Unit {
  uint32_t w[2][VEC == 8 ? 4 : 1];   // as they are stored
  uint16_t *dst;                     // the head's first element; null: nothing to do
  int turn;                          // where its token's and first pair's turns lie in shared memory
  int e0, e1;                        // elements of the runs; e1 < 0: one run
  int kind;                          // 0: copied; 1: pairs across the runs; 2, 3: adjacent pairs in the first, in both
};

// Unit u of the CTA's tokens [t0, ..): where it goes, and the loads of what it holds.
template <int VEC>
__device__ __forceinline__ void fetch_unit(const RopeParams &p, int t0, uint32_t u, uint32_t units, Unit<VEC> &x) {
  x.dst = nullptr;
  if (u >= units) return;
  const uint32_t tl = div_by(u, p.per_token);
  const int t = t0 + static_cast<int>(tl);
  int r = static_cast<int>(u - tl * p.per_token.d);
  const int g = (p.segments > 1 && r >= p.first_unit[1]) + (p.segments > 2 && r >= p.first_unit[2]);
  const Segment &s = p.seg[g];
  r -= p.first_unit[g];
  const uint32_t h = div_by(static_cast<uint32_t>(r), s.per_head);
  const int c = r - static_cast<int>(h * s.per_head.d);
  x.kind = 0;
  x.turn = static_cast<int>(tl) * p.turns;
  // across: pairs half a rotation apart, and element by element any pairs
  const bool across = s.rotate && (VEC == 1 || !p.interleaved);
  if (across && c * VEC < p.half) {
    const int pair = c * VEC;
    x.e0 = p.interleaved ? 2 * pair : pair;
    x.e1 = p.interleaved ? 2 * pair + 1 : pair + p.half;
    x.turn += turn_at<VEC>(p, pair);
    x.kind = 1;
  } else {
    // (behind the rotation, if there are units across)
    x.e0 = across ? 2 * p.half + (c * VEC - p.half) * 2 : c * VEC * 2;
    x.e1 = x.e0 + VEC < p.D ? x.e0 + VEC : -1;
    if (s.rotate && !across && x.e0 < 2 * p.half) {
      x.turn += turn_at<VEC>(p, x.e0 / 2);
      x.kind = x.e0 + VEC < 2 * p.half ? 3 : 2;
    }
  }
  // (before the token's slot is looked at: the loads need not wait for it)
  const uint16_t *src = s.src + t * s.src_t + h * s.src_h;
  if constexpr (VEC == 8) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(src + x.e0));
    x.w[0][0] = a.x, x.w[0][1] = a.y, x.w[0][2] = a.z, x.w[0][3] = a.w;
    if (x.e1 >= 0) {
      const uint4 b = __ldcs(reinterpret_cast<const uint4 *>(src + x.e1));
      x.w[1][0] = b.x, x.w[1][1] = b.y, x.w[1][2] = b.z, x.w[1][3] = b.w;
    }
  } else {
    x.w[0][0] = src[x.e0];
    if (x.e1 >= 0) x.w[1][0] = src[x.e1];
  }
  const bool left_out = p.skip_negative && p.positions && __ldg(p.positions + t) < 0;
  uint16_t *d;
  if (s.paged) {
    const int slot = __ldg(p.slots + t);
    const uint32_t page = div_by(static_cast<uint32_t>(max(slot, 0)), p.page_size);
    d = slot < 0 || page >= static_cast<uint32_t>(p.pages)
            ? nullptr
            : s.dst + page * s.dst_t + (slot - page * p.page_size.d) * s.dst_r + h * s.dst_h;
  } else {
    d = s.dst + t * s.dst_t + h * s.dst_h;
  }
  x.dst = left_out ? nullptr : d;
}

// Adjacent pairs of a run of 8.
template <class A>
__device__ __forceinline__ void turn_run(uint32_t (&w)[4], const float2 *cs, int groups) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 f = reinterpret_cast<const float4 *>(cs)[j * groups];      // cos, sin, cos, sin
    const float a0 = A::lo(w[2 * j]), a1 = A::hi(w[2 * j]), b0 = A::lo(w[2 * j + 1]), b1 = A::hi(w[2 * j + 1]);
    w[2 * j] = A::pack2(a0 * f.x - a1 * f.y, a1 * f.x + a0 * f.y);
    w[2 * j + 1] = A::pack2(b0 * f.z - b1 * f.w, b1 * f.z + b0 * f.w);
  }
}

// Turns and stores a unit.
template <class A, int VEC>
__device__ __forceinline__ void store_unit(const float2 *turn, int groups, Unit<VEC> &x) {
  if (!x.dst) return;
  const float2 *cs = turn + x.turn;
  if constexpr (VEC == 8) {
    if (x.kind == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 f = reinterpret_cast<const float4 *>(cs)[j * groups];
        const float a0 = A::lo(x.w[0][j]), a1 = A::hi(x.w[0][j]);
        const float b0 = A::lo(x.w[1][j]), b1 = A::hi(x.w[1][j]);
        x.w[0][j] = A::pack2(a0 * f.x - b0 * f.y, a1 * f.z - b1 * f.w);
        x.w[1][j] = A::pack2(b0 * f.x + a0 * f.y, b1 * f.z + a1 * f.w);
      }
    } else {
      if (x.kind >= 2) turn_run<A>(x.w[0], cs, groups);
      if (x.kind == 3) turn_run<A>(x.w[1], cs + 4 * groups, groups);
    }
    *reinterpret_cast<uint4 *>(x.dst + x.e0) = make_uint4(x.w[0][0], x.w[0][1], x.w[0][2], x.w[0][3]);
    if (x.e1 >= 0) *reinterpret_cast<uint4 *>(x.dst + x.e1) = make_uint4(x.w[1][0], x.w[1][1], x.w[1][2], x.w[1][3]);
  } else if (x.kind == 1) {
    const float2 f = *cs;
    const float x0 = A::lo(x.w[0][0]), x1 = A::lo(x.w[1][0]);
    x.dst[x.e0] = A::store(x0 * f.x - x1 * f.y);
    x.dst[x.e1] = A::store(x1 * f.x + x0 * f.y);
  } else {
    x.dst[x.e0] = static_cast<uint16_t>(x.w[0][0]);
    if (x.e1 >= 0) x.dst[x.e1] = static_cast<uint16_t>(x.w[1][0]);
  }
}

template <class A, int VEC>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) float2 turn[];       // [tokens][turns]: cos, sin
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * p.tokens;
  const int count = min(p.tokens, p.T - t0);
  const uint32_t units = static_cast<uint32_t>(count) * p.per_token.d;
  Unit<VEC> x[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) fetch_unit(p, t0, threadIdx.x + a * kThreads, units, x[a]);
  if (p.half) {
    for (uint32_t i = threadIdx.x; i < static_cast<uint32_t>(count * p.half); i += kThreads) {
      const uint32_t t = div_by(i, p.halves), pair = i - t * p.half;
      const uint64_t at = static_cast<uint64_t>(static_cast<int64_t>(p.positions ? __ldg(p.positions + t0 + t) : 0)) *
                          static_cast<uint64_t>(__ldg(p.table + pair));
      float s, c;
      sincospif(static_cast<float>(static_cast<int32_t>(at >> 32)) * 0x1p-31f, &s, &c);
      turn[t * p.turns + turn_at<VEC>(p, static_cast<int>(pair))] = make_float2(c * p.scale, s * p.scale);
    }
    __syncthreads();
  }
  for (uint32_t u0 = threadIdx.x;;) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) store_unit<A>(turn, p.groups, x[a]);
    u0 += kThreads * kAhead;
    if (u0 >= units) break;
#pragma unroll
    for (int a = 0; a < kAhead; ++a) fetch_unit(p, t0, u0 + a * kThreads, units, x[a]);
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, int num_sms, cudaStream_t stream) {
  if (num_sms <= 0) return cudaErrorInvalidDevice;
  RopeParams p = {};
  p.positions = a.positions;
  p.slots = a.slots;
  p.table = a.table;
  p.T = static_cast<int>(a.T);
  p.D = static_cast<int>(a.D);
  p.half = static_cast<int>(a.rot / 2);
  p.interleaved = a.interleaved;
  p.skip_negative = a.slots != nullptr;
  p.pages = static_cast<int>(a.cache.pages);
  p.scale = a.scale;
  // 16-byte runs where every row, run and half allows
  uintptr_t bits = static_cast<uintptr_t>(a.D) * 2;
  if (p.half) bits |= static_cast<uintptr_t>(a.interleaved ? a.rot : p.half) * 2;
  auto add = [&](const void *src, int64_t st, int64_t sh, void *dst, int64_t dt, int64_t dh, int64_t dr, int64_t heads,
                 int rotate, int paged) {
    Segment &s = p.seg[p.segments++];
    s.src = static_cast<const uint16_t *>(src);
    s.dst = static_cast<uint16_t *>(dst);
    s.src_t = st, s.src_h = sh, s.dst_t = dt, s.dst_h = dh, s.dst_r = dr;
    s.heads = static_cast<int>(heads);
    s.rotate = rotate && p.half;
    s.paged = paged;
    bits |= reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
            static_cast<uintptr_t>((st | sh | dt | dh | dr) * 2);
  };
  if (a.q.data)
    add(a.q.data, a.q.token_stride, a.q.head_stride, a.out, a.out_token_stride, a.out_head_stride, 0, a.heads, 1, 0);
  if (a.slots) {
    const qsw_kv_cache &c = a.cache;
    add(a.k.data, a.k.token_stride, a.k.head_stride, c.k, c.k_strides[0], c.k_strides[1], c.k_strides[2], c.kv_heads, 1,
        1);
    add(a.v.data, a.v.token_stride, a.v.head_stride, c.v, c.v_strides[0], c.v_strides[1], c.v_strides[2], c.kv_heads, 0,
        1);
    p.page_size = make_div(static_cast<uint32_t>(c.page_size));
  }
  const bool wide = bits % 16 == 0;
  const int vec = wide ? 8 : 1;
  int units = 0;
  for (int i = 0; i < p.segments; ++i) {
    Segment &s = p.seg[i];
    const int across = s.rotate && (!p.interleaved || !wide) ? p.half : 0;
    const int per = across / vec + (p.D - 2 * across + 2 * vec - 1) / (2 * vec);
    s.per_head = make_div(static_cast<uint32_t>(per));
    p.first_unit[i] = units;
    units += per * s.heads;
  }
  p.per_token = make_div(static_cast<uint32_t>(units));
  p.halves = make_div(static_cast<uint32_t>(p.half ? p.half : 1));
  p.groups = (p.half + 7) / 8;
  p.turns = p.groups * 8;
  // as many tokens a CTA as its threads hold in one go, where there are CTAs enough; their turns
  // 32 KB at most
  int64_t tokens = kThreads * kAhead / units;
  const int64_t fair = a.T / (2 * static_cast<int64_t>(num_sms)), most = p.turns ? 4096 / p.turns : 16;
  tokens = tokens > fair ? fair : tokens;
  tokens = tokens > most ? most : tokens;
  tokens = tokens < 1 ? 1 : tokens > 16 ? 16 : tokens;
  p.tokens = static_cast<int>(tokens);
  const dim3 grid(static_cast<unsigned>((a.T + tokens - 1) / tokens));
  const size_t smem = static_cast<size_t>(tokens) * p.turns * sizeof(float2);
  const bool f16 = a.act == ActF16::kId;
  if (wide)
    return f16 ? launch_on(rope_kernel<ActF16, 8>, grid, kThreads, smem, stream, false, p)
               : launch_on(rope_kernel<ActBf16, 8>, grid, kThreads, smem, stream, false, p);
  return f16 ? launch_on(rope_kernel<ActF16, 1>, grid, kThreads, smem, stream, false, p)
             : launch_on(rope_kernel<ActBf16, 1>, grid, kThreads, smem, stream, false, p);
}

}  // namespace qsw
