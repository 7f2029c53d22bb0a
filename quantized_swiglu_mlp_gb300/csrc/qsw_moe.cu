// The router of a mixture of experts and the combination of its experts' rows.
//
// topk_kernel: per token the k largest logits (the lowest index first among
// equals) and their weights.  Selection looks at the logits themselves -- softmax
// and sigmoid keep their order -- so it is exact whatever the exponential does.
// sort_kernel: the stable counting sort of the (token, choice) pairs by expert.
// route_small_kernel: both, for few tokens.
// combine_kernel: y[t] = T(sum_j weights[t, j] rows[slots[t, j]] (+ residual[t])),
// each token summing its own rows in order: no atomics, the same bits every time.
#include "qsw_fp4.cuh"
#include "qsw_internal.h"

namespace qsw {
namespace {

constexpr int kTopkWarps = 8;
constexpr float kNoScore = -700.0f;   // logits up to this one have the sigmoid 0: masks of any type's lowest value

template <class L>
__device__ __forceinline__ float load_logit(const L *p);
template <>
__device__ __forceinline__ float load_logit<float>(const float *p) { return __ldg(p); }
template <>
__device__ __forceinline__ float load_logit<ActBf16>(const ActBf16 *p) {
  return ActBf16::lo(__ldg(reinterpret_cast<const unsigned short *>(p)));
}
template <>
__device__ __forceinline__ float load_logit<ActF16>(const ActF16 *p) {
  return ActF16::lo(__ldg(reinterpret_cast<const unsigned short *>(p)));
}

// A float's bits in an order-preserving unsigned form that is never 0; NaN
// counts as -infinity, -0 as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) v = -INFINITY;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

struct RouteParams {
  const void *logits;
  int64_t T;
  int E, k, scoring, renormalize;
  float scale;
  int *ids;
  float *weights;
  int *offsets, *slots, *order;
};

// One warp per token t; lane l holds experts l, l + 32, ... (PER of them).  Each of
// the k rounds takes the warp's largest key and, among its holders, the lowest
// index (key 0: taken or past the end).  Returns lane j's choice j.
template <class L, int PER>
__device__ __forceinline__ int topk_row(const RouteParams &p, int64_t t) {
  const int lane = threadIdx.x & 31;
  const int E = p.E, k = p.k, scoring = p.scoring, renormalize = p.renormalize;
  const L *logits = static_cast<const L *>(p.logits);
  const int wide = static_cast<int>(sizeof(L) == 4 ? 1 : 0);
  const uint8_t *row = reinterpret_cast<const uint8_t *>(logits) + t * E * (wide ? 4 : 2);
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < E ? order_key(load_logit<L>(reinterpret_cast<const L *>(row + e * (wide ? 4 : 2)))) : 0u;
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = max(top, key[i]);
  top = __reduce_max_sync(0xffffffffu, top);
  const float peak = key_value(top);
  const bool none = peak == -INFINITY;      // every logit masked: all weights 0
  float sum = 0.0f;
  if (scoring == QSW_ROUTE_SOFTMAX && !renormalize) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const float v = key_value(key[i]);
      if (key[i]) sum += v == peak ? 1.0f : expf(v - peak);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  }
  // sigmoid scores that are only looked at for their ratios, all below 1/2: e^-peak
  // times as large, so that none that counts is lost below f32's range
  const float far = renormalize && peak < 0.0f ? peak : 0.0f;
  // round j's choice stays with lane j
  float mine = 0.0f;
  int id = 0;
  for (int j = 0; j < k; ++j) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xffffffffu, best);
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i)
      if (key[i] == best) at = lane + 32 * i;
    at = __reduce_min_sync(0xffffffffu, at);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at == lane + 32 * i) key[i] = 0;
    const float v = key_value(best);
    float p;
    if (scoring == QSW_ROUTE_SIGMOID)
      p = v > 0.0f ? 1.0f / (1.0f + expf(-v)) : v > kNoScore ? expf(v - far) / (1.0f + expf(v)) : 0.0f;
    else
      p = none ? 0.0f : v == peak ? 1.0f : expf(v - peak);
    if (lane == j) {
      mine = p;
      id = at;
    }
    if (renormalize) sum += p;
  }
  if (lane < k) {
    float w = mine;
    if (scoring == QSW_ROUTE_SOFTMAX || renormalize) w = sum > 0.0f ? mine / sum : 0.0f;
    p.ids[t * k + lane] = id;
    p.weights[t * k + lane] = w * p.scale;
  }
  return id;
}

template <class L, int PER>
__global__ void __launch_bounds__(kTopkWarps * 32) topk_kernel(const RouteParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kTopkWarps + (threadIdx.x >> 5);
  if (t < p.T) topk_row<L, PER>(p, t);
}

// Few tokens: choices and sort in one CTA and one launch.  The ids stay in shared
// memory; thread i places pair i, counting the pairs of smaller experts and those
// of its own before it.  (64 experts, k = 8, one launch and two: 1 token 2.9 and 3.9
// us, 8 tokens 3.6 and 4.1, 12 tokens 4.1 both, 32 tokens 8.0 and 4.1.)
constexpr int kSmallPairs = 64;
template <class L, int PER>
__global__ void __launch_bounds__(1024) route_small_kernel(const RouteParams p) {
  __shared__ int ids[kSmallPairs];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, n = static_cast<int>(p.T) * p.k;
  for (int t = threadIdx.x >> 5; t < static_cast<int>(p.T); t += blockDim.x >> 5) {
    const int id = topk_row<L, PER>(p, t);
    if (lane < p.k) ids[t * p.k + lane] = id;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = ids[i];
    int at = 0;
    for (int j = 0; j < n; ++j) at += ids[j] < e || (ids[j] == e && j < i);
    p.slots[i] = at;
    p.order[at] = i;
  }
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
    int at = 0;
    for (int j = 0; j < n; ++j) at += ids[j] < e;
    p.offsets[e] = at;
  }
}

constexpr int kSortThreads = 1024;

// One CTA per expert e.  Each warp takes a contiguous run of the n = T k ids, 128
// at a time, four consecutive ones per lane: the ballots of id == e and the count
// of id < e give, summed over the warps, the expert's first row and the run's place
// in it, and the ballots again each match's rank, so that rows are in the order of
// the pairs.  The ballots of up to 32 groups stay in registers of the lane of that
// number (n <= 131072); longer runs are read a second time.  Ids outside [0, E) are
// ignored (their slot is -1).  Bound by the latency of the loads, so 8 of 16 bytes are
// in flight.  `wide`: ids starts at a 16-byte boundary.  The ids are not read through
// the read-only path: the kernel that writes them may still run when this one starts.
__global__ void __launch_bounds__(kSortThreads)
    sort_kernel(const int *ids, int n, int E, bool wide, int *offsets, int *slots, int *order) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ int warp_eq[32], warp_lt[32];
  const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int groups = (n + 127) / 128;
  const int per = (groups + warps - 1) / warps;
  const int g0 = min(warp * per, groups), g1 = min(g0 + per, groups);
  auto load = [&](int g) {
    const int i = g * 128 + lane * 4;
    if (wide && g < g1 && i + 4 <= n) return *reinterpret_cast<const int4 *>(ids + i);
    int v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = g < g1 && i + c < n ? ids[i + c] : E;   // neither equal nor below
    return make_int4(v[0], v[1], v[2], v[3]);
  };
  constexpr int AHEAD = 8;      // loads in flight: a ballot waits for its own
  uint32_t kept[4] = {};
  int eq = 0, lt = 0;
  for (int g = g0; g < g1; g += AHEAD) {
    int4 v[AHEAD];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) v[a] = load(g + a);
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      if (g + a >= g1) break;
      const int id[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t match = __ballot_sync(0xffffffffu, id[c] == e);
        if (((g + a - g0) & 31) == lane) kept[c] = match;
        eq += __popc(match);
        lt += id[c] >= 0 && id[c] < e;
      }
    }
    if (e == 0) {       // one CTA marks the pairs of no expert
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        const int id[4] = {v[a].x, v[a].y, v[a].z, v[a].w};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int i = (g + a) * 128 + lane * 4 + c;
          if ((id[c] < 0 || id[c] >= E) && g + a < g1 && i < n) slots[i] = -1;
        }
      }
    }
  }
  lt = __reduce_add_sync(0xffffffffu, lt);
  if (lane == 0) {
    warp_eq[warp] = eq;
    warp_lt[warp] = lt;
  }
  __syncthreads();
  const int o_eq = lane < warps ? warp_eq[lane] : 0, o_lt = lane < warps ? warp_lt[lane] : 0;
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? o_eq : 0);
  const int total = __reduce_add_sync(0xffffffffu, o_eq);
  const int first = __reduce_add_sync(0xffffffffu, o_lt);
  if (threadIdx.x == 0) {
    offsets[e] = first;
    if (e == E - 1) offsets[E] = first + total;
  }
  int at = first + before;
  auto place = [&](int g, const uint32_t(&match)[4]) {
    int pos = at;                              // of this lane's first match
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      pos += __popc(match[c] & ((1u << lane) - 1u));
      at += __popc(match[c]);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (((match[c] >> lane) & 1u) == 0) continue;
      const int i = g * 128 + lane * 4 + c;
      slots[i] = pos;
      order[pos++] = i;
    }
  };
  if (per <= 32) {
    // only the groups with a match
    for (uint32_t left = __ballot_sync(0xffffffffu, (kept[0] | kept[1] | kept[2] | kept[3]) != 0); left;
         left &= left - 1) {
      const int a = __ffs(left) - 1;
      uint32_t match[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) match[c] = __shfl_sync(0xffffffffu, kept[c], a);
      place(g0 + a, match);
    }
  } else {
    for (int g = g0; g < g1; ++g) {
      const int4 v = load(g);
      const uint32_t match[4] = {__ballot_sync(0xffffffffu, v.x == e), __ballot_sync(0xffffffffu, v.y == e),
                                 __ballot_sync(0xffffffffu, v.z == e), __ballot_sync(0xffffffffu, v.w == e)};
      place(g, match);
    }
  }
}

// Eight columns of an expert's row.  Read once, so evicted first (4096 tokens of 2048, k = 8:
// the expert MLP took 224.5 us with ordinary loads, 216.6 so).  Not through the read-only path: the
// products that write the rows may still run when this kernel starts.
struct Eight {
  float4 v[2];
  __device__ __forceinline__ void load(const float *p) {
    v[0] = __ldcs(reinterpret_cast<const float4 *>(p));
    v[1] = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ float value(int i) const {
    const float4 &q = v[i >> 2];
    return (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  }
};

// One warp, a CTA, per token and run of 256 columns; 8 columns per lane.  The rows of
// eight choices are on their way before the first is added.
template <class A>
__global__ void __launch_bounds__(32)
    combine_kernel(const float *rows, int64_t n_rows, const int *__restrict__ slots, const float *__restrict__ weights,
                   const uint16_t *residual, int k, int64_t H, int chunks, uint16_t *y) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int AHEAD = 8;
  const int lane = threadIdx.x;
  const int64_t t = blockIdx.x / chunks;
  const int64_t h = (blockIdx.x - t * chunks) * 256 + lane * 8;
  // lane j holds choice j
  int slot = -1;
  float weight = 0.0f;
  if (lane < k) {
    slot = __ldg(slots + t * k + lane);
    weight = __ldg(weights + t * k + lane);
    if (slot >= n_rows) slot = -1;
  }
  const bool in = h < H;
  float acc[8] = {};
  if (residual && in) {
    const uint4 v = *reinterpret_cast<const uint4 *>(residual + t * H + h);
    const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = A::lo(q[i]);
      acc[2 * i + 1] = A::hi(q[i]);
    }
  }
  for (int j0 = 0; j0 < k; j0 += AHEAD) {
    Eight v[AHEAD] = {};
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int s = __shfl_sync(0xffffffffu, slot, (j0 + a) & 31);
      if (j0 + a < k && s >= 0 && in) v[a].load(rows + static_cast<int64_t>(s) * H + h);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const float g = __shfl_sync(0xffffffffu, weight, (j0 + a) & 31);
      const int s = __shfl_sync(0xffffffffu, slot, (j0 + a) & 31);
      if (j0 + a >= k || s < 0) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = fmaf(g, v[a].value(i), acc[i]);
    }
  }
  if (in)
    *reinterpret_cast<uint4 *>(y + t * H + h) = make_uint4(A::pack2(acc[0], acc[1]), A::pack2(acc[2], acc[3]),
                                                          A::pack2(acc[4], acc[5]), A::pack2(acc[6], acc[7]));
}

template <class L, int PER>
cudaError_t launch_route(const RouteParams &p, cudaStream_t stream) {
  const int64_t n = p.T * p.k;
  if (n <= kSmallPairs) {
    const int warps = p.T < 1 ? 1 : p.T > 32 ? 32 : static_cast<int>(p.T);
    const int threads = warps * 32 > p.E ? warps * 32 : (p.E + 31) / 32 * 32;
    return launch_on(route_small_kernel<L, PER>, dim3(1), threads, 0, stream, false, p);
  }
  const dim3 grid(static_cast<unsigned>((p.T + kTopkWarps - 1) / kTopkWarps));
  const cudaError_t e = launch_on(topk_kernel<L, PER>, grid, kTopkWarps * 32, 0, stream, false, p);
  if (e != cudaSuccess) return e;
  // 64 experts, k = 8, both launches with 256 and 1024 sorting threads: 512 tokens 4.6
  // and 5.9 us, 2048 tokens 8.1 and 7.5, 16384 tokens 63 and 31
  const int threads = n >= 16384 ? kSortThreads : 256;
  const bool wide = reinterpret_cast<uintptr_t>(p.ids) % 16 == 0;
  return launch_on(sort_kernel, dim3(static_cast<unsigned>(p.E)), threads, 0, stream, true, p.ids, static_cast<int>(n),
                   p.E, wide, p.offsets, p.slots, p.order);
}

template <class L>
cudaError_t launch_route_of(const RouteParams &p, cudaStream_t stream) {
  if (p.E <= 32) return launch_route<L, 1>(p, stream);
  if (p.E <= 64) return launch_route<L, 2>(p, stream);
  if (p.E <= 128) return launch_route<L, 4>(p, stream);
  if (p.E <= 256) return launch_route<L, 8>(p, stream);
  if (p.E <= 512) return launch_route<L, 16>(p, stream);
  return launch_route<L, 32>(p, stream);
}

}  // namespace

cudaError_t launch_moe_route(const void *logits, int logit_dtype, int64_t T, int E, int k, int scoring,
                             int renormalize, float scale, int *ids, float *weights, int *offsets, int *slots,
                             int *order, cudaStream_t stream) {
  const RouteParams p = {logits, T, E, k, scoring, renormalize, scale, ids, weights, offsets, slots, order};
  if (logit_dtype == QSW_LOGITS_F32) return launch_route_of<float>(p, stream);
  return logit_dtype == QSW_ACT_BF16 ? launch_route_of<ActBf16>(p, stream) : launch_route_of<ActF16>(p, stream);
}

cudaError_t launch_moe_combine(const float *rows, int64_t n_rows, const int *slots, const float *weights,
                               const void *residual, int64_t T, int k, int64_t H, int act, void *y,
                               cudaStream_t stream, bool dependent) {
  const int chunks = static_cast<int>((H + 255) / 256);
  // CTAs of a warp, on as many SMs as there are (the expert MLP of 64 tokens, 8 of 64 experts
  // of 2048 x 1024: 46.7 us, with CTAs of 8 warps 47.8; of 1024 tokens 75.3 and 77.6, of 16384
  // 706 and 738)
  const dim3 grid(static_cast<unsigned>(T * chunks));
  const auto *res = static_cast<const uint16_t *>(residual);
  auto *o = static_cast<uint16_t *>(y);
  return launch_on(act == ActF16::kId ? combine_kernel<ActF16> : combine_kernel<ActBf16>, grid, 32, 0, stream,
                   dependent, rows, n_rows, slots, weights, res, k, H, chunks, o);
}

}  // namespace qsw
