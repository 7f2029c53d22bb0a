// Attention over a paged cache for many rows per kv head, on the tensor core
// (qsw_attention.cuh):
//
//   S = Q K^T      tile of 128 rows by 128 keys, f32 in tensor memory
//   P = 2^(scale log2(e) S - base)     one pass with a running base per row, in registers,
//                                      back to tensor memory in the activation type
//   O = O + P V    f32 in tensor memory
//
// An item is 256 rows: two tiles of 128 rows that share K and V and take turns, so that one
// tile's softmax runs under the other's products.  (Where a head's rows are 128 or fewer and items
// many, two kv heads make an item, a row tile and keys of its own each.)  12 warps: warps 0-3 and 4-7 each own a
// row tile (a thread per row: row maximum and sum need no exchange), warp 8 issues the
// products, warps 9 and 10 copy K and V pages by TMA (a box per page, or per 8 to 128 rows
// of one; a page outside the cache is a coordinate outside the tensor and reads zeros), warp
// 11 works out the items ahead.
// P lies where S was: the products that read P and overwrite S run in the order of issue.
//
// What bounds it (GB300): the products.  A step of two row tiles and 128 keys is four products of
// 128 x 128 x 128, 2048 cycles at the full rate and about 2480 as measured alone, since S takes
// both operands from shared memory, at all it delivers.  A prompt of 8192 tokens with 32 heads of 128
// takes 337 us, 1.63 PFLOP/s.  (Two tiles of 64 rows, or one tile and the keys of two, would
// read K and V twice as often.)
//
// The base of a row is raised (and O rescaled in tensor memory) only when a score passes
// it by 8, so that weights reach 256 at most and most tiles leave O alone; in f16 it lies 7 below the
// score that raised it and weights reach 2^15.
#include <type_traits>

#include "qsw_attention.cuh"

namespace qsw {

namespace {

__device__ unsigned int g_attn_error;

constexpr int kRows = 128;            // of a tile
constexpr int kKeys = 128;
constexpr int kThreads = 384;
constexpr int kWarpMma = 8, kWarpK = 9, kWarpV = 10, kWarpItems = 11;
constexpr int kItems = 4;             // items worked out ahead
constexpr int kItemReaders = 11;      // warps that read them
constexpr float kRaise = 8.0f, kTileLift = 7.0f;

template <int DP>
struct Shape {
  static constexpr int kHalves = DP / 64;                    // 128-byte columns of a tile
  static constexpr int kHalfBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;    // 128 rows of K, V or Q
  static constexpr int kKStages = DP == 128 ? 2 : 4;
  static constexpr int kVStages = DP == 128 ? 3 : 4;
  static constexpr int kStages = kKStages + kVStages;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + 1024;
};

// D[tmem] (+)= A[tmem] . B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of V as the B operand with the columns contiguous (keys are the product's
// K): blocks of 64 columns by 8 keys, 128-byte swizzle; the next 8 keys 1024 bytes on, the
// next 64 columns a half on.
__device__ __forceinline__ uint64_t v_desc(uint32_t smem_addr, uint32_t half_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(half_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,"
      "%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// (a, b) * (c, c) + (d, d), and sums, two at a time.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The item of a CTA's step: every second wave in reverse, since items come longest first.
__device__ __forceinline__ int item_of(int step) {
  const int G = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  return step * G + ((step & 1) ? G - 1 - c : c);
}

// Of N consecutive lanes with N pieces each, lane i gets piece i of all (pieces in the
// lanes' order).
template <int N>
__device__ __forceinline__ void turn_rows(uint4 (&v)[N], int lane) {
#pragma unroll
  for (int m = N / 2; m; m >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i & m) continue;
      const bool up = lane & m;
      const uint4 give = up ? v[i] : v[i | m];
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, give.x, m);
      got.y = __shfl_xor_sync(0xffffffffu, give.y, m);
      got.z = __shfl_xor_sync(0xffffffffu, give.z, m);
      got.w = __shfl_xor_sync(0xffffffffu, give.w, m);
      if (up)
        v[i] = got;
      else
        v[i | m] = got;
    }
}

struct Barriers {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t mma_done;
};

// A reader's place in the ring of items; the item it is at stays until it moves on.
struct ItemCursor {
  uint32_t at = 0;
  // Waits for the next item; null at the end, or when given up.
  __device__ __forceinline__ const Item *next(Barriers &bar, const Item *items, volatile int *abort, uint64_t timeout_ns,
                                              unsigned int *err) {
    const uint32_t slot = at % kItems;
    if (!wait_all(&bar.item_full[slot], (at / kItems) & 1, abort, timeout_ns, err)) return nullptr;
    ++at;
    return items[slot].rows > 0 ? items + slot : nullptr;
  }
  // The item before the last `ahead` ones is no longer needed.
  __device__ __forceinline__ void done(Barriers &bar, uint32_t ahead) {
    __syncwarp();
    if (lane_id() == 0) mbar_arrive(&bar.item_empty[(at - 1 - ahead) % kItems]);
  }
};

__device__ __forceinline__ int tiles_of_item(const Item *t) { return (t->k1 - t->k0 + kKeys - 1) / kKeys; }

// The odd values taken out of the tiles of all items of the CTA, for the rows of one warp (of four of
// a row tile): once the row tiles are through with them and no other warp waits.
template <class A>
__device__ __noinline__ void add_odd_values(const AttnParams &p, int tile, int quarter, int total) {
#pragma unroll 1
  for (int step = 0, id; (id = item_of(step)) < total; ++step) {
    const Item t = find_item(p, id);
    const int first = (t.pair ? 0 : tile * kRows) + quarter * 32, kv_head = t.head + (t.pair ? tile : 0);
    if (t.rows > first) add_odd<A>(p, t, kv_head, first, min(t.rows - first, 32));
  }
}

template <class A, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tiles_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CacheMaps maps) {
  using S = Shape<DP>;
  constexpr int KS = S::kKStages, VS = S::kVStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *q_smem = smem, *k_smem = smem + 2 * S::kTileBytes, *v_smem = k_smem + KS * S::kTileBytes;
  __shared__ Barriers bar;
  __shared__ Item items[kItems];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ int taken;          // values were taken out of V
  volatile int *abort_flag = &abort_word;
  unsigned int *err = &g_attn_error;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  griddep_wait();
  griddep_launch_dependents();
  // (often there are no such sequences: nothing to set up then)
  const int total = __ldg(p.plan.head + LIST_TILES);
  if (item_of(0) >= total) return;
  if constexpr (kDebugBounds) debug_poison_smem(smem, (2 + S::kStages) * S::kTileBytes);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.k_full[i], 1);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], 1);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 4);
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_half[i], 4);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.o_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&bar.item_full[i], 1);
      mbar_init(&bar.item_empty[i], kItemReaders);
    }
    mbar_init(&bar.mma_done, 1);
    abort_word = taken = 0;
    fence_mbar_init();
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  fence_proxy_async_smem();      // (debug build: the fill, before the copies)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  if constexpr (kDebugBounds) {
    // every column := NaN before the first product (a warp per lane quarter)
    if (warp < 4) {
      uint32_t nan16[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) nan16[i] = ~0u;
      for (uint32_t col = 0; col < 512; col += 16) tmem_st16(tmem + (static_cast<uint32_t>(warp) << 21) + col, nan16);
      tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  // Tensor memory: S (and P) of the two row tiles, then O of both.
  const uint32_t o_col = 256;

  if (warp < 8) {
    // ------------------------------------------------------------- softmax --
    // (2 x 224 + 56 = 3 x 168, the registers of the launch; with 208 some of a row's values spilled)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int tile = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;      // this warp's 32 lanes
    const uint32_t s_addr = tmem + lanes + tile * 128, o_addr = tmem + lanes + o_col + tile * DP;
    const int r = (warp & 3) * 32 + lane;                              // row of the tile
    uint8_t *q_tile = q_smem + tile * S::kTileBytes;
    uint32_t s_count = 0, o_count = 0, v_count = 0;
    const float scale = p.scale_log2;

    // The tile's first row and kv head: 128 rows on, or the pair's other head.
    auto row_base = [&](const Item *t) { return t->pair ? 0 : tile * kRows; };
    auto kv_head = [&](const Item *t) { return t->head + (t->pair ? tile : 0); };
    // The tile's rows of an item, from q into shared memory as the products take them: this
    // warp's 32, a row to 16 (8) lanes.
    auto load_q = [&](const Item *t) {
      constexpr int CH = DP / 8, PER = 32 / CH;      // lanes of a row, rows at once
      const int x = row_base(t) + r;
      int64_t token;
      int head, pos;
      row_of(p, *t, kv_head(t), x < t->rows ? x : 0, token, head, pos);
      const uint64_t row = x < t->rows ? reinterpret_cast<uint64_t>(p.q + token * p.q_t + head * p.q_h) : 0;
      const int c = lane % CH;
#pragma unroll
      for (int i = 0; i < 32 / PER; ++i) {
        const int from = i * PER + lane / CH, y = (warp & 3) * 32 + from;
        const uint64_t src = __shfl_sync(0xffffffffu, row, from);
        const bool ok = src != 0 && c * 8 < p.D;
        const uint32_t dst = smem_u32(q_tile + (c >> 3) * S::kHalfBytes + y * 128 + (((c ^ y) & 7) << 4));
        const void *at = ok ? reinterpret_cast<const uint16_t *>(src) + c * 8 : p.q;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(at), "r"(ok ? 16u : 0u) : "memory");
      }
    };
    auto q_loaded = [&] {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full[tile]);
    };
    auto needs_q = [&](const Item *t) { return t->rows > row_base(t) && t->k1 > t->k0; };

    ItemCursor cursor;
    const Item *t = cursor.next(bar, items, abort_flag, p.timeout_ns, err);
    if (t && needs_q(t)) {
      load_q(t);
      q_loaded();
    }
    bool ok = true;
    while (t) {
      const int n = tiles_of_item(t);
      const int base_row = row_base(t), mine = t->rows - base_row;      // live rows of the tile
      const int v_tiles = t->pair ? 2 * n : n;
      const Item *after = nullptr;
      if (mine <= 0) {
        v_count += v_tiles;
        after = cursor.next(bar, items, abort_flag, p.timeout_ns, err);
        if (after && needs_q(after)) {
          load_q(after);
          q_loaded();
        }
        cursor.done(bar, 1);
        t = after;
        continue;
      }
      const bool live = r < mine, warp_live = (warp & 3) * 32 < mine;
      int64_t token;
      int head, pos;
      row_of(p, *t, kv_head(t), live ? base_row + r : 0, token, head, pos);
      // keys that the row sees, from the item's first on: [lo, hi); a row of nobody all, so that
      // it asks for no mask
      const int hi = live ? min(pos + 1, t->k1) - t->k0 : INT_MAX;
      const int lo = live && p.window ? pos - p.window + 1 - t->k0 : 0;
      float base = live ? -INFINITY : 0.0f, sum = 0.0f;
      for (int i = 0; i < n; ++i, ++s_count) {
        const int key0 = t->k0 + i * kKeys;
        if (!(ok = wait_all(&bar.s_full[tile], s_count & 1, abort_flag, p.timeout_ns, err))) break;
        tc_fence_after();
        if (i == n - 1) {
          // the last scores are out: the next item's rows of q take the place of these
          after = cursor.next(bar, items, abort_flag, p.timeout_ns, err);
          if (after && needs_q(after)) load_q(after);
        }
        if ((t->pair || tile == 0) && !all_seen(*t, key0, kKeys)) {
          // rows of V that no row of the item sees, or not every one, may hold anything: a weight of 0
          // does not take out infinities or NaN.  (Before both tiles' products: tile 0's go
          // first; of a pair, each has its own.)
          const uint32_t at = v_count + (t->pair ? 2 * i + tile : i);
          if (!(ok = wait_all(&bar.v_full[at % VS], (at / VS) & 1, abort_flag, p.timeout_ns, err))) break;
          const int key = key0 + r;
          uint8_t *v = v_smem + (at % VS) * S::kTileBytes + r * 128;
          // (neighbouring lanes in different banks)
          auto piece = [&](int c) {
            return reinterpret_cast<uint4 *>(v + (c >> 3) * S::kHalfBytes + (((c ^ r) & 7) << 4));
          };
          if (key >= t->k1 || key < t->first) {
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) *piece(c) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          } else if (!all_seen(*t, key, 1)) {
            uint32_t sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) Odd<A>::gather(*piece(c), sum);
            if (Odd<A>::of(sum[0]) | Odd<A>::of(sum[1])) {
#pragma unroll 1
              for (int c = 0; c < DP / 8; ++c) *piece(c) = Odd<A>::without(*piece(c));
              taken = 1;
              fence_proxy_async_smem();
            }
          }
        }
        if (warp_live) {
          float s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + c * 32, reinterpret_cast<uint32_t *>(s) + c * 32);
          tmem_ld_wait();
          const int h = hi - i * kKeys, l = lo - i * kKeys;
          if (!__all_sync(0xffffffffu, h >= kKeys && l <= 0)) {
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = c < h && c >= l ? s[c] : -INFINITY;
          }
          float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < 124; c += 8)
#pragma unroll
            for (int x = 0; x < 4; ++x) top[x] = max3(top[x], s[c + 2 * x], s[c + 2 * x + 1]);
          top[0] = max3(top[0], s[124], s[125]);
          top[1] = max3(top[1], s[126], s[127]);
          const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]) * scale;
          const float lift = lift_of<A>(most, kTileLift);
          const bool raise = most - base > kRaise + lift;      // (false between infinities of one sign)
          if (__any_sync(0xffffffffu, raise)) {
            const float now = raise ? most - lift : base;
            const float shrink = raise ? ex2(base - now) : 1.0f;
            base = now;
            sum *= shrink;
            if (i > 0) {
#pragma unroll 1
              for (int c = 0; c < DP; c += 16) {
                uint32_t o[16];
                tmem_ld16(o_addr + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * shrink);
                tmem_st16(o_addr + c, o);
              }
            }
          }
          const float off = base == -INFINITY ? 0.0f : -base;
          const uint64_t scale2 = pair(scale, scale), off2 = pair(off, off);
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < 128; c += 32) {
            uint32_t w[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              float a, b;
              unpair(fma2(pair(s[c + 2 * x], s[c + 2 * x + 1]), scale2, off2), a, b);
              a = ex2(a);
              b = ex2(b);
              sums[x & 1] = add2(sums[x & 1], pair(a, b));
              w[x] = A::pack2(a, b);     // the weights as the products take them
            }
            tmem_st16(s_addr + c / 2, w);
            if (c == 32) {
              // half of the weights: their products start under the other half's exponentials
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bar.p_half[tile]);
            }
          }
          float a, b, c, d;
          unpair(sums[0], a, b);
          unpair(sums[1], c, d);
          sum += (a + b) + (c + d);
          tmem_st_wait();
        } else {
          // (all lanes' zeros of V come before the products)
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_half[tile]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[tile]);
      }
      if (!ok) break;
      v_count += v_tiles;
      if (n == 0) {
        after = cursor.next(bar, items, abort_flag, p.timeout_ns, err);
        if (after && needs_q(after)) load_q(after);
      }
      // the next item's scores run under this one's last steps
      if (after && needs_q(after)) q_loaded();
      if (n > 0) {
        if (!(ok = wait_all(&bar.o_full[tile], o_count & 1, abort_flag, p.timeout_ns, err))) break;
        ++o_count;
        tc_fence_after();
      }
      if (warp_live) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int64_t at = token * p.heads + head;
        const bool split = t->s.splits > 1;
        const int64_t part_at = t->split * static_cast<int64_t>(p.T) * p.heads + at;
        // where this lane's row goes, in bytes from the first row; and the rows of its 8 lanes
        uint8_t *const to = split ? reinterpret_cast<uint8_t *>(p.part) : reinterpret_cast<uint8_t *>(p.out);
        const int size = split ? 4 : 2;
        const int64_t mine_at = live ? (split ? part_at : at) * p.D * size : -1;
        // (loops that run once a tile or less are not unrolled: a call of few items spends much of its
        // time on fetching code)
#pragma unroll 1
        for (int c = 0; c < DP; c += 32) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(o_addr + c, o);
            tmem_ld_wait();
          }
          float y[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) y[x] = sum == 0.0f ? 0.0f : __uint_as_float(o[x]) * inv;
          // 8 lanes turn their rows so that a store covers runs of each row: 128 bytes of f32, or 64
          // of the type, 4 lanes to a row
          if (split) {
            uint4 v[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
              v[x] = make_uint4(__float_as_uint(y[4 * x]), __float_as_uint(y[4 * x + 1]), __float_as_uint(y[4 * x + 2]),
                                __float_as_uint(y[4 * x + 3]));
            turn_rows<8>(v, lane);
            const int col = c + (lane & 7) * 4;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const int64_t row = __shfl_sync(0xffffffffu, mine_at, (lane & ~7) + x);
              if (row >= 0 && col < p.D) *reinterpret_cast<uint4 *>(to + row + col * 4) = v[x];
            }
          } else {
            uint4 v[4];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              v[x] = make_uint4(A::pack2(y[8 * x], y[8 * x + 1]), A::pack2(y[8 * x + 2], y[8 * x + 3]),
                                A::pack2(y[8 * x + 4], y[8 * x + 5]), A::pack2(y[8 * x + 6], y[8 * x + 7]));
            turn_rows<4>(v, lane);
            const int col = c + (lane & 3) * 8;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int64_t row = __shfl_sync(0xffffffffu, mine_at, (lane & ~3) + x);
              if (row >= 0 && col < p.D) *reinterpret_cast<uint4 *>(to + row + col * 2) = v[x];
            }
          }
        }
        debug_check(!live || (token >= 0 && token < p.T && head >= 0 && head < p.heads), err);
        if (split && live) p.part_lse[part_at] = sum == 0.0f ? -INFINITY : base + __log2f(sum);
        tc_fence_before();
      }
      cursor.done(bar, 1);
      t = after;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    // (all row tiles' warps: what one has taken out another may have to add)
    asm volatile("bar.sync 1, 256;" ::: "memory");
    if (taken && !*abort_flag) add_odd_values<A>(p, tile, warp & 3, total);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == kWarpMma) {
      // ---------------------------------------------------------- products --
      const uint32_t idesc_s = umma_idesc_f16kind(kRows, kKeys, A::kUmmaFormat);
      const uint32_t idesc_o = umma_idesc_f16kind(kRows, DP, A::kUmmaFormat) | (1u << 16);     // B: columns contiguous
      uint32_t q_count[2] = {0, 0}, p_count[2] = {0, 0};
      bool ok = true;
      auto commit = [&](uint64_t *b) {
        if (elect_one()) umma_commit(b);
        __syncwarp();
      };
      auto wait = [&](uint64_t *b, uint32_t parity) {
        ok = ok && wait_all(b, parity & 1, abort_flag, p.timeout_ns, err);
        return ok;
      };
      // (a tile's number and the loop bodies are fixed at compile time: with either left to
      // run time the operands were no longer uniform registers, and an instruction took
      // over 100 cycles to issue instead of 40)
      const uint64_t q_desc = umma_desc_sw128(smem_u32(q_smem)), k_desc = umma_desc_sw128(smem_u32(k_smem));
      const uint64_t v_desc0 = v_desc(smem_u32(v_smem), S::kHalfBytes);
      auto scores = [&](auto x, uint32_t slot, uint64_t *done) {
        if (elect_one()) {
          const uint64_t a = q_desc + x.value * (S::kTileBytes >> 4), b = k_desc + slot * (S::kTileBytes >> 4);
#pragma unroll
          for (int k = 0; k < DP / 16; ++k) {
            const uint64_t at = (k >> 2) * (S::kHalfBytes >> 4) + (k & 3) * 2;
            umma_bf16(tmem + x.value * 128, a + at, b + at, idesc_s, k > 0);
          }
          umma_commit(&bar.s_full[x.value]);
          if (done) umma_commit(done);
        }
        __syncwarp();
      };
      // the products of a tile's weights, half by half; false when given up
      auto values = [&](auto x, uint32_t slot, uint32_t first, uint64_t *done) {
        const uint64_t b = v_desc0 + slot * (S::kTileBytes >> 4);
        auto half = [&](auto from) {
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = from.value; k < from.value + kKeys / 32; ++k)
              umma_ts(tmem + o_col + x.value * DP, tmem + x.value * 128 + k * 8, b + k * (2048 >> 4), idesc_o,
                      k > 0 ? 1u : first ^ 1u);
            if (from.value > 0 && done) umma_commit(done);
          }
          __syncwarp();
        };
        const uint32_t parity = p_count[x.value]++;
        if (!wait(&bar.p_half[x.value], parity)) return false;
        half(std::integral_constant<int, 0>{});
        if (!wait(&bar.p_full[x.value], parity)) return false;
        half(std::integral_constant<int, kKeys / 32>{});
        return true;
      };
      constexpr std::integral_constant<int, 0> X0{};
      constexpr std::integral_constant<int, 1> X1{};
      uint32_t k_slot = 0, k_turn = 0, v_slot = 0, v_turn = 0;
      auto next_k = [&] { k_slot = k_slot + 1 == KS ? (k_turn ^= 1, 0) : k_slot + 1; };
      auto next_v = [&] { v_slot = v_slot + 1 == VS ? (v_turn ^= 1, 0) : v_slot + 1; };
      ItemCursor cursor;
#pragma unroll 1
      for (const Item *t; ok && (t = cursor.next(bar, items, abort_flag, p.timeout_ns, err));) {
        // (from one lane: the compiler then knows them, and what the loop carries, as uniform)
        const int n = __shfl_sync(0xffffffffu, tiles_of_item(t), 0);
        // two tiles share a tile of keys, or, as a pair, have one each
        const bool pair = __shfl_sync(0xffffffffu, t->pair, 0), two = pair || __shfl_sync(0xffffffffu, t->rows, 0) > kRows;
        const bool share = two && !pair;
        cursor.done(bar, 0);
        if (n <= 0) continue;
        if (!wait(&bar.k_full[k_slot], k_turn) || !wait(&bar.q_full[0], q_count[0]++)) break;
        tc_fence_after();
        scores(X0, k_slot, share ? nullptr : &bar.k_empty[k_slot]);
        if (two) {
          if (pair) {
            next_k();
            if (!wait(&bar.k_full[k_slot], k_turn)) break;
          }
          if (!wait(&bar.q_full[1], q_count[1]++)) break;
          tc_fence_after();
          scores(X1, k_slot, &bar.k_empty[k_slot]);
        }
        next_k();
#pragma unroll 1
        for (int i = 0; i < n - 1; ++i) {
          if (!wait(&bar.k_full[k_slot], k_turn) || !wait(&bar.v_full[v_slot], v_turn)) break;
          if (!values(X0, v_slot, i == 0, share ? nullptr : &bar.v_empty[v_slot])) break;
          scores(X0, k_slot, share ? nullptr : &bar.k_empty[k_slot]);
          if (two) {
            if (pair) {
              next_v();
              next_k();
              if (!wait(&bar.k_full[k_slot], k_turn) || !wait(&bar.v_full[v_slot], v_turn)) break;
            }
            if (!values(X1, v_slot, i == 0, &bar.v_empty[v_slot])) break;
            scores(X1, k_slot, &bar.k_empty[k_slot]);
          }
          next_v();
          next_k();
        }
        if (!ok || !wait(&bar.v_full[v_slot], v_turn)) break;
        if (!values(X0, v_slot, n == 1, share ? nullptr : &bar.v_empty[v_slot])) break;
        commit(&bar.o_full[0]);
        if (two) {
          if (pair) {
            next_v();
            if (!wait(&bar.v_full[v_slot], v_turn)) break;
          }
          if (!values(X1, v_slot, n == 1, &bar.v_empty[v_slot])) break;
          commit(&bar.o_full[1]);
        }
        next_v();
      }
      // given up: the products in flight
      if (*abort_flag) {
        commit(&bar.mma_done);
        mbar_wait_drain(&bar.mma_done, 0, p.timeout_ns);
      }
    } else if (warp == kWarpK || warp == kWarpV) {
      // ------------------------------------------------------------ copies --
      const bool is_k = warp == kWarpK;
      const uint32_t stages = is_k ? KS : VS;
      uint64_t *full = is_k ? bar.k_full : bar.v_full, *empty = is_k ? bar.k_empty : bar.v_empty;
      uint8_t *ring = is_k ? k_smem : v_smem;
      const CUtensorMap *map = is_k ? &maps.k : &maps.v;
      // a lane per box of rows (of all halves, or of one) looks its page up
      const int boxes = kKeys / maps.box, parts = S::kHalves / maps.halves;
      uint32_t count = 0;
      ItemCursor cursor;
      for (const Item *next; (next = cursor.next(bar, items, abort_flag, p.timeout_ns, err));) {
        const Item t = *next;
        const int n = tiles_of_item(next);
        cursor.done(bar, 0);
        const int head = __shfl_sync(0xffffffffu, t.head, 0), heads = __shfl_sync(0xffffffffu, t.pair, 0) + 1;
        int page = -1, row = 0;
        auto look_up = [&](int i) {
          const int64_t key = static_cast<int64_t>(t.k0) + static_cast<int64_t>(i) * kKeys + lane * maps.box;
          page = -1;
          row = 0;
          if (lane < boxes && key < t.k1 && key + maps.box > t.first) {
            const int x = static_cast<int>(key) / p.page_size;
            row = static_cast<int>(key) - x * p.page_size;
            page = page_entry(p, t.b, x);
          }
        };
        look_up(0);
        bool ok = true;
        for (int i = 0; i < n && ok; ++i) {
          const int checked = checked_page(p, page), checked_row = row;
          for (int x = 0; x < heads; ++x, ++count) {
            const uint32_t slot = count % stages;
            if (!(ok = wait_all(&empty[slot], ((count / stages) & 1) ^ 1, abort_flag, p.timeout_ns, err))) break;
            const bool withheld = p.withhold && is_k && count == 0;
            if (!withheld && elect_one()) mbar_arrive_expect_tx(&full[slot], S::kTileBytes);
            __syncwarp();
            for (int j = 0; j < boxes && !withheld; ++j) {
              const int pg = __shfl_sync(0xffffffffu, checked, j), rw = __shfl_sync(0xffffffffu, checked_row, j);
              if (elect_one()) {
                uint8_t *dst = ring + slot * S::kTileBytes + j * maps.box * 128;
                debug_check(rw >= 0 && rw + maps.box <= p.page_size && pg < p.pages, err);
                tma_load_5d(dst, map, &full[slot], 0, rw, 0, head + x, pg);
                if (S::kHalves > 1 && parts > 1) tma_load_5d(dst + S::kHalfBytes, map, &full[slot], 64, rw, 0, head + x, pg);
              }
              __syncwarp();
            }
            if (x == 0 && i + 1 < n) look_up(i + 1);
          }
        }
        if (!ok) break;
      }
      // given up: the copies in flight
      if (*abort_flag)
        for (uint32_t c = count > stages ? count - stages : 0; c < count; ++c)
          mbar_wait_drain(&full[c % stages], (c / stages) & 1, p.timeout_ns);
    } else if (warp == kWarpItems) {
      // ------------------------------------------------------------- items --
      for (int step = 0;; ++step) {
        const int slot = step % kItems, id = item_of(step);
        Item t = find_item(p, id);
        if (id >= total) t.rows = 0;
        if (!wait_all(&bar.item_empty[slot], ((step / kItems) & 1) ^ 1, abort_flag, p.timeout_ns, err)) break;
        if (lane == 0) {
          items[slot] = t;
          mbar_arrive(&bar.item_full[slot]);
        }
        __syncwarp();
        if (id >= total) break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool encode_cache(CUtensorMap *map, const void *base, const int64_t (&strides)[3], const qsw_kv_cache &c, int64_t D,
                  int act, int box, int halves) {
  const EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(halves > 1 ? 64 : D), static_cast<cuuint64_t>(c.page_size),
                              static_cast<cuuint64_t>(halves), static_cast<cuuint64_t>(c.kv_heads),
                              static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t bytes[4] = {static_cast<cuuint64_t>(strides[2]) * 2, 128, static_cast<cuuint64_t>(strides[1]) * 2,
                               static_cast<cuuint64_t>(strides[0]) * 2};
  const cuuint32_t boxes[5] = {64, static_cast<cuuint32_t>(box), static_cast<cuuint32_t>(halves), 1, 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return fn(map, act == ActF16::kId ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5,
            const_cast<void *>(base), dims, bytes, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class A, int DP>
cudaError_t launch_shape(const AttnParams &p, const CacheMaps &maps, int grid, cudaStream_t stream) {
  static DeviceOnce once;
  auto kernel = attn_tiles_kernel<A, DP>;
  const cudaError_t e = allow_smem(once, kernel, Shape<DP>::kSmem);
  return e != cudaSuccess ? e : launch_on(kernel, dim3(static_cast<unsigned>(grid)), kThreads, Shape<DP>::kSmem, stream,
                                          false, p, maps);
}

}  // namespace

bool encode_cache_maps(CacheMaps *maps, const qsw_kv_cache &cache, int64_t D, int act, int most_rows, bool whole) {
  // the largest power of two of a page's rows: no box leaves a page
  const int64_t box = cache.page_size & -cache.page_size;
  maps->box = static_cast<int>(box < most_rows ? box : most_rows);
  maps->halves = whole && D % 64 == 0 ? static_cast<int>(D / 64) : 1;
  return encode_cache(&maps->k, cache.k, cache.k_strides, cache, D, act, maps->box, maps->halves) &&
         encode_cache(&maps->v, cache.v, cache.v_strides, cache, D, act, maps->box, maps->halves);
}

cudaError_t launch_attention_tiles(const AttnParams &p, const ListForm &f, int act, const qsw_kv_cache &cache,
                                   cudaStream_t stream) {
  const bool f16 = act == ActF16::kId;
  CacheMaps maps = {};
  // (the products take a tile's halves one after the other: only a box of a whole tile may
  // hold both)
  if (!encode_cache_maps(&maps, cache, p.D, act, kKeys, cache.page_size % kKeys == 0)) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(f.items < f.slots ? f.items : f.slots);
  if (p.D <= 64)
    return f16 ? launch_shape<ActF16, 64>(p, maps, grid, stream) : launch_shape<ActBf16, 64>(p, maps, grid, stream);
  return f16 ? launch_shape<ActF16, 128>(p, maps, grid, stream) : launch_shape<ActBf16, 128>(p, maps, grid, stream);
}

cudaError_t tiles_take_errors(unsigned int *out) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_attn_error, sizeof v);
  if (e != cudaSuccess) return e;
  if (v) {
    e = cudaMemcpyToSymbol(g_attn_error, &zero, sizeof zero);
    if (e != cudaSuccess) return e;
  }
  *out = v;
  return cudaSuccess;
}

}  // namespace qsw
