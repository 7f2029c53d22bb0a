// Attention over a paged cache (qsw_attention.cuh): the plan of a step, the kernel for
// few rows, the join of split histories.
#include <atomic>

#include "qsw_attention.cuh"

namespace qsw {
namespace {

__device__ unsigned int g_rows_error;
std::atomic<int> g_withhold{0};

// -------------------------------------------------------------------- plan --

// New tokens of sequence b.
__device__ __forceinline__ void new_tokens(const int *offsets, int b, int T, int &lo, int &hi) {
  lo = min(max(__ldg(offsets + b), 0), T);
  hi = min(max(__ldg(offsets + b + 1), lo), T);
}

struct PlanParams {
  const int *offsets, *lengths, *page_table;
  int64_t table_stride;
  PlanView out;
  int *positions, *slots;
  int B, T, group, kv_heads, window;
  int pages, page_size, max_len;
  int most_rows, max_splits;
  int tile_rows[2], tile_keys[2], cta_slots[2];
};

constexpr int kPlanThreads = 1024;

// CTA 0 decides how histories are split, the others write each token's position and
// cache row.
//
// The split, for each list: a chunk of keys that its sequences are cut into, chosen among 32
// (a warp each) by the time it would take in tiles -- the longest item, or the work of all
// over the CTAs that run at once, in whole waves; an item costs kItemCost tiles more for its
// beginning and end, and one of a split history kSplitCost more for what it leaves to the join
// (up to 256 rows of f32 written and read again; 16 in the other list).
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  constexpr float kItemCost = 3.0f, kSplitCost[2] = {2.0f, 7.0f};
  constexpr int kLeast = 4;        // tiles of a split, at least
  griddep_wait();
  griddep_launch_dependents();
  const int tid = static_cast<int>(threadIdx.x);
  if (blockIdx.x > 0) {
    const int t = (static_cast<int>(blockIdx.x) - 1) * kPlanThreads + tid;
    if (t >= p.T) return;
    // the last sequence that begins at or before t
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.offsets + mid) <= t)
        lo = mid;
      else
        hi = mid;
    }
    int a, e;
    new_tokens(p.offsets, lo, p.T, a, e);
    int pos = -1, slot = -1, seq = -1;
    if (t >= a && t < e) {
      const int len = min(max(__ldg(p.lengths + lo), 0), p.max_len);
      seq = lo;
      pos = len - (e - t);
      if (pos >= 0) {
        const int id = __ldg(p.page_table + lo * p.table_stride + pos / p.page_size);
        if (id >= 0 && id < p.pages) slot = id * p.page_size + pos % p.page_size;
      } else {
        pos = -1;
      }
    }
    p.positions[t] = pos;
    p.slots[t] = slot;
    p.out.seq_of[t] = seq;
    return;
  }
  __shared__ int sums[32];
  __shared__ unsigned long long best[2];
  const int warp = tid >> 5, lane = tid & 31;
  if (tid < 2) best[tid] = ~0ull;
  int longest[2] = {0, 0}, top = 0, tile_blocks = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    // offsets as an ascending table: an entry counts as no less than any before it (no row
    // then belongs to two sequences, and there are no more items than rows allow)
    const int b = b0 + tid;
    int first = b < p.B ? min(max(__ldg(p.offsets + b), 0), p.T) : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, first, d);
      if (lane >= d) first = max(first, o);
    }
    if (lane == 31) sums[warp] = first;
    __syncthreads();
    const int before = __reduce_max_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
    const int all = __reduce_max_sync(0xffffffffu, sums[lane]);
    first = max(max(first, before), top);
    top = max(top, all);
    __syncthreads();
    if (b >= p.B) continue;
    SeqRec s = {};
    s.row = first;
    s.n = max(min(__ldg(p.offsets + b + 1), p.T) - first, 0);
    s.len = min(max(__ldg(p.lengths + b), 0), p.max_len);
    // (T group < 2^31: checked on the host)
    const int rows = s.n * p.group, list = rows > p.most_rows ? LIST_TILES : LIST_ROWS;
    const int tile_rows = p.tile_rows[list], tile_keys = p.tile_keys[list];
    s.blocks = (rows + tile_rows - 1) / tile_rows;
    // keys of the last row tile, and of a middling one, in tiles
    const int tokens = min(s.n, (tile_rows + p.group - 1) / p.group + 1);
    int keys = s.len, mean = max(s.len - s.n / 2, min(s.len, 1));
    if (p.window) {
      keys = min(static_cast<int64_t>(keys), static_cast<int64_t>(p.window) + tokens + tile_keys);
      mean = min(mean, keys);
    }
    // (for now: tiles, mean tiles, the list)
    s.chunk = (keys + tile_keys - 1) / tile_keys;
    s.splits = (mean + tile_keys - 1) / tile_keys;
    s.first[0] = list;
    if (s.blocks) longest[list] = max(longest[list], s.chunk);
    if (list == LIST_TILES) tile_blocks += s.blocks;
    p.out.rec[b] = s;
  }
  // Two kv heads an item, for sequences of the list of many rows whose rows fill half a tile at
  // most: where the items without that are more than run at once.  (An item of one head's 128
  // rows takes as long as one of two.)
  tile_blocks = __reduce_add_sync(0xffffffffu, tile_blocks);
  if (lane == 0) sums[warp] = tile_blocks;
  __syncthreads();
  tile_blocks = __reduce_add_sync(0xffffffffu, sums[lane]);
  __syncthreads();
  const bool pairing =
      p.kv_heads % 2 == 0 && static_cast<int64_t>(tile_blocks) * p.kv_heads > p.cta_slots[LIST_TILES];
  auto pair_of = [&](const SeqRec &s, int list) {
    return pairing && list == LIST_TILES && s.n * p.group <= p.tile_rows[LIST_TILES] / 2;
  };
  int chunk[2];
#pragma unroll
  for (int list = 0; list < 2; ++list) {
    int most = __reduce_max_sync(0xffffffffu, longest[list]);
    if (lane == 0) sums[warp] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, sums[lane]);
    __syncthreads();
    chunk[list] = max(most, 1);      // (no keys at all: it divides)
    if (p.max_splits == 1 || most <= kLeast) continue;
    const int parts = 1 + warp * (p.max_splits - 1) / 31;
    const int c = max((most + parts - 1) / parts, kLeast);
    float work = 0.0f, long_item = 0.0f, items = 0.0f;
    for (int b = lane; b < p.B; b += 32) {
      const SeqRec s = p.out.rec[b];
      if (!s.blocks || s.first[0] != list) continue;
      const int splits = max(1, min(p.max_splits, (s.chunk + c - 1) / c));
      const float n = static_cast<float>(s.blocks) * (p.kv_heads >> pair_of(s, list)), cost = splits > 1 ? kItemCost + kSplitCost[list] : kItemCost;
      items += n * splits;
      work += n * (s.splits + cost * splits);
      long_item = fmaxf(long_item, (s.chunk + splits - 1) / splits + cost);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
      work += __shfl_xor_sync(0xffffffffu, work, d);
      items += __shfl_xor_sync(0xffffffffu, items, d);
      long_item = fmaxf(long_item, __shfl_xor_sync(0xffffffffu, long_item, d));
    }
    // whole waves of items (exact for equal ones)
    const float slots = static_cast<float>(p.cta_slots[list]), waves = items / slots;
    const float cost = fmaxf(long_item, work / slots * (ceilf(waves) / waves));
    // the cheapest, the fewest splits among equals
    if (lane == 0)
      atomicMin(&best[list], static_cast<unsigned long long>(__float_as_uint(cost)) << 32 | static_cast<unsigned>(warp));
    __syncthreads();
    const int chosen = 1 + static_cast<int>(best[list] & 31u) * (p.max_splits - 1) / 31;
    chunk[list] = max((most + chosen - 1) / chosen, kLeast);
  }
  // splits of each sequence, and its first item
  int total[2] = {0, 0}, any = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    SeqRec s = {};
    int items = 0, list = LIST_ROWS;
    if (b < p.B) {
      s = p.out.rec[b];
      list = s.first[0];
      const int c = list == LIST_ROWS ? chunk[0] : chunk[1];
      s.splits = s.blocks && p.max_splits > 1 ? max(1, min(p.max_splits, (s.chunk + c - 1) / c)) : 1;
      any |= s.splits > 1;
      s.chunk = max(1, (s.chunk + s.splits - 1) / s.splits) * p.tile_keys[list];
      const bool pair = pair_of(s, list);
      items = s.blocks * s.splits * (p.kv_heads >> pair);
    }
#pragma unroll
    for (int l = 0; l < 2; ++l) {
      const int mine = l == list ? items : 0;
      int sum = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      if (lane == 31) sums[warp] = sum;
      __syncthreads();
      const int before = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
      const int all = __reduce_add_sync(0xffffffffu, sums[lane]);
      s.first[l] = total[l] + before + sum - mine;
      total[l] += all;
      __syncthreads();
    }
    if (b < p.B) {
      if (pair_of(s, list)) s.splits |= kPairBit;
      p.out.rec[b] = s;
    }
  }
  any = __syncthreads_or(any);
  if (tid == 0) {
    p.out.head[0] = total[0];
    p.out.head[1] = total[1];
    p.out.head[2] = any;
  }
}

// ---------------------------------------------------------------- few rows --

constexpr int kRowWarps = 4;       // each with keys of its own
// Keys of a warp's step: 8 KB of K and V.  32 take a warp little longer than 16 (its softmax is mostly
// latency), but of 128 columns two CTAs then no longer fit on an SM.
constexpr int step_keys(int DP) { return DP == 128 ? 16 : 32; }
constexpr float kRowLift = 14.0f;
constexpr int kRowStages = 3;      // 96 KB of ring a CTA: two on an SM
constexpr int kRowStageBytes = 8192;

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
template <class A>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (A::kId == 0)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Up to 16 rows of one kv head.  Each of four warps takes every fourth run of KEYS keys with a
// ring of its own, which it fills by TMA (boxes of 8 to 32 rows of a page), and a softmax of its
// own (no barrier over the CTA in the loop); the warps' results meet at the end.
//
// HBM-bound: 64 sequences of 128 to 16000 keys, 8 kv heads of 128: 152 us for 983 MB, 6.4 TB/s. With few
// keys latency: 4 sequences of up to 180 keys take 6 us.
template <class A, int DP>
__global__ void __launch_bounds__(32 * kRowWarps, 2)
    attn_rows_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CacheMaps maps) {
  constexpr int KEYS = DP == 128 ? 16 : 32, STAGE = 2 * KEYS * DP * 2;      // step_keys
  static_assert(STAGE == kRowStageBytes, "a step's K and V");
  constexpr int H = DP / 64;                     // halves of a head
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ float warp_m[kRowWarps][16], warp_l[kRowWarps][16];
  __shared__ uint64_t full[kRowWarps][kRowStages];
  __shared__ int taken;          // values were taken out of V
  __shared__ int abort_word;
  volatile int *abort_flag = &abort_word;
  unsigned int *err = &g_rows_error;
  const int tid = static_cast<int>(threadIdx.x), warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (!p.after_tiles) griddep_wait();      // (else all before the tiles' kernel is complete)
  griddep_launch_dependents();
  const int total = __ldg(p.plan.head + LIST_ROWS);
  if (static_cast<int>(blockIdx.x) >= total) {
    if (p.after_tiles) griddep_wait();
    return;
  }
  if constexpr (kDebugBounds) {
    debug_poison_smem(ring, kRowWarps * kRowStages * STAGE);
    fence_proxy_async_smem();
  }
  if (tid < kRowWarps * kRowStages) {
    mbar_init(&full[0][0] + tid, 1);
    fence_mbar_init();
  } else if (tid == kRowWarps * kRowStages) {
    abort_word = 0;
    prefetch_tensormap(&maps.k);
    prefetch_tensormap(&maps.v);
  }
  uint8_t *mine = ring + warp * kRowStages * STAGE;

  // Copies: boxes of rows, of all halves or of one; a lane per box of rows looks its page
  // up.  In a stage a box's rows of 128 bytes lie half by half, chunk c of row j at c ^ (j mod 8).
  const int subs = KEYS / maps.box, parts = H / maps.halves;
  const int half_bytes = maps.box * 128;
  uint32_t issued = 0, used = 0;           // stages
  bool ok = true;
  // row j of a stage's K or V; of its 16 keys b, this lane's in the K and the V operand
  auto row_at = [&](int j) { return (j & -maps.box) * (H * 128) + (j & (maps.box - 1)) * 128; };
  int k_row[KEYS / 16], v_row[KEYS / 16];
#pragma unroll
  for (int b = 0; b < KEYS / 16; ++b) {
    k_row[b] = row_at(b * 16 + (lane >> 4) * 8 + (lane & 7));
    v_row[b] = row_at(b * 16 + ((lane >> 3) & 1) * 8 + (lane & 7));
  }

  for (int id = static_cast<int>(blockIdx.x);; id += static_cast<int>(gridDim.x)) {
    const Item t = find_item(p, id);
    if (id >= total) break;
    __syncthreads();      // the ring of the item before is free, its flags have been read
    if (tid == 0) taken = 0;
    const int runs = (t.k1 - t.k0 + KEYS - 1) / KEYS;       // of the item
    const int my_runs = runs > warp ? (runs - warp + kRowWarps - 1) / kRowWarps : 0;
    const int kv_head = __shfl_sync(0xffffffffu, t.head, 0);

    // the page of a box of the warp's run i, -1 (zeros) where no row of the item sees it; a step
    // ahead: the table's entry arrives while the step is computed
    auto look_up = [&](int i, int &page, int &row) {
      const int64_t key =
          static_cast<int64_t>(t.k0) + (static_cast<int64_t>(i) * kRowWarps + warp) * KEYS + lane * maps.box;
      page = -1;
      row = 0;
      if (lane < subs && key < t.k1 && key + maps.box > t.first) {
        const int n = static_cast<int>(key) / p.page_size;
        page = page_entry(p, t.b, n);
        row = static_cast<int>(key) - n * p.page_size;
      }
    };
    // the copies of the warp's next run
    auto issue = [&](int page, int row) {
      const uint32_t slot = issued % kRowStages;
      if (p.withhold && issued == 0) {
        ++issued;
        return;
      }
      const int checked = checked_page(p, page);
      uint8_t *dst = mine + slot * STAGE;
      if (elect_one()) mbar_arrive_expect_tx(&full[warp][slot], STAGE);
      __syncwarp();
      for (int j = 0; j < subs; ++j) {
        const int pg = __shfl_sync(0xffffffffu, checked, j), rw = __shfl_sync(0xffffffffu, row, j);
        if (elect_one()) {
          debug_check(rw >= 0 && rw + maps.box <= p.page_size && pg < p.pages, err);
          tma_load_5d(dst, &maps.k, &full[warp][slot], 0, rw, 0, kv_head, pg);
          tma_load_5d(dst + STAGE / 2, &maps.v, &full[warp][slot], 0, rw, 0, kv_head, pg);
          if (H > 1 && parts > 1) {
            tma_load_5d(dst + half_bytes, &maps.k, &full[warp][slot], 64, rw, 0, kv_head, pg);
            tma_load_5d(dst + STAGE / 2 + half_bytes, &maps.v, &full[warp][slot], 64, rw, 0, kv_head, pg);
          }
        }
        dst += H * half_bytes;
        __syncwarp();
      }
      ++issued;
    };
    int page[kRowStages + 1], row[kRowStages + 1];
#pragma unroll
    for (int i = 0; i <= kRowStages; ++i) look_up(i, page[i], row[i]);
#pragma unroll
    for (int i = 0; i < kRowStages; ++i)
      if (i < my_runs) issue(page[i], row[i]);
    int next_page = page[kRowStages], next_row = row[kRowStages];

    // q, as the A operand: rows lane / 4 and + 8, pairs (lane % 4) of each 8 columns
    uint32_t q[DP / 16][4];
    int64_t token;
    int head, begin[2], end[2];      // keys that the rows see
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane / 4 + 8 * h;
      const bool live = r < t.rows;
      int pos;
      row_of(p, t, t.head, live ? r : 0, token, head, pos);
      begin[h] = p.window ? pos - p.window + 1 : 0;
      end[h] = min(pos + 1, t.k1);
      const uint16_t *src = p.q + token * p.q_t + head * p.q_h;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int c = kk * 16 + x * 8 + (lane & 3) * 2;
          q[kk][h + 2 * x] = live && c < p.D ? *reinterpret_cast<const uint32_t *>(src + c) : 0u;
        }
    }

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    bool odd = false;
    for (int i = 0; i < my_runs; ++i) {
      const uint32_t slot = used % kRowStages;
      if (!(ok = ok && wait_all(&full[warp][slot], (used / kRowStages) & 1, abort_flag, p.timeout_ns, err))) break;
      uint8_t *stage = mine + slot * STAGE;
      const int run0 = t.k0 + (i * kRowWarps + warp) * KEYS;
      if (!all_seen(t, run0, KEYS)) {
        // rows of V that no row of the item sees, or not every one, may hold anything: a weight of 0 does
        // not take out infinities or NaN
        // (rows before those that all see, and behind them)
        const int from = min(max(max(t.first, t.all_lo) - run0, 0), KEYS);
        const int to = min(max(min(t.k1, t.all_hi) - run0, from), KEYS);
        for (int x = lane; x < (KEYS - to + from) * (DP / 8); x += 32) {
          const int i = x / (DP / 8), c = x % (DP / 8), j = i < from ? i : i + to - from;
          auto *at = reinterpret_cast<uint4 *>(stage + STAGE / 2 + row_at(j) + (c >> 3) * half_bytes + (c & 7) * 16);
          const bool seen = run0 + j < t.k1 && run0 + j >= t.first;
          const uint4 v = *at;
          if (!seen || Odd<A>::of(v)) {
            *at = seen ? Odd<A>::without(v) : make_uint4(0, 0, 0, 0);
            odd |= seen;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t ks = smem_u32(stage), vs = ks + STAGE / 2;
      float s[KEYS / 8][4] = {};
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        const int c = 2 * kk + ((lane >> 3) & 1);
#pragma unroll
        for (int n = 0; n < KEYS / 16; ++n) {
          uint32_t b[4];
          ldmatrix4(ks + k_row[n] + (c >> 3) * half_bytes + (((c ^ lane) & 7) << 4), b);
          mma16816<A>(s[2 * n], q[kk], b[0], b[1]);
          mma16816<A>(s[2 * n + 1], q[kk], b[2], b[3]);
        }
      }
      const int key0 = run0 + (lane & 3) * 2;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = key0 + n * 8 + (x & 1);
          const bool seen = key < end[x >> 1] && key >= begin[x >> 1];
          s[n][x] = seen ? s[n][x] * p.scale_log2 : -INFINITY;
          top[x >> 1] = fmaxf(top[x >> 1], s[n][x]);
        }
      float base[2], shrink[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        const float now = fmaxf(m[h], top[h] - lift_of<A>(top[h], kRowLift));
        base[h] = now == -INFINITY ? 0.0f : now;       // nothing seen yet
        shrink[h] = ex2(m[h] - base[h]);
        m[h] = now;
        l[h] *= shrink[h];
      }
      uint32_t a[KEYS / 16][4];
#pragma unroll
      for (int n = 0; n < KEYS / 8; ++n) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[n][x] = ex2(s[n][x] - base[x >> 1]);
          l[x >> 1] += s[n][x];
        }
        // weights as the products take them: rounded to the activations' type (half a step, 2^-8
        // of a weight in bf16, 2^-11 in f16, of either sign, and in f16 2^-39 of the largest); the sum l is that
        // of the f32 weights
        a[n / 2][2 * (n & 1)] = A::pack2(s[n][0], s[n][1]);
        a[n / 2][2 * (n & 1) + 1] = A::pack2(s[n][2], s[n][3]);
      }
      if (shrink[0] != 1.0f || shrink[1] != 1.0f) {
#pragma unroll
        for (int d = 0; d < DP / 8; ++d) {
          o[d][0] *= shrink[0];
          o[d][1] *= shrink[0];
          o[d][2] *= shrink[1];
          o[d][3] *= shrink[1];
        }
      }
#pragma unroll
      for (int n = 0; n < KEYS / 16; ++n)
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          const int c = 2 * d + (lane >> 4);
          uint32_t b[4];
          ldmatrix4_trans(vs + v_row[n] + (c >> 3) * half_bytes + (((c ^ lane) & 7) << 4), b);
          mma16816<A>(o[2 * d], a[n], b[0], b[1]);
          mma16816<A>(o[2 * d + 1], a[n], b[2], b[3]);
        }
      // the stage is read: the run kRowStages further takes its place
      ++used;
      __syncwarp();
      if (i + kRowStages < my_runs) {
        issue(next_page, next_row);
        look_up(i + kRowStages + 1, next_page, next_row);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();
    if (*abort_flag) break;
    if (odd) taken = 1;
    // the warps' sums, in the rings' place
    constexpr int PITCH = DP + 4;
    float *sum = reinterpret_cast<float *>(ring);
    static_assert(kRowWarps * 16 * PITCH * 4 <= kRowWarps * kRowStages * STAGE, "the sums fit");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = lane / 4 + 8 * h;
      if ((lane & 3) == 0) {
        warp_m[warp][r] = m[h];
        warp_l[warp][r] = l[h];
      }
#pragma unroll
      for (int d = 0; d < DP / 8; ++d)
        *reinterpret_cast<float2 *>(sum + (warp * 16 + r) * PITCH + d * 8 + (lane & 3) * 2) =
            make_float2(o[d][2 * h], o[d][2 * h + 1]);
    }
    __syncthreads();
    // a row to 8 threads, 8 columns at a time
    const int r = tid / 8;
    fence_proxy_async_smem();      // (the next copies overwrite the sums)
    if (r < t.rows) {
      float top = warp_m[0][r];
#pragma unroll
      for (int w = 1; w < kRowWarps; ++w) top = fmaxf(top, warp_m[w][r]);
      const float base = top == -INFINITY ? 0.0f : top;
      float f[kRowWarps], all = 0.0f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        f[w] = ex2(warp_m[w][r] - base);
        all = fmaf(f[w], warp_l[w][r], all);
      }
      const float inv = all == 0.0f ? 0.0f : 1.0f / all;
      int at_pos;
      row_of(p, t, t.head, r, token, head, at_pos);
      debug_check(token >= 0 && token < p.T && head >= 0 && head < p.heads, err);
      const int64_t at = token * p.heads + head, part = t.split * static_cast<int64_t>(p.T) * p.heads + at;
      for (int c = (tid & 7) * 8; c < p.D; c += 64) {
        float y[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kRowWarps; ++w) v = fmaf(f[w], sum[(w * 16 + r) * PITCH + c + x], v);
          y[x] = v * inv;
        }
        if (t.s.splits > 1) {
          float4 *dst = reinterpret_cast<float4 *>(p.part + part * p.D + c);
          dst[0] = make_float4(y[0], y[1], y[2], y[3]);
          dst[1] = make_float4(y[4], y[5], y[6], y[7]);
        } else {
          *reinterpret_cast<uint4 *>(p.out + at * p.D + c) =
              make_uint4(A::pack2(y[0], y[1]), A::pack2(y[2], y[3]), A::pack2(y[4], y[5]), A::pack2(y[6], y[7]));
        }
      }
      if (t.s.splits > 1 && (tid & 7) == 0) p.part_lse[part] = all == 0.0f ? -INFINITY : base + __log2f(all);
    }
    // (a warp's rows are those it has written)
    constexpr int kOfWarp = 16 / kRowWarps;
    const int mine0 = warp * kOfWarp;
    if (taken && t.rows > mine0) add_odd<A>(p, t, t.head, mine0, min(t.rows - mine0, kOfWarp));
  }
  // given up: the copies in flight
  if (*abort_flag)
    for (uint32_t c = used; c < issued; ++c)
      mbar_wait_drain(&full[warp][c % kRowStages], (c / kRowStages) & 1, p.timeout_ns);
  if (p.after_tiles) griddep_wait();       // the next kernel comes after both
}

// -------------------------------------------------------------------- join --

// Rows of split sequences: o = sum_s 2^(lse_s - top) o_s / sum_s 2^(lse_s - top), in a fixed
// order.  WARPS warps to a row (8 where there are few rows: each takes every eighth split);
// a split without a key the row sees holds zeros and -infinity.  What the plan says is read
// before the attention has ended: it was complete before that began.
template <class A, int WARPS>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kStep = 8;       // splits in flight
  constexpr int kRowsOfCta = 8 / WARPS;
  __shared__ float4 sums[WARPS > 1 ? 8 : 1][32];
  __shared__ float2 tops[8];
  const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(lane_id()), c = lane * 4;
  const int64_t rows = static_cast<int64_t>(p.T) * p.heads;
  const int any = __ldg(p.plan.head + 2);
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRowsOfCta + warp / WARPS;
  bool waited = false;
  for (; any && row < rows; row += static_cast<int64_t>(gridDim.x) * kRowsOfCta) {
    const int b = __ldg(p.plan.seq_of + row / p.heads);
    const int splits = b < 0 ? 1 : __ldg(&p.plan.rec[b].splits) & (kPairBit - 1);
    if (!waited) griddep_wait();
    waited = true;
    if (splits <= 1) continue;
    float top = -INFINITY, all = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = warp % WARPS; s0 < splits; s0 += kStep * WARPS) {
      float lse[kStep];
      float4 v[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int s = s0 + i * WARPS;
        const int64_t at = s * rows + row;
        lse[i] = s < splits ? p.part_lse[at] : -INFINITY;
        v[i] = s < splits && c < p.D ? *reinterpret_cast<const float4 *>(p.part + at * p.D + c)
                                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
      float now = top;
#pragma unroll
      for (int i = 0; i < kStep; ++i) now = fmaxf(now, lse[i]);
      const float base = now == -INFINITY ? 0.0f : now, shrink = ex2(top - base);
      top = now;
      all *= shrink;
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] *= shrink;
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const float w = ex2(lse[i] - base);
        all += w;
        o[0] = fmaf(w, v[i].x, o[0]);
        o[1] = fmaf(w, v[i].y, o[1]);
        o[2] = fmaf(w, v[i].z, o[2]);
        o[3] = fmaf(w, v[i].w, o[3]);
      }
    }
    if constexpr (WARPS > 1) {
      sums[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
      if (lane == 0) tops[warp] = make_float2(top, all);
      __syncthreads();
      if (warp == 0) {
        float now = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) now = fmaxf(now, tops[w].x);
        const float base = now == -INFINITY ? 0.0f : now;
        all = o[0] = o[1] = o[2] = o[3] = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float f = ex2(tops[w].x - base);
          const float4 v = sums[w][lane];
          all = fmaf(f, tops[w].y, all);
          o[0] = fmaf(f, v.x, o[0]);
          o[1] = fmaf(f, v.y, o[1]);
          o[2] = fmaf(f, v.z, o[2]);
          o[3] = fmaf(f, v.w, o[3]);
        }
      }
      __syncthreads();
      if (warp > 0) continue;
    }
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    if (c < p.D)
      *reinterpret_cast<uint2 *>(p.out + row * p.D + c) =
          make_uint2(A::pack2(o[0] * inv, o[1] * inv), A::pack2(o[2] * inv, o[3] * inv));
  }
  if (!waited) griddep_wait();
}

template <class A>
cudaError_t launch_join(const AttnParams &p, int num_sms, cudaStream_t stream) {
  // few CTAs: often no sequence is split, and they only begin and end
  const int64_t rows = static_cast<int64_t>(p.T) * p.heads, most = 8 * static_cast<int64_t>(num_sms);
  const auto grid = [&](int64_t ctas) { return dim3(static_cast<unsigned>(ctas < most ? ctas : most)); };
  return rows <= most ? launch_on(join_kernel<A, 8>, grid(rows), 256, 0, stream, true, p)
                      : launch_on(join_kernel<A, 1>, grid((rows + 7) / 8), 256, 0, stream, true, p);
}

template <class A, int DP>
cudaError_t launch_rows_form(const AttnParams &p, const ListForm &f, const qsw_kv_cache &cache, cudaStream_t stream) {
  constexpr int bytes = kRowWarps * kRowStages * kRowStageBytes + 1024;
  static DeviceOnce once;
  auto kernel = attn_rows_kernel<A, DP>;
  const cudaError_t e = allow_smem(once, kernel, bytes);
  if (e != cudaSuccess) return e;
  const int64_t most = 2 * static_cast<int64_t>(f.slots);
  const dim3 grid(static_cast<unsigned>(f.items < most ? f.items : most));
  CacheMaps maps = {};
  if (!encode_cache_maps(&maps, cache, p.D, A::kId, step_keys(DP), true)) return cudaErrorInvalidValue;
  return launch_on(kernel, grid, 32 * kRowWarps, bytes, stream, p.after_tiles != 0, p, maps);
}

template <class A>
cudaError_t launch_rows(const AttnParams &p, const ListForm &f, const qsw_kv_cache &cache, cudaStream_t stream) {
  return p.D <= 64 ? launch_rows_form<A, 64>(p, f, cache, stream) : launch_rows_form<A, 128>(p, f, cache, stream);
}

}  // namespace

void attention_withhold_next() { g_withhold.store(1); }

cudaError_t attention_take_errors(unsigned int *out) {
  unsigned int tiles = 0, rows = 0, zero = 0;
  cudaError_t e = tiles_take_errors(&tiles);
  if (e != cudaSuccess) return e;
  e = cudaMemcpyFromSymbol(&rows, g_rows_error, sizeof rows);
  if (e == cudaSuccess && rows) e = cudaMemcpyToSymbol(g_rows_error, &zero, sizeof zero);
  *out = tiles | rows;
  return e;
}

// Largest buffer of split results, and the most splits of a sequence.
constexpr int64_t kPartBytes = int64_t(128) << 20;
constexpr int kMaxSplits = 128;

AttnForm attention_form(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t D, int64_t max_len, int num_sms) {
  AttnForm f = {};
  const int64_t group = heads / kv_heads, seqs = T < B ? T : B;
  // Up to 16 rows go with the few, which one warp's products take (us, tiles of 256 rows for more
  // than 16 / for more than 32 rows, two warps sharing keys: 64 sequences of 1000 keys with 24 rows 65 / 80,
  // with 12 on the lone warp's kernel 55 / 78; 16 drafting ones 27.9 / 26.0).  Where the sizes
  // alone say which, there is one list: one token a sequence, or a single sequence.
  const int64_t rows = T <= B ? group : T * group;
  f.most_rows = T <= B || B == 1 ? (rows <= 16 ? INT32_MAX : 0) : 16;
  ListForm &r = f.list[LIST_ROWS], &t = f.list[LIST_TILES];
  r.tile_rows = 16;
  r.tile_keys = kRowWarps * step_keys(D <= 64 ? 64 : 128);
  r.slots = 2 * num_sms;
  t.tile_rows = 256;
  t.tile_keys = 128;
  t.slots = num_sms;
  // at least so many items without splits
  const int64_t least = (T * group + t.tile_rows - 1) / t.tile_rows * kv_heads;
  int64_t splits = kPartBytes / (T * heads * D * 4 + 1);
  if (splits > kMaxSplits) splits = kMaxSplits;
  // 256 keys a split at least; and where the items are many waves there is nothing to gain
  if (splits > (max_len + 255) / 256) splits = (max_len + 255) / 256;
  if (least >= 8 * static_cast<int64_t>(num_sms) || splits < 1) splits = 1;
  f.max_splits = static_cast<int>(splits);
  for (ListForm *l : {&r, &t})
    l->items = ((T * group + l->tile_rows - 1) / l->tile_rows + seqs) * kv_heads * splits;
  if (f.most_rows == 0) r.items = 0;
  if (f.most_rows == INT32_MAX) t.items = 0;
  return f;
}

int64_t paged_plan_bytes(int64_t B, int64_t T) {
  const PlanView v = plan_view(nullptr, B);
  return reinterpret_cast<intptr_t>(v.seq_of) + T * 4;
}

size_t attention_workspace_bytes(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t D, int64_t max_len,
                                 int num_sms) {
  if (T == 0 || B == 0) return 0;
  const AttnForm f = attention_form(T, B, heads, kv_heads, D, max_len, num_sms);
  return f.max_splits == 1 ? 0 : static_cast<size_t>(f.max_splits * T * heads * (D + 1) * 4);
}

cudaError_t launch_paged_plan(const PlanArgs &a, int num_sms, cudaStream_t stream) {
  if (num_sms <= 0) return cudaErrorInvalidDevice;
  const AttnForm f = attention_form(a.T, a.B, a.heads, a.cache.kv_heads, a.D, a.max_pages * a.cache.page_size, num_sms);
  PlanParams p = {};
  p.offsets = a.offsets;
  p.lengths = a.lengths;
  p.page_table = a.page_table;
  p.table_stride = a.table_stride;
  p.out = plan_view(a.plan, a.B);
  p.positions = a.positions;
  p.slots = a.slots;
  p.B = static_cast<int>(a.B);
  p.T = static_cast<int>(a.T);
  p.kv_heads = static_cast<int>(a.cache.kv_heads);
  p.group = static_cast<int>(a.heads / a.cache.kv_heads);
  p.window = static_cast<int>(a.window);
  p.pages = static_cast<int>(a.cache.pages);
  p.page_size = static_cast<int>(a.cache.page_size);
  p.max_len = static_cast<int>(a.max_pages * a.cache.page_size);
  p.most_rows = static_cast<int>(f.most_rows);
  p.max_splits = f.max_splits;
  for (int l = 0; l < 2; ++l) {
    p.tile_rows[l] = f.list[l].tile_rows;
    p.tile_keys[l] = f.list[l].tile_keys;
    p.cta_slots[l] = f.list[l].slots;
  }
  const dim3 grid(static_cast<unsigned>(1 + (a.T + kPlanThreads - 1) / kPlanThreads));
  return launch_on(plan_kernel, grid, kPlanThreads, 0, stream, false, p);
}

cudaError_t launch_paged_attention(const AttentionArgs &a, int num_sms, uint64_t timeout_ns, cudaStream_t stream) {
  if (num_sms <= 0) return cudaErrorInvalidDevice;
  const qsw_kv_cache &c = a.cache;
  const AttnForm f = attention_form(a.T, a.B, a.heads, c.kv_heads, a.D, a.max_pages * c.page_size, num_sms);
  AttnParams p = {};
  p.q = static_cast<const uint16_t *>(a.q.data);
  p.q_t = a.q.token_stride;
  p.q_h = a.q.head_stride;
  p.out = static_cast<uint16_t *>(a.out);
  p.k = static_cast<const uint16_t *>(c.k);
  p.v = static_cast<const uint16_t *>(c.v);
  p.k_page = c.k_strides[0], p.k_head = c.k_strides[1], p.k_row = c.k_strides[2];
  p.v_page = c.v_strides[0], p.v_head = c.v_strides[1], p.v_row = c.v_strides[2];
  p.page_table = a.page_table;
  p.table_stride = a.table_stride;
  p.plan = plan_view(const_cast<void *>(a.plan), a.B);
  p.B = static_cast<int>(a.B);
  p.T = static_cast<int>(a.T);
  p.heads = static_cast<int>(a.heads);
  p.kv_heads = static_cast<int>(c.kv_heads);
  p.group = p.heads / p.kv_heads;
  p.D = static_cast<int>(a.D);
  p.pages = static_cast<int>(c.pages);
  p.page_size = static_cast<int>(c.page_size);
  p.max_pages = static_cast<int>(a.max_pages);
  p.window = static_cast<int>(a.window);
  p.scale_log2 = a.scale * kLog2e;
  p.timeout_ns = timeout_ns;
  p.withhold = g_withhold.exchange(0, std::memory_order_relaxed);
  p.part = static_cast<float *>(a.workspace);
  p.part_lse = p.part + static_cast<int64_t>(f.max_splits) * a.T * a.heads * a.D;
  const bool f16 = a.act == ActF16::kId;
  cudaError_t e = cudaSuccess;
  auto set = [&](int list) {
    p.list = list;
    p.tile_rows = f.list[list].tile_rows;
    p.tile_keys = f.list[list].tile_keys;
    return f.list[list].items > 0;
  };
  // The few rows start in what the tiles leave free, without waiting for them: neither
  // reads what the other writes.
  if (set(LIST_TILES)) {
    e = launch_attention_tiles(p, f.list[LIST_TILES], a.act, c, stream);
    p.after_tiles = 1;
  }
  if (e == cudaSuccess && set(LIST_ROWS))
    e = f16 ? launch_rows<ActF16>(p, f.list[LIST_ROWS], c, stream)
            : launch_rows<ActBf16>(p, f.list[LIST_ROWS], c, stream);
  if (e != cudaSuccess || f.max_splits == 1) return e;
  return f16 ? launch_join<ActF16>(p, num_sms, stream) : launch_join<ActBf16>(p, num_sms, stream);
}

}  // namespace qsw
