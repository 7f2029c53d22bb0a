// Attention over a paged cache (qsw_attention.cuh): the plan of a step, the kernel for
// few rows, the join of split histories.
#include "qsw_attention.cuh"

namespace qsw {
namespace {

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
// beginning and end, and one of a split history kSplitCost more for what it leaves to the join.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ PlanParams p) {
  constexpr float kItemCost = 3.0f, kSplitCost = 3.0f;
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
  int longest[2] = {0, 0}, top = 0;
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
    p.out.rec[b] = s;
  }
  int chunk[2];
#pragma unroll
  for (int list = 0; list < 2; ++list) {
    int most = __reduce_max_sync(0xffffffffu, longest[list]);
    if (lane == 0) sums[warp] = most;
    __syncthreads();
    most = __reduce_max_sync(0xffffffffu, sums[lane]);
    __syncthreads();
    chunk[list] = most;
    if (p.max_splits == 1 || most <= kLeast) continue;
    const int parts = 1 + warp * (p.max_splits - 1) / 31;
    const int c = max((most + parts - 1) / parts, kLeast);
    float work = 0.0f, long_item = 0.0f, items = 0.0f;
    for (int b = lane; b < p.B; b += 32) {
      const SeqRec s = p.out.rec[b];
      if (!s.blocks || s.first[0] != list) continue;
      const int splits = max(1, min(p.max_splits, (s.chunk + c - 1) / c));
      const float n = static_cast<float>(s.blocks) * p.kv_heads, cost = splits > 1 ? kItemCost + kSplitCost : kItemCost;
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
      items = s.blocks * s.splits * p.kv_heads;
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
    if (b < p.B) p.out.rec[b] = s;
  }
  any = __syncthreads_or(any);
  if (tid == 0) {
    p.out.head[0] = total[0];
    p.out.head[1] = total[1];
    p.out.head[2] = any;
  }
}

// ---------------------------------------------------------------- few rows --

constexpr int kKeyGroups = 4;      // of warps, each with keys of its own
constexpr int kSubKeys = 16;       // keys of a group's step
template <int RG>
constexpr int row_stages = RG == 1 ? 3 : 6;      // two CTAs on an SM, or one

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
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

template <int DP>
constexpr int row_stage_bytes = 2 * kSubKeys * DP * 2;

// Up to 16 RG rows of one kv head.  Four groups of RG warps each take every fourth run of 16
// keys with a ring of their own; a warp has 16 rows and a softmax of its own (no barrier over
// the CTA in the loop), and the groups' results meet at the end.  With RG = 2 one warp of a
// group copies K and the other V, and they meet once a step.  K and V rows lie in 16-byte
// chunks, chunk c of key j at c ^ (j mod 8).
//
// HBM-bound: 64 sequences of 128 to 16000 keys, 8 kv heads of 128: 162 us for 983 MB, 6.1 TB/s.
template <class A, int DP, int RG>
__global__ void __launch_bounds__(32 * kKeyGroups * RG, 3 - RG)
    attn_rows_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kRowWarps = kKeyGroups * RG, kRowStages = row_stages<RG>, ROWS = 16 * RG;
  constexpr int CH = DP / 8;                     // 16-byte chunks of a row
  constexpr int PASS = 32 / CH;                  // keys per pass of a warp's copies
  constexpr int STAGE = row_stage_bytes<DP>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float warp_m[kKeyGroups][ROWS], warp_l[kKeyGroups][ROWS];
  __shared__ unsigned redo;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int kg = warp / RG, rg = warp % RG;
  if constexpr (kDebugBounds) debug_poison_smem(ring, kKeyGroups * kRowStages * STAGE);
  if (!p.after_tiles) griddep_wait();      // (then all before the tiles' kernel is complete)
  griddep_launch_dependents();
  const int total = __ldg(p.plan.head + LIST_ROWS);
  const int ch = lane % CH, sub = lane / CH;
  const uint32_t mine = smem_u32(ring) + kg * kRowStages * STAGE;

  for (int id = static_cast<int>(blockIdx.x);; id += static_cast<int>(gridDim.x)) {
    const Item t = find_item(p, id);
    if (id >= total) break;
    __syncthreads();      // the ring of the item before is free, its flags have been read
    if (tid == 0) redo = 0;
    const int runs = (t.k1 - t.k0 + kSubKeys - 1) / kSubKeys;       // of the item
    const int my_runs = runs > kg ? (runs - kg + kKeyGroups - 1) / kKeyGroups : 0;

    // q, as the A operand: rows lane / 4 and + 8, pairs (lane % 4) of each 8 columns
    uint32_t q[DP / 16][4];
    int64_t token;
    int head, pos[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = rg * 16 + lane / 4 + 8 * h;
      const bool live = r < t.rows;
      row_of(p, t, live ? r : 0, token, head, pos[h]);
      const uint16_t *src = p.q + token * p.q_t + head * p.q_h;
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int c = kk * 16 + x * 8 + (lane & 3) * 2;
          q[kk][h + 2 * x] = live && c < p.D ? *reinterpret_cast<const uint32_t *>(src + c) : 0u;
        }
    }

    // pages of the warp's next runs: lane l has the 8 keys l % 2 of run l / 2
    int page = -1, row = 0, page_next = -1, row_next = 0;
    auto fetch_pages = [&](int from, int &pg, int &rw) {
      const int run = (from + lane / 2) * kKeyGroups + kg;
      const int64_t key = static_cast<int64_t>(t.k0) + static_cast<int64_t>(run) * kSubKeys + (lane & 1) * 8;
      pg = -1;
      rw = 0;
      if (key < t.k1) {
        const int n = static_cast<int>(key) / p.page_size;
        pg = page_of(p, t.b, n);
        rw = static_cast<int>(key) - n * p.page_size;
      }
    };
    fetch_pages(0, page_next, row_next);
    auto issue = [&](int i) {       // copies of the warp's run i
      if (i < my_runs) {
        if ((i & 15) == 0) {
          page = page_next;
          row = row_next;
          fetch_pages(i + 16, page_next, row_next);
        }
        const uint32_t dst = mine + (i % kRowStages) * STAGE;
        const int key0 = t.k0 + (i * kKeyGroups + kg) * kSubKeys;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int pg = __shfl_sync(0xffffffffu, page, 2 * (i & 15) + g);
          const int rw = __shfl_sync(0xffffffffu, row, 2 * (i & 15) + g);
          const bool ok = pg >= 0 && ch * 8 < p.D;
          const int64_t pg0 = ok ? pg : 0;
          const int c0 = ok ? ch * 8 : 0;
          const uint16_t *k = p.k + pg0 * p.k_page + t.head * p.k_head + (rw + sub) * p.k_row + c0;
          const uint16_t *v = p.v + pg0 * p.v_page + t.head * p.v_head + (rw + sub) * p.v_row + c0;
#pragma unroll
          for (int x = 0; x < 8 / PASS; ++x) {
            const int j = g * 8 + x * PASS + sub;
            const uint32_t bytes = ok && key0 + j < t.k1 && key0 + j >= t.first ? 16u : 0u;
            const uint32_t at = dst + j * (DP * 2) + ((ch ^ (j & 7)) << 4);
            if (RG == 1 || rg == 0) cp_async16(at, k + x * PASS * p.k_row, bytes);
            if (RG == 1 || rg == 1) cp_async16(at + kSubKeys * DP * 2, v + x * PASS * p.v_row, bytes);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };

    float o[DP / 8][4];
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kRowStages - 1; ++i) issue(i);
    for (int i = 0; i < my_runs; ++i) {
      if constexpr (RG == 1) {
        __syncwarp();                  // every lane has read the stage that is filled next
        issue(i + kRowStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kRowStages - 1) : "memory");
        __syncwarp();
      } else {
        // both halves of stage i are there, and stage i - 1 has been read
        asm volatile("cp.async.wait_group %0;" ::"n"(kRowStages - 2) : "memory");
        asm volatile("bar.sync %0, %1;" ::"r"(1 + kg), "n"(32 * RG) : "memory");
        issue(i + kRowStages - 1);
      }
      const uint32_t ks = mine + (i % kRowStages) * STAGE, vs = ks + kSubKeys * DP * 2;
      float s[2][4] = {};
      {
        const int j = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          uint32_t b[4];
          ldmatrix4(ks + j * (DP * 2) + (((2 * kk + ((lane >> 3) & 1)) ^ (j & 7)) << 4), b);
          mma16816<A>(s[0], q[kk], b[0], b[1]);
          mma16816<A>(s[1], q[kk], b[2], b[3]);
        }
      }
      const int key0 = t.k0 + (i * kKeyGroups + kg) * kSubKeys + (lane & 3) * 2;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int key = key0 + n * 8 + (x & 1), at = pos[x >> 1];
          const bool seen = key <= at && key < t.k1 && (!p.window || key > at - p.window);
          s[n][x] = seen ? s[n][x] * p.scale_log2 : -INFINITY;
          top[x >> 1] = fmaxf(top[x >> 1], s[n][x]);
        }
      float base[2], shrink[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
        const float now = fmaxf(m[h], top[h]);
        base[h] = now == -INFINITY ? 0.0f : now;       // nothing seen yet
        shrink[h] = ex2(m[h] - base[h]);
        m[h] = now;
        l[h] *= shrink[h];
      }
      uint32_t a[4];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          s[n][x] = ex2(s[n][x] - base[x >> 1]);
          l[x >> 1] += s[n][x];
        }
        // weights as the products take them: rounded to the activations' type (one part in
        // 256 for bf16, of either sign); the sum l is that of the f32 weights
        a[2 * n] = A::pack2(s[n][0], s[n][1]);
        a[2 * n + 1] = A::pack2(s[n][2], s[n][3]);
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
      {
        const int j = ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
        for (int d = 0; d < DP / 16; ++d) {
          uint32_t b[4];
          ldmatrix4_trans(vs + j * (DP * 2) + (((2 * d + (lane >> 4)) ^ (j & 7)) << 4), b);
          mma16816<A>(o[2 * d], a, b[0], b[1]);
          mma16816<A>(o[2 * d + 1], a, b[2], b[3]);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();
    // the warps' sums, in the rings' place
    constexpr int PITCH = DP + 4;
    float *sum = reinterpret_cast<float *>(ring);
    static_assert(kKeyGroups * ROWS * PITCH * 4 <= kKeyGroups * kRowStages * STAGE, "the sums fit");
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = rg * 16 + lane / 4 + 8 * h;
      if ((lane & 3) == 0) {
        warp_m[kg][r] = m[h];
        warp_l[kg][r] = l[h];
      }
#pragma unroll
      for (int d = 0; d < DP / 8; ++d)
        *reinterpret_cast<float2 *>(sum + (kg * ROWS + r) * PITCH + d * 8 + (lane & 3) * 2) =
            make_float2(o[d][2 * h], o[d][2 * h + 1]);
    }
    __syncthreads();
    // a row to 8 threads, 8 columns at a time
    const int r = tid / 8;
    bool finite = true;
    if (r < t.rows) {
      float top = warp_m[0][r];
#pragma unroll
      for (int w = 1; w < kKeyGroups; ++w) top = fmaxf(top, warp_m[w][r]);
      const float base = top == -INFINITY ? 0.0f : top;
      float f[kKeyGroups], all = 0.0f;
#pragma unroll
      for (int w = 0; w < kKeyGroups; ++w) {
        f[w] = ex2(warp_m[w][r] - base);
        all = fmaf(f[w], warp_l[w][r], all);
      }
      const float inv = all == 0.0f ? 0.0f : 1.0f / all;
      int at_pos;
      row_of(p, t, r, token, head, at_pos);
      const int64_t at = token * p.heads + head, part = t.split * static_cast<int64_t>(p.T) * p.heads + at;
      for (int c = (tid & 7) * 8; c < p.D; c += 64) {
        float y[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          float v = 0.0f;
#pragma unroll
          for (int w = 0; w < kKeyGroups; ++w) v = fmaf(f[w], sum[(w * ROWS + r) * PITCH + c + x], v);
          y[x] = v * inv;
          finite &= isfinite(y[x]) != 0;
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
    if (!finite) atomicOr(&redo, 1u << r);
    __syncthreads();
    for (unsigned again = redo; again; again &= again - 1) {
      const int x = __ffs(again) - 1;
      if (x % kRowWarps == warp) exact_row<A>(p, t, x);
    }
  }
  if (p.after_tiles) griddep_wait();       // the next kernel comes after both
}

// -------------------------------------------------------------------- join --

// Rows of split sequences: o = sum_s 2^(lse_s - top) o_s / sum_s 2^(lse_s - top), in the
// order of the splits.  A warp per row; a split without a key the row sees holds zeros
// and -infinity.  What the plan says is read before the attention has ended: it was
// complete before that began.
template <class A>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ AttnParams p) {
  constexpr int kStep = 8;       // splits in flight
  const int lane = static_cast<int>(lane_id()), c = lane * 4;
  const int64_t rows = static_cast<int64_t>(p.T) * p.heads;
  const int any = __ldg(p.plan.head + 2);
  int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  bool waited = false;
  for (; any && row < rows; row += static_cast<int64_t>(gridDim.x) * 8) {
    const int b = __ldg(p.plan.seq_of + row / p.heads);
    const int splits = b < 0 ? 1 : __ldg(&p.plan.rec[b].splits);
    if (!waited) griddep_wait();
    waited = true;
    if (splits <= 1) continue;
    float top = -INFINITY, all = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = 0; s0 < splits; s0 += kStep) {
      float lse[kStep];
      float4 v[kStep];
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int64_t at = (s0 + i) * rows + row;
        lse[i] = s0 + i < splits ? p.part_lse[at] : -INFINITY;
        v[i] = s0 + i < splits && c < p.D ? *reinterpret_cast<const float4 *>(p.part + at * p.D + c)
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
    const float inv = all == 0.0f ? 0.0f : 1.0f / all;
    if (c < p.D)
      *reinterpret_cast<uint2 *>(p.out + row * p.D + c) =
          make_uint2(A::pack2(o[0] * inv, o[1] * inv), A::pack2(o[2] * inv, o[3] * inv));
  }
  if (!waited) griddep_wait();
}

template <class A>
cudaError_t launch_rows(const AttnParams &p, const ListForm &f, cudaStream_t stream) {
  const int64_t most = 2 * static_cast<int64_t>(f.slots);
  const dim3 grid(static_cast<unsigned>(f.items < most ? f.items : most));
  auto go = [&](auto kernel, int groups, int bytes) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return e != cudaSuccess ? e : launch_on(kernel, grid, 32 * kKeyGroups * groups, bytes, stream, p.after_tiles, p);
  };
  const bool one = f.tile_rows == 16;
  if (p.D <= 64)
    return one ? go(attn_rows_kernel<A, 64, 1>, 1, kKeyGroups * row_stages<1> * row_stage_bytes<64>)
               : go(attn_rows_kernel<A, 64, 2>, 2, kKeyGroups * row_stages<2> * row_stage_bytes<64>);
  return one ? go(attn_rows_kernel<A, 128, 1>, 1, kKeyGroups * row_stages<1> * row_stage_bytes<128>)
             : go(attn_rows_kernel<A, 128, 2>, 2, kKeyGroups * row_stages<2> * row_stage_bytes<128>);
}

}  // namespace

// Largest buffer of split results, and the most splits of a sequence.
constexpr int64_t kPartBytes = int64_t(128) << 20;
constexpr int kMaxSplits = 128;

AttnForm attention_form(int64_t T, int64_t B, int64_t heads, int64_t kv_heads, int64_t D, int64_t max_len, int num_sms) {
  AttnForm f = {};
  const int64_t group = heads / kv_heads, seqs = T < B ? T : B;
  // Which lists there are: one token a sequence, as far as the sizes say, or the rows of a
  // single one, need one; else sequences with up to 32 rows go with the few.
  f.most_rows = B == 1 || T <= B ? (T <= B || T * group <= 32 ? INT32_MAX : 0) : 32;
  const int64_t few = T <= B ? group : B == 1 ? T * group : 32;
  ListForm &r = f.list[LIST_ROWS], &t = f.list[LIST_TILES];
  r.tile_rows = few <= 16 ? 16 : 32;
  r.tile_keys = kKeyGroups * kSubKeys;
  r.slots = r.tile_rows == 16 ? 2 * num_sms : num_sms;
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
    e = f16 ? launch_rows<ActF16>(p, f.list[LIST_ROWS], stream) : launch_rows<ActBf16>(p, f.list[LIST_ROWS], stream);
  if (e != cudaSuccess || f.max_splits == 1) return e;
  // (few CTAs: often no sequence is split, and they only begin and end)
  const int64_t ctas = (a.T * a.heads + 7) / 8, most = 8 * static_cast<int64_t>(num_sms);
  const dim3 grid(static_cast<unsigned>(ctas < most ? ctas : most));
  return f16 ? launch_on(join_kernel<ActF16>, grid, 256, 0, stream, true, p)
             : launch_on(join_kernel<ActBf16>, grid, 256, 0, stream, true, p);
}

}  // namespace qsw
