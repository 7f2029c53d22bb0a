// Attention over a paged cache: what the plan, the two kernels and the join share.
//
//   o = sum_j softmax_j(scale q . k_j) v_j      over the keys j that the token sees
//
// Query rows of one kv head are numbered token * group + (head in the group): the heads
// that share a kv head are rows of one tile, and K and V are read once for all of them.
// A tile of rows over a range of keys is an item; a sequence whose history is long
// against the number of rows is cut into splits, whose normalised results and
// log-sum-exps are joined by a kernel of their own.  Sequences with few rows and with many
// are two lists of items, each with a kernel.
#pragma once

#include <climits>

#include "qsw_fp4.cuh"
#include "qsw_internal.h"
#include "qsw_once.h"

namespace qsw {

constexpr float kLog2e = 1.4426950408889634f;

// One sequence of a plan.
struct alignas(16) SeqRec {
  int row;       // its first new token
  int n;         // new tokens
  int len;       // tokens in the cache, the new ones among them
  int blocks;    // row tiles per kv head
  int splits;    // and kPairBit: two kv heads an item
  int chunk;     // keys per split
  int first[2];  // its first item in each list (it has items in one of them)
};

constexpr int kPairBit = 1 << 16;

// Lists of items: sequences with few rows, and with many.
enum : int { LIST_ROWS = 0, LIST_TILES = 1 };

// The plan in device memory: words 0 and 1 (items of each list) and 2 (whether any sequence
// is split), the records, the sequence of each token (-1: none).
struct PlanView {
  int *head;
  SeqRec *rec;       // [B]
  int *seq_of;       // [T]
};
constexpr int kPlanHead = 8;
__host__ __device__ inline PlanView plan_view(void *base, int64_t B) {
  PlanView v;
  v.head = static_cast<int *>(base);
  v.rec = reinterpret_cast<SeqRec *>(v.head + kPlanHead);
  v.seq_of = reinterpret_cast<int *>(v.rec + B);
  return v;
}

struct AttnParams {
  const uint16_t *q;
  uint16_t *out;                   // [T, heads, D]
  const uint16_t *k, *v;
  int64_t q_t, q_h;                // strides in elements
  int64_t k_page, k_head, k_row, v_page, v_head, v_row;
  const int *page_table;
  int64_t table_stride;
  PlanView plan;
  int B, T, heads, kv_heads, group, D;
  int pages, page_size, max_pages;
  int window;                      // 0: none
  int list, tile_rows, tile_keys;
  int withhold;                    // test hook: the first keys are never requested
  int after_tiles;                 // few rows: launched as a dependent of the tiles' kernel
  float scale_log2;                // scale log2(e)
  float *part;                     // [splits][T][heads][D], normalised
  float *part_lse;                 // [splits][T][heads], log2
  uint64_t timeout_ns;
};

// One item: rows [row0, row0 + rows) (token * group + head in the group) of a sequence's
// kv head, keys [k0, k1), of which no row sees those before `first`, and all rows see those of
// [all_lo, all_hi).  A pair: the same rows of two kv heads, head and head + 1.
struct Item {
  SeqRec s;
  int b, head, row0, rows, k0, k1, first, all_lo, all_hi, split, pair;
};

// First and last + 1 key that the tokens [a, b) of a sequence see.
__device__ __forceinline__ void seen_keys(const SeqRec &s, int a, int b, int window, int &lo, int &hi) {
  hi = min(max(s.len - s.n + b, 0), s.len);
  lo = window ? max(s.len - s.n + a - window + 1, 0) : 0;
}

// Item `id` of the call's list, by a converged warp: the sequence by a search 32 wide, whose last
// step holds the records themselves.  (An id past the last item gives an item that must
// not be run: its loads need not wait for the number of items.)
__device__ __forceinline__ Item find_item(const AttnParams &p, int id) {
  const int lane = static_cast<int>(lane_id());
  int lo = 0, n = p.B;                 // the last sequence of [lo, lo + n) whose first item is at most id
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool le = at < n && __ldg(&p.plan.rec[lo + at].first[p.list]) <= id;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    lo += last * step;
    n = min(step, n - last * step);
  }
  int4 a = make_int4(0, 0, 0, 0), c = make_int4(1, 1, INT_MAX, INT_MAX);
  if (lane < n) {
    const int4 *r = reinterpret_cast<const int4 *>(p.plan.rec + lo + lane);
    a = __ldg(r);
    c = __ldg(r + 1);
  }
  const int first = p.list == LIST_ROWS ? c.z : c.w;
  const int last = 31 - __clz(__ballot_sync(0xffffffffu, first <= id) | 1u);
  Item t;
  t.b = lo + last;
  t.s.row = __shfl_sync(0xffffffffu, a.x, last);
  t.s.n = __shfl_sync(0xffffffffu, a.y, last);
  t.s.len = __shfl_sync(0xffffffffu, a.z, last);
  t.s.blocks = __shfl_sync(0xffffffffu, a.w, last);
  const int splits = __shfl_sync(0xffffffffu, c.x, last);
  t.s.splits = splits & (kPairBit - 1);
  t.pair = splits >= kPairBit;
  t.s.chunk = __shfl_sync(0xffffffffu, c.y, last);
  const int local = id - __shfl_sync(0xffffffffu, first, last);
  // the last rows first (they see the most keys), then splits, kv heads innermost: CTAs
  // that run together read the same keys of a head
  const int heads = p.kv_heads >> t.pair, per = heads * t.s.splits;
  const int up = local / per, r2 = local - up * per;
  const int block = t.s.blocks - 1 - up;
  t.split = r2 / heads;
  t.head = (r2 - t.split * heads) << t.pair;
  t.row0 = block * p.tile_rows;
  t.rows = min(p.tile_rows, t.s.n * p.group - t.row0);
  int end;
  const int from = t.row0 / p.group, to = (t.row0 + t.rows - 1) / p.group;
  seen_keys(t.s, from, to + 1, p.window, t.first, end);
  t.all_lo = p.window ? t.s.len - t.s.n + to - p.window + 1 : 0;
  t.all_hi = t.s.len - t.s.n + from + 1;
  const int start = t.first / p.tile_keys * p.tile_keys;
  // (64 bits: the last split's end)
  t.k0 = static_cast<int>(min(static_cast<int64_t>(start) + static_cast<int64_t>(t.split) * t.s.chunk,
                              static_cast<int64_t>(end)));
  t.k1 = static_cast<int>(min(static_cast<int64_t>(t.k0) + t.s.chunk, static_cast<int64_t>(end)));
  // the last split takes what is left
  if (t.split == t.s.splits - 1) t.k1 = max(end, t.k0);
  return t;
}

// Token and head of row r of an item and kv head.
__device__ __forceinline__ void row_of(const AttnParams &p, const Item &t, int kv_head, int r, int64_t &token, int &head,
                                       int &pos) {
  const int row = t.row0 + r, i = row / p.group;
  token = t.s.row + i;
  head = kv_head * p.group + row - i * p.group;
  pos = t.s.len - t.s.n + i;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The softmax weights as the products take them are f16 or bf16.  f16 has 5 bits of exponent: weights
// of up to 1 would lose bits below 2^-14 and vanish below 2^-25, though many of them may lie behind
// one large one.  There a row's base lies `lift` below its maximum, and weights reach 2^lift: what
// they are off by is then at most 2^-(25 + lift) of the largest, each.  (Not where scores are
// so far from 0 that the difference would be rounded.)
template <class A>
__device__ __forceinline__ float lift_of(float top, float lift) {
  return A::kId != 0 && fabsf(top) < 0x1p20f ? lift : 0.0f;
}

// Page of a sequence's tokens [page * page_size, ..) as the table has it, and as it is used: -1
// where it is not in the cache.  (Apart, so that a copy's page can be asked for ahead.)
__device__ __forceinline__ int page_entry(const AttnParams &p, int b, int page) {
  return page < p.max_pages ? __ldg(p.page_table + b * p.table_stride + page) : -1;
}
__device__ __forceinline__ int checked_page(const AttnParams &p, int id) { return id >= 0 && id < p.pages ? id : -1; }
__device__ __forceinline__ int page_of(const AttnParams &p, int b, int page) {
  return checked_page(p, page_entry(p, b, page));
}

// Values that are infinite or NaN.  Of a key that some rows of an item see and others do not, the
// products would give the others 0 * inf = NaN.  Such values are taken out of the tile of V, and
// add_odd gives them to the rows that see them: who does not keeps every bit, and only those keys,
// as many as an item has tokens (twice, with a window), are looked through.
template <class A>
struct Odd {
  static constexpr uint32_t kExp = A::kId == 0 ? 0x7F807F80u : 0x7C007C00u;       // of two values
  static constexpr uint32_t kLeast = A::kId == 0 ? 0x00800080u : 0x04000400u;
  // The sign bit of each that is odd: an exponent of all ones carries into it.
  static __device__ __forceinline__ uint32_t of(uint32_t x) { return ((x & kExp) + kLeast) & 0x80008000u; }
  static __device__ __forceinline__ uint32_t of(const uint4 &x) { return of(x.x) | of(x.y) | of(x.z) | of(x.w); }
  // Adds 0 times each: odd where one of them is.  (An instruction a pair, instead of three.)
  static __device__ __forceinline__ void gather(uint32_t x, uint32_t &sum) {
    if constexpr (A::kId == 0)
      asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
    else
      asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
  }
  static __device__ __forceinline__ void gather(const uint4 &x, uint32_t (&sum)[2]) {
    gather(x.x, sum[0]), gather(x.y, sum[1]), gather(x.z, sum[0]), gather(x.w, sum[1]);
  }
  static __device__ __forceinline__ uint32_t without(uint32_t x) { return x & ~((of(x) >> 15) * 0xFFFFu); }
  static __device__ __forceinline__ uint4 without(const uint4 &x) {
    return make_uint4(without(x.x), without(x.y), without(x.z), without(x.w));
  }
};

// Whether all rows of the item see the keys [key, key + n).
__device__ __forceinline__ bool all_seen(const Item &t, int key, int n) {
  return key >= max(t.first, t.all_lo) && key + n <= min(t.k1, t.all_hi);
}

// Adds the odd values of the keys that not all rows of an item see to its rows [row0, row0 +
// rows), at most 32, a lane each, once the warp has written them.  (Inline: with a call at the end of
// the few rows' items 64 decoding sequences took 161 us instead of 155, though nothing called it.)
template <class A>
__device__ __forceinline__ void add_odd(const AttnParams &p, const Item &t, int kv_head, int row0, int rows) {
  const int lane = static_cast<int>(lane_id());
  int64_t token;
  int head, pos;
  row_of(p, t, kv_head, row0 + (lane < rows ? lane : 0), token, head, pos);
  const uint16_t *q = p.q + token * p.q_t + head * p.q_h;
  const int64_t at = (token * p.heads + head) * p.D;
  float *part = t.s.splits > 1 ? p.part + t.split * static_cast<int64_t>(p.T) * p.heads * p.D + at : nullptr;
  __syncwarp();
  // the keys before those that all see, and behind them
  const int begin = max(t.k0, t.first), lo_end = min(max(t.all_lo, begin), t.k1);
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int from = side ? max(max(begin, t.all_hi), lo_end) : begin, to = side ? t.k1 : lo_end;
    for (int first = from; first < to; first += 32) {
      // each lane a key: where its value lies, and whether something in it is odd
      const int mine = first + lane;
      uint64_t v_at = 0, k_at = 0;
      bool odd = false;
      if (mine < to) {
        const int page = page_of(p, t.b, mine / p.page_size);
        if (page >= 0) {
          const uint16_t *v = p.v + page * p.v_page + kv_head * p.v_head + (mine % p.page_size) * p.v_row;
          v_at = reinterpret_cast<uint64_t>(v);
          k_at = reinterpret_cast<uint64_t>(p.k + page * p.k_page + kv_head * p.k_head + (mine % p.page_size) * p.k_row);
          for (int c = 0; c < p.D; c += 8) odd |= Odd<A>::of(*reinterpret_cast<const uint4 *>(v + c)) != 0;
        }
      }
      const unsigned keys = __ballot_sync(0xffffffffu, odd);
      if (!keys) continue;
      // which of them the lane's row sees, and of those the ones of weight 0 (0 * inf is NaN)
      unsigned seen = 0, none = 0;
      for (unsigned left = keys; left; left &= left - 1) {
        const int i = __ffs(left) - 1, key = first + i;
        const auto *k = reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, k_at, i));
        if (lane >= rows || key > pos || (p.window && key <= pos - p.window)) continue;
        seen |= 1u << i;
        float s = 0.0f;
        for (int c = 0; c < p.D; c += 2) {
          const uint32_t x = *reinterpret_cast<const uint32_t *>(q + c), y = *reinterpret_cast<const uint32_t *>(k + c);
          s = fmaf(A::hi(x), A::hi(y), fmaf(A::lo(x), A::lo(y), s));
        }
        if (s == -INFINITY) none |= 1u << i;
      }
      for (int c = 0; c < p.D; c += 2) {
        float lo = 0.0f, hi = 0.0f;
        for (unsigned left = keys; left; left &= left - 1) {
          const int i = __ffs(left) - 1;
          const auto *v = reinterpret_cast<const uint16_t *>(__shfl_sync(0xffffffffu, v_at, i));
          const uint32_t x = *reinterpret_cast<const uint32_t *>(v + c), which = Odd<A>::of(x);
          if (!(seen >> i & 1)) continue;
          const float w = none >> i & 1 ? 0.0f : 1.0f;
          if (which & 0x8000u) lo = fmaf(w, A::lo(x), lo);
          if (which >> 16) hi = fmaf(w, A::hi(x), hi);
        }
        if (part) {
          if (lo != 0.0f) part[c] = __ldcg(part + c) + lo;
          if (hi != 0.0f) part[c + 1] = __ldcg(part + c + 1) + hi;
        } else if (lo != 0.0f || hi != 0.0f) {
          uint32_t *out = reinterpret_cast<uint32_t *>(p.out + at + c);
          const uint32_t x = __ldcg(out);
          *out = A::pack2(lo != 0.0f ? A::lo(x) + lo : A::lo(x), hi != 0.0f ? A::hi(x) + hi : A::hi(x));
        }
      }
    }
  }
}

// The form of a call, a function of its sizes alone: the plan and the attention work it
// out for themselves and agree.
struct ListForm {
  int tile_rows, tile_keys;
  int slots;              // CTAs that run at once
  int64_t items;          // at most; 0: the list is not used
};
struct AttnForm {
  ListForm list[2];
  int64_t most_rows;      // of a sequence (and kv head) in the list of few rows
  int max_splits;         // 1: no history is split
};

// K and V of a cache as tensors of (column, row, half of a head, head, page), boxes of 64
// columns by `box` rows of a page.  One box holds all halves of its rows where D is a
// multiple of 64; else (halves == 1) a half is a box at its first column, and columns past D
// read 0.
struct CacheMaps {
  CUtensorMap k, v;
  int box;
  int halves;            // of a box
};
// Boxes of at most `most_rows` rows (a power of two); `whole`: of all halves, if D allows.  False
// where the cache cannot be described.
bool encode_cache_maps(CacheMaps *maps, const qsw_kv_cache &cache, int64_t D, int act, int most_rows, bool whole);

__device__ __forceinline__ void tma_load_5d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}

// A kernel's shared memory, allowed once per device: `once` belongs to the kernel.
template <class K>
cudaError_t allow_smem(DeviceOnce &once, K kernel, int bytes) {
  return once_per_device(once,
                         [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
}

// One thread of a converged warp.  Copies are issued by a thread chosen this way, with
// operands from one lane of a shuffle: with a lane per copy and operands of its own a copy
// took about 400 cycles to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// A wait of a whole warp, one vote where the phase is complete.
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, volatile int *abort, uint64_t timeout_ns,
                                         unsigned int *err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, timeout_ns, err));
}

cudaError_t launch_attention_tiles(const AttnParams &p, const ListForm &f, int act, const qsw_kv_cache &cache,
                                   cudaStream_t stream);
cudaError_t tiles_take_errors(unsigned int *out);

}  // namespace qsw
