// Products of microscaled 4-bit matrices on the block-scaled tensor core,
// grouped by expert:
//
//   acc[r, n] = sum_k x[r, k] w[e(r), n, k]         rows of x sorted by expert
//
// with x and w e2m1 codes and their scale blocks (qsw_fp4.cuh), and either
//   linear  out[r, n] = T(x_scale w_scale[e] acc[r, n]), or
//   swiglu  the weight rows hold gate and up rows in alternating runs of 16;
//           hidden = silu(gate) up in f32 is held in 4 bits again, codes and
//           scales written ready for the down projection.
//
// The weights are the MMA's M side (128 rows) and the tokens its N side, for
// every token count: N is a run-time operand of the instruction (a multiple of
// 16 up to 192), so one token and a ragged group of 150 waste no more than 15
// columns, and a single token streams its weights through TMA at HBM rate
// without a second kernel.  (Tiles of 64, 32 or 16 weight rows, to have more CTAs for
// few rows, gained nothing: a tile's time is that of its chain of stages.)
//
// One persistent CTA per SM, 17 warps: warps 0 and 14-16 issue the copies of the
// weights' and activations' codes and scales (a ring of stages of 256 elements of
// K: 128-byte swizzled code tiles by TMA, scale blocks by TMA or bulk copies; one
// warp each, since a copy takes its issuer over 100 cycles), warp 1 moves the
// scales into tensor memory and issues the MMAs, warps 2-13 run the epilogue.
// Tensor memory: two accumulators of 192 columns, so that a tile's epilogue runs
// under the next tile's products, and two scale buffers of 48 columns.  A tile is
// the work of one CTA, of a CTA pair (256 weight rows, many tokens) or of a
// cluster that splits K (few tiles, long K); little x is quantised in the kernel.
//
// What bounds it (GB300): few rows, the weights' bytes -- 8 experts of 4096 x 16384
// at 5.8 TB/s -- or, below about 30 MB, the launch and one tile's chain of stages
// (1 x 2048 x 8192, 9.5 MB: 7.4 us, of which launch and set-up 2, stages 2.5).  Many
// rows, the tensor pipe: 4096 x 4096 x 14336 takes 97 us, 5.0 PFLOP/s, and 12 scale
// copies per 4 products (192 tokens) are a quarter of that: 85 us without an epilogue, 63
// also without the scale copies, 54 with the loads alone.
//
// Programmatic dependent launch: everything a CTA does before griddep_wait --
// the group table, the weights of its first stages -- reads only what was
// complete before the launch in front of this one began (each kernel of a chain
// lets the next one start only after its own wait).
#include <atomic>
#include <mutex>
#include <type_traits>

#include "qsw_fp4.cuh"
#include "qsw_internal.h"
#include "qsw_tiles.h"

namespace qsw {
namespace {

__device__ unsigned int g_fp4_error;
std::atomic<int> g_withhold{0};

constexpr int kTileTokens = 192;
constexpr int kMaxStages = 16;               // (and at most 28: a lane initialises each)
constexpr int kFuseRows = 16;                // rows of x that a CTA quantises itself, at most
constexpr int64_t kFuseElements = 8192;      // and elements
constexpr int kEpiGroups = 3;                // epilogue groups of four warps
constexpr int kEpiWarps = 4 * kEpiGroups;
// Warps: the first producer, the MMA issuer, the epilogue, three more producers.
constexpr int kWarpMma = 1, kWarpEpi0 = 2, kWarpProd1 = kWarpEpi0 + kEpiWarps;
constexpr int kThreads = 32 * (kWarpProd1 + 3);
enum Role : int { W_CODES = 0, W_SCALES = 1, X_CODES = 2, X_SCALES = 3 };   // of the producers
constexpr int kStageK = 256;                 // elements of K per stage: one 128-byte swizzle row
constexpr int kSfCol = 2 * kTileTokens;      // first scale column of tensor memory
constexpr int kSfCols = 48;                  // per scale buffer: 16 weight, 32 token columns
// Exchange buffer of an epilogue group, 32 tokens: swiglu, f32 rows of 64
// features; linear, 16-bit rows of 128.
constexpr int kHPitch = 80;                  // floats
constexpr int kYPitch = 136;                 // 16-bit values
constexpr int kExBytes = 32 * kHPitch * 4;
static_assert(32 * kYPitch * 2 <= kExBytes, "both layouts fit");

struct GemmParams {
  const uint8_t *w_scales;
  const uint8_t *x_scales;
  const int *offsets;       // [groups + 1], null: one group of `rows`
  const float *w_scale;     // [groups], null: 1
  float x_scale;
  int groups;
  int rows;                 // rows of x
  int max_group;            // no group has more rows
  int N, K;
  int n_tiles;              // weight tiles per group
  int k_blocks;             // scale blocks along K
  int w_row_blocks;         // scale row blocks of a group's weights
  int bt;                   // most tokens of a tile
  int split;                // CTAs (a cluster) that share a tile's K: 1, 2 or 4
  int x_box, x_rows;        // rows of the small TMA box of x, and of a stage (the large box)
  int x_sf;                 // scale row blocks of x in a stage
  int stages;
  int recs;                 // tiles per CTA at most
  bool wide;                // rows of the output start at 16-byte boundaries
  bool out_f32;             // the output is f32
  int x_off, w_off, sf_off, fuse_sf_off, ex_off, rec_off, table_off;   // byte offsets in shared memory
  void *out;
  uint8_t *h_codes;
  uint8_t *h_scales;
  int h_k_blocks;
  Fp4Scale hq;
  uint64_t timeout_ns;
  int withhold;             // test hook: the weights' codes are never requested
  // few rows: x itself, [<= kFuseRows, K], quantised by every CTA into shared memory
  const void *x;
  Fp4Scale xq;
  int x_f16, x_tokens;      // its type and row count
  const int *order;         // sorted row r is row order[r] / fan of x; null: row r
  int fan;
};

// One tile of a CTA (or of a CTA pair), worked out before the first one starts: the
// roles walk these records, since finding the next tile from the group table
// (search, division) in the issuing warp cost more than a short tile's products.
struct alignas(16) TileRec {
  int e;        // group
  int row;      // first row of x
  int valid;    // tokens
  int n;        // valid rounded up to the MMA's step
  int w0;       // first weight row of this CTA within the group
  int w_block;  // its scale row block
  int x_block;  // scale row block of the first token's 128 rows
  int t0;       // first token within the group
};

// Tile `id` (< the number of tiles): token tiles fastest, then weight tiles, then
// groups.  off, first: first row and first tile of each group.  More than one token
// tile in a group: equal sizes, multiples of 64 (the scale lanes of a tile then start
// at column 0 or 2 of a block).
template <bool PAIR>
__device__ __forceinline__ TileRec make_rec(const GemmParams &p, const int *off, const int *first, int id,
                                            uint32_t rank) {
  constexpr int kStep = PAIR ? 32 : 16;      // of an MMA's N
  int e = 0;                                 // the last group whose first tile is at most id
  for (int hi = p.groups; hi - e > 1;) {
    const int mid = (e + hi) >> 1;
    if (first[mid] <= id)
      e = mid;
    else
      hi = mid;
  }
  const int m = min(off[e + 1] - off[e], p.max_group);
  const int nt = token_tiles(m, p.bt);
  const int local = id - first[e];
  const int wt = local / nt, tt = local - wt * nt;
  const int size = nt > 1 ? (ceil_div(m, nt) + 63) & ~63 : m;
  TileRec t;
  t.e = e;
  t.t0 = tt * size;
  t.row = off[e] + t.t0;
  t.valid = min(size, m - t.t0);
  t.n = max(kStep, (t.valid + kStep - 1) & ~(kStep - 1));
  if (!PAIR && p.x) t.n = kFuseRows;
  t.w0 = wt * (PAIR ? 2 * kSfRows : kSfRows) + (PAIR ? static_cast<int>(rank) * kSfRows : 0);
  t.w_block = e * p.w_row_blocks + t.w0 / kSfRows;
  t.x_block = (p.offsets ? static_cast<int>(ragged_row_block(off[e], e)) : 0) + t.t0 / kSfRows;
  return t;
}

// ------------------------------------------------------------- PTX pieces --

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Descriptor of a 512-byte scale block: 32 rows of 16 bytes, no swizzle.
__device__ __forceinline__ uint64_t scales_desc(uint32_t smem_addr) {
  uint64_t d = (smem_addr & 0x3FFFFu) >> 4;
  d |= static_cast<uint64_t>(128 >> 4) << 32;   // 8 rows of 16 bytes
  d |= static_cast<uint64_t>(1) << 46;          // descriptor version
  return d;
}
// A scale block into four columns of tensor memory, repeated in the four lane
// quarters.
template <bool PAIR>
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
  if (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// ---- CTA pairs (clusters of two): rank, barriers across the pair, copies that
// signal the leader's (rank 0) barrier, arrivals on it.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t leader_address(const void *p) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
  return a;
}
__device__ __forceinline__ uint32_t peer_address(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ float load_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// Hands the thread's shared memory over to the waiting CTA.
__device__ __forceinline__ void mbar_arrive_release_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// mbar_wait for what other CTAs of the cluster handed over.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, volatile int *abort,
                                                  uint64_t timeout_ns, unsigned int *err) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 63u) == 0) {
      if (*abort) return false;
      if (globaltimer_ns() - t0 > timeout_ns) {
        *abort = 1;
        atomicOr(err, DEVERR_TIMEOUT);
        return false;
      }
    }
  }
}
// Relaxed: nothing in memory is handed over (a releasing arrival would wait for the
// thread's global stores to be performed).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                                 int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// Arrive on `bar` -- of both CTAs of a pair -- once the issued tcgen05 work is done.
template <bool PAIR>
__device__ __forceinline__ void commit_to(uint64_t *bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc_all(uint32_t *slot) {
  if (PAIR) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(slot, 512);
    tmem_relinquish();
  }
}
template <bool PAIR>
__device__ __forceinline__ void tmem_free_all(uint32_t taddr) {
  if (PAIR)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(512) : "memory");
  else
    tmem_dealloc(taddr, 512);
}

// One thread of a converged warp.  The copies and products are issued by a
// thread chosen this way: the compiler then keeps their operands in uniform
// registers (chosen with `lane == 0`, each instruction took about 100 cycles).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

template <int FMT, bool PAIR>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  if constexpr (FMT == FP4_MX && !PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::
            "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else if constexpr (FMT == FP4_MX)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else if constexpr (!PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: e2m1 A and B, M = 128 (256 over a pair); the scale
// selectors are added per step.
template <int FMT, bool PAIR>
__device__ __forceinline__ uint32_t fp4_idesc(int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (FMT == FP4_MX ? 1u << 23 : 0u) |   // E8M0 or E4M3 scales
         ((PAIR ? 16u : 8u) << 24);          // M / 16
}

// The copies and products of one stage: `nkb` scale blocks, `steps` products of 64
// elements of K.  One thread's copies and products run in the order of issue.
template <int FMT, int XSF, bool PAIR>
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t idesc, uint64_t wd, uint64_t xd, uint32_t sf,
                                            uint64_t sfw, uint64_t sfx, uint32_t x_col, int nkb, int steps, bool first) {
  constexpr int kSfPerStage = kStageK / Fp4<FMT>::kSfK;
#pragma unroll
  for (int kb = 0; kb < kSfPerStage; ++kb) {
    if (kb >= nkb) break;
    scales_to_tmem<PAIR>(sf + kb * 4, sfw + kb * (kSfBytes >> 4));
#pragma unroll
    for (int b = 0; b < XSF; ++b)
      scales_to_tmem<PAIR>(sf + 16 + kb * 8 + b * 4, sfx + (kSfPerStage * b + kb) * (kSfBytes >> 4));
  }
#pragma unroll
  for (int kk = 0; kk < kStageK / 64; ++kk) {
    if (kk >= steps) break;
    const int kb = FMT == FP4_MX ? kk >> 1 : kk;
    // MX: an MMA takes two of a scale block's four scales
    const uint32_t sel = FMT == FP4_MX ? static_cast<uint32_t>(kk & 1) * 2u : 0u;
    umma_fp4<FMT, PAIR>(d, wd + 2 * kk, xd + 2 * kk, idesc | (sel << 4) | (sel << 29), sf + kb * 4,
                        sf + 16 + kb * 8 + x_col, first && kk == 0 ? 0u : 1u);
  }
}

__device__ __forceinline__ void bar_sync_group(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(128) : "memory");
}
// All threads of the group agree: every one's `ok`.
__device__ __forceinline__ bool bar_and_group(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "r"(id), "r"(128)
      : "memory");
  return r != 0;
}

// Rows of x into shared memory as the MMA takes them: per stage 16 rows of 128
// swizzled bytes of codes and the scale blocks, stages [k_first, k_end).  Elements
// past K are 0; rows past the last are left as they are (their columns are never read).
template <class A, int FMT>
__device__ __forceinline__ void quantize_to_smem(const GemmParams &p, uint8_t *codes, uint8_t *scales, int k_first,
                                                 int k_end, int tid, int threads) {
  constexpr int B = Fp4<FMT>::kBlock, AHEAD = 64 / B;   // 128 bytes in flight per thread
  const int per_row = (k_end - k_first) * (kStageK / B);   // scales of a row's stages, padding included
  const int n = per_row * p.x_tokens;
  for (int i0 = tid; i0 < n; i0 += AHEAD * threads) {
    uint4 v[AHEAD][B / 8];
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int i = i0 + a * threads, row = i / per_row, k0 = (i - row * per_row) * B + k_first * kStageK;
      const bool in = i < n && k0 < p.K;
      const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.x) +
                                                         static_cast<int64_t>(row) * p.K + k0);
#pragma unroll
      for (int q = 0; q < B / 8; ++q) v[a][q] = in ? __ldg(src + q) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int a = 0; a < AHEAD; ++a) {
      const int i = i0 + a * threads, row = i / per_row, j = i - row * per_row + k_first * (kStageK / B), k0 = j * B;
      if (i >= n) break;
      uint32_t amax = amax_pairs<A>(v[a][0], v[a][1]);
      if (B == 32) amax = max(amax, amax_pairs<A>(v[a][B / 8 - 2], v[a][B / 8 - 1]));
      float inv;
      const uint32_t byte = fp4_scale_of<FMT>(amax, p.xq, inv);
      uint32_t c[B / 8];
#pragma unroll
      for (int q = 0; q < B / 8; ++q) c[q] = fp4_code8<A>(v[a][q], inv);
      uint8_t *dst = codes + (k0 / kStageK) * (kFuseRows * 128) + row * 128 +
                     ((((k0 % kStageK) / 32) ^ (row & 7)) << 4) + (k0 % 32) / 2;
      if (B == 16)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(c[0], c[1]);
      else
        *reinterpret_cast<uint4 *>(dst) = make_uint4(c[0], c[1], c[B / 8 - 2], c[B / 8 - 1]);
      scales[(j >> 2) * kSfBytes + row * 16 + (j & 3)] = k0 < p.K ? static_cast<uint8_t>(byte) : 0;
    }
  }
}

// A group's run of `tokens` rows out of the exchange buffer: features of the
// weight tile at column n0 of an [.., N] output.  `cols`: null, or the buffer row
// of each.  `wide`: rows start at 16-byte boundaries, 16-byte stores; else pairs
// from each row's first 4-byte boundary on, single values around them.
__device__ __forceinline__ void store_rows(const uint16_t *ex, uint16_t *out, int N, int n0, int tokens,
                                           int tid, bool wide, const int *cols) {
  const int hi = min(kSfRows, N - n0);
  if (wide) {
    const int f = (tid & 15) * 8;
    if (f >= hi) return;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = (tid >> 4) + 8 * i;
      v[i] = *reinterpret_cast<const uint4 *>(ex + (cols ? cols[tok] : tok) * kYPitch + f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = (tid >> 4) + 8 * i;
      if (tok < tokens) *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(tok) * N + n0 + f) = v[i];
    }
    return;
  }
  for (int tok = tid >> 5; tok < tokens; tok += 4) {
    uint16_t *dst = out + static_cast<int64_t>(tok) * N + n0;
    const uint16_t *src = ex + (cols ? cols[tok] : tok) * kYPitch;
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(dst) >> 1) & 1;
    for (int f = (tid & 31) * 2 - odd; f < hi; f += 64) {
      const bool a = f >= 0, b = f + 1 < hi;
      if (a && b)
        *reinterpret_cast<uint32_t *>(dst + f) = src[f] | static_cast<uint32_t>(src[f + 1]) << 16;
      else if (a)
        dst[f] = src[f];
      else if (b)
        dst[f + 1] = src[f + 1];
    }
  }
}

// ------------------------------------------------------------------ kernel --

// The tensor maps: weights' codes, activations' codes in large and small boxes
// and, for pairs, the scale blocks of both.
struct GemmMaps {
  CUtensorMap w, x, xb, sfw, sfx;
};

// The group table of offsets that go backwards, entry by entry, by one lane of a warp;
// returns the number of tiles.  (A function of its own, not unrolled: inline it cost
// ascending tables 0.2 to 0.4 us, and so did raising every table's entries in the loop
// that fills it; one token through 8 of 64 experts takes 19.0 us.)
__device__ __noinline__ int raise_table(const int *offsets, int groups, int rows, int max_group, int bt, int n_tiles,
                                        int *table) {
  int *first = table + groups + 1;
  int total = 0;
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
#pragma unroll 1
    for (int e = 0, top = 0; e < groups; ++e) {
      top = raised_offset(__ldg(offsets + e), top, rows);
      const int end = raised_offset(__ldg(offsets + e + 1), top, rows);
      table[e] = top;
      table[e + 1] = end;
      first[e] = total;
      total += token_tiles(min(end - top, max_group), bt) * n_tiles;
    }
    first[groups] = total;
  }
  return __shfl_sync(0xffffffffu, total, 0);
}

// How a tile's work is shared: one CTA, a cluster that splits K, a CTA pair.  (A
// template: the code of the others in a lone CTA's kernel cost a 1 x 2048 x 8192 product
// half a microsecond.)
enum Mode : int { LONE = 0, SPLIT = 1, PAIRED = 2 };

template <class A, int FMT, bool SWIGLU, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ GemmMaps maps) {
  constexpr bool PAIR = MODE == PAIRED;
  constexpr int kSfPerStage = kStageK / Fp4<FMT>::kSfK;   // scale blocks per stage: 2 (MX), 4 (NV)
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], mma_done;
  __shared__ uint32_t tmem_slot;
  __shared__ uint64_t x_ready, part_ready;
  __shared__ int fills[4];      // stages that each producer has requested
  __shared__ int abort_word, rec_count, cols[32];
  volatile int *abort_flag = &abort_word;
  int *table = reinterpret_cast<int *>(smem + p.table_off);
  TileRec *recs = reinterpret_cast<TileRec *>(smem + p.rec_off);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  unsigned int *err = &g_fp4_error;
  const int S = p.stages;
  const uint32_t rank = PAIR ? cluster_rank() : 0;
  const int split = MODE == SPLIT ? p.split : 1, unit = PAIR ? 2 : split;   // CTAs that share a tile
  const int k_rank = MODE == SPLIT ? static_cast<int>(cluster_rank()) : 0;
  const bool fuse = !PAIR && p.x != nullptr;     // x is quantised here, and stays for all tiles

  if constexpr (kDebugBounds) {
    debug_poison_smem(smem, static_cast<uint32_t>(p.rec_off));
    __syncthreads();
  }
  if (warp == 0) {
    // a lane per barrier pair
    if (lane < S) {
      mbar_init(&full[lane], fuse ? 2 : 4);      // the producers
      mbar_init(&empty[lane], 1);
    } else if (lane >= kMaxStages && lane < kMaxStages + 2) {
      mbar_init(&acc_full[lane - kMaxStages], 1);
      mbar_init(&acc_empty[lane - kMaxStages], PAIR ? 2 * kEpiWarps : kEpiWarps);
    } else if (lane == kMaxStages + 2) {
      mbar_init(&mma_done, 1);
      mbar_init(&x_ready, kEpiWarps);
      mbar_init(&part_ready, split * kEpiWarps);
    } else if (lane == kMaxStages + 3) {
      abort_word = 0;
      for (int r = 0; r < 4; ++r) fills[r] = 0;
    }
    fence_mbar_init();
    if (lane == 0) {
      prefetch_tensormap(&maps.w);
      prefetch_tensormap(&maps.x);
      prefetch_tensormap(&maps.xb);
      if (PAIR) {
        prefetch_tensormap(&maps.sfw);
        prefetch_tensormap(&maps.sfx);
      }
    }
  }
  if (warp == kWarpMma) {
    __syncwarp();
    tmem_alloc_all<PAIR>(&tmem_slot);
  }
  if (warp == kWarpEpi0) {
    // group table: the offsets as they are used (raised_offset: the records below
    // hold the tiles of any table) and the first tile id of each group
    int *first = table + p.groups + 1;
    int total = 0;
    bool backward = false;
    for (int e0 = 0; e0 < p.groups; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, hi = 0;
      if (e < p.groups) {
        hi = p.rows;
        if (p.offsets) {
          lo = raised_offset(__ldg(p.offsets + e), 0, p.rows);
          hi = raised_offset(__ldg(p.offsets + e + 1), 0, p.rows);
        }
      }
      backward |= hi < lo;
      const int tiles = token_tiles(min(hi - lo, p.max_group), p.bt) * p.n_tiles;
      int sum = tiles;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      if (e < p.groups) {
        table[e] = lo;
        first[e] = total + sum - tiles;
        if (e == p.groups - 1) {
          table[p.groups] = hi;
          first[p.groups] = total + sum;
        }
      }
      total += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (__any_sync(0xffffffffu, backward))
      total = raise_table(p.offsets, p.groups, p.rows, p.max_group, p.bt, p.n_tiles, table);
    __syncwarp();
    // this CTA's tiles: every gridDim-th from its own index on
    const int start = static_cast<int>(blockIdx.x) / unit, step = static_cast<int>(gridDim.x) / unit;
    const int count = min(tiles_of(total, start, step), p.recs);
    debug_check(tiles_of(total, start, step) <= p.recs, err);
    for (int j = lane; j < count; j += 32) recs[j] = make_rec<PAIR>(p, table, first, start + j * step, rank);
    if (lane == 0) rec_count = count;
  }
  tc_fence_before();
  __syncthreads();
  if (MODE != LONE) cluster_sync();      // the partners' barriers are ready too
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  // this CTA's stages of K: all, or its part of a split tile's
  const int k_stages = ceil_div(p.K, kStageK);
  const int k_first = k_stages * k_rank / split, k_end = k_stages * (k_rank + 1) / split;
  const int tiles = rec_count;
  if constexpr (kDebugBounds) {
    // every column := NaN before the first product (a warp per lane quarter)
    if (warp >= kWarpEpi0 && warp < kWarpEpi0 + 4) {
      uint32_t nan16[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) nan16[i] = ~0u;
      for (uint32_t col = 0; col < 512; col += 16)
        tmem_st16(tmem + (static_cast<uint32_t>(warp & 3) << 21) + col, nan16);
      tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();
    tc_fence_after();
  }

  // Ring positions are counted, not divided: a division by the run-time stage
  // count in every iteration cost the issuing thread more than its products.
  if (warp == 0 || warp >= kWarpProd1) {
    // --------------------------------------------------------- producers ----
    auto produce = [&](auto role) {
      constexpr int ROLE = decltype(role)::value;
      constexpr bool X = ROLE == X_CODES || ROLE == X_SCALES, SCALES = ROLE == W_SCALES || ROLE == X_SCALES;
      // the weights' first stages go out before the wait
      if (X) griddep_wait();
      if (ROLE == X_CODES) griddep_launch_dependents();
      const int stage = SCALES ? kSfPerStage * kSfBytes * (1 + (fuse ? 0 : p.x_sf)) : (X ? p.x_rows : kSfRows) * 128;
      uint8_t *const base = smem + (SCALES ? p.sf_off + (X ? kSfPerStage * kSfBytes : 0) : X ? p.x_off : p.w_off);
      [[maybe_unused]] const uint32_t leader_full = PAIR ? leader_address(&full[0]) : 0;
      int s = 0, filled = 0;
      uint32_t phase = 1;      // of the wait for a free slot; the first round has none
      bool ok = true;
      for (int j = 0; ok && j < tiles; ++j) {
        const TileRec t = recs[j];
        // codes of x: each CTA of a pair copies half of the tokens; one box of a
        // stage's rows, or small boxes where they come to less (256 experts of
        // 2048 x 2048, 20000 rows unevenly: 144.3 us with large boxes alone, 143.5)
        const int n = PAIR ? t.n / 2 : t.n;
        const bool whole = !X || n > p.x_rows - p.x_box;
        const int boxes = whole ? 1 : ceil_div(n, p.x_box);
        const int row = X ? t.row + (PAIR ? static_cast<int>(rank) * n : 0) : t.e * p.N + t.w0;
        const CUtensorMap *tm = !X ? &maps.w : whole ? &maps.x : &maps.xb;
        // scale row blocks: a pair's box always holds x_sf of x
        const int block = X ? t.x_block : t.w_block;
        const int blocks = !X ? 1 : PAIR ? p.x_sf : ceil_div((t.t0 & (kSfRows - 1)) + t.n, kSfRows);
        [[maybe_unused]] const uint8_t *src = (X ? p.x_scales : p.w_scales) + static_cast<int64_t>(block) * p.k_blocks * kSfBytes;
        const uint32_t bytes = SCALES ? blocks * kSfPerStage * kSfBytes : whole ? stage : boxes * p.x_box * 128;
        debug_check(blocks <= p.x_sf && (!X || SCALES || n * 128 <= static_cast<int>(bytes)), err);
        for (int ks = k_first; ks < k_end; ++ks) {
          if (filled >= S && !mbar_wait(&empty[s], phase, abort_flag, p.timeout_ns, err)) {
            ok = false;
            break;
          }
          uint8_t *dst = base + s * stage;
          if constexpr (PAIR) {
            // the leader's barrier counts both CTAs' bytes
            const uint32_t bar = leader_full + s * 8;
            if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * bytes);
            if constexpr (SCALES) {
              tma_load_3d_pair(dst, X ? &maps.sfx : &maps.sfw, bar, 0, ks * kSfPerStage, block);
            } else {
              tma_load_2d_pair(dst, tm, bar, ks * 128, row);
              for (int b = 1; b < boxes; ++b)
                tma_load_2d_pair(dst + b * p.x_box * 128, tm, bar, ks * 128, row + b * p.x_box);
            }
          } else if constexpr (SCALES) {
            const int nkb = min(kSfPerStage, p.k_blocks - ks * kSfPerStage) * kSfBytes;
            mbar_arrive_expect_tx(&full[s], nkb * blocks);
            for (int b = 0; b < blocks; ++b)
              bulk_load(dst + b * kSfPerStage * kSfBytes,
                        src + (static_cast<int64_t>(b) * p.k_blocks + ks * kSfPerStage) * kSfBytes, nkb, &full[s]);
          } else {
            mbar_arrive_expect_tx(&full[s], bytes);
            tma_load_2d(dst, tm, &full[s], ks * 128, row);
            for (int b = 1; b < boxes; ++b)
              tma_load_2d(dst + b * p.x_box * 128, tm, &full[s], ks * 128, row + b * p.x_box);
          }
          ++filled;
          if (++s == S) {
            s = 0;
            phase ^= 1;
          }
        }
      }
      fills[ROLE] = filled;
    };
    const bool x_side = warp == kWarpProd1 || warp == kWarpProd1 + 2;
    if (elect_one() && !(fuse && x_side) && !(p.withhold && warp == 0)) {
      if (warp == 0)
        produce(std::integral_constant<int, W_CODES>());
      else if (warp == kWarpProd1)
        produce(std::integral_constant<int, X_CODES>());
      else if (warp == kWarpProd1 + 1)
        produce(std::integral_constant<int, W_SCALES>());
      else
        produce(std::integral_constant<int, X_SCALES>());
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // --------------------------------------------------------- MMA issuer ---
    // Of a pair, only the leader's issues, for both CTAs.
    // The whole warp walks the tiles and waits, one elected lane issues: with
    // control flow and operands the same in all lanes, descriptors and
    // addresses live in uniform registers, as these instructions want them.
    const bool issuer = elect_one();
    const uint32_t x_stage = p.x_rows * 128 >> 4, w_stage = kSfRows * 128 >> 4;
    const uint32_t sf_stage = kSfPerStage * kSfBytes * (1 + (fuse ? 0 : p.x_sf)) >> 4;
    const uint64_t sfx0 = scales_desc(smem_u32(smem + p.fuse_sf_off));
    const uint64_t wd0 = umma_desc_sw128(smem_u32(smem + p.w_off));
    const uint64_t xd0 = umma_desc_sw128(smem_u32(smem + p.x_off));
    const uint64_t sfd0 = scales_desc(smem_u32(smem + p.sf_off));
    const int steps_all = ceil_div(p.K, 64);
    int s = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.timeout_ns, err)) != 0;
    };
    if (fuse && tiles > 0) ok = wait(&x_ready, 0);
    for (int j = 0; ok && rank == 0 && j < tiles; ++j) {
      const int buf = j & 1;
      const int n = __shfl_sync(0xffffffffu, recs[j].n, 0), t0 = __shfl_sync(0xffffffffu, recs[j].t0, 0);
      ok = wait(&acc_empty[buf], ((j >> 1) & 1) ^ 1u);
      if (!ok) break;
      const uint32_t d = tmem + buf * kTileTokens;
      const uint32_t idesc = fp4_idesc<FMT, PAIR>(n);
      const uint32_t x_col = (t0 & 64) ? 2u : 0u;        // scale column of the tile's first token
      const int x_sf = ceil_div((t0 & (kSfRows - 1)) + n, kSfRows);
      int kb_left = p.k_blocks - k_first * kSfPerStage, steps_left = steps_all - k_first * (kStageK / 64);
      for (int ks = k_first; ks < k_end; ++ks) {
        ok = wait(&full[s], phase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sf = tmem + kSfCol + (it & 1) * kSfCols;
        const uint64_t wd = wd0 + s * w_stage, xd = xd0 + (fuse ? ks : s) * x_stage, sfw = sfd0 + s * sf_stage;
        constexpr uint32_t kSfStep = kSfPerStage * kSfBytes >> 4;
        const uint64_t sfx = fuse ? sfx0 + ks * kSfStep : sfw + kSfStep;
        if (issuer) {
          if (x_sf == 1)
            issue_stage<FMT, 1, PAIR>(d, idesc, wd, xd, sf, sfw, sfx, x_col, kb_left, steps_left, ks == k_first);
          else
            issue_stage<FMT, 2, PAIR>(d, idesc, wd, xd, sf, sfw, sfx, x_col, kb_left, steps_left, ks == k_first);
          commit_to<PAIR>(&empty[s]);
        }
        __syncwarp();
        kb_left -= kSfPerStage;
        steps_left -= kStageK / 64;
        ++it;
        if (++s == S) {
          s = 0;
          phase ^= 1;
        }
      }
      if (ok && issuer) commit_to<PAIR>(&acc_full[buf]);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue --
    // Groups of four warps (one per lane quarter) take turns at runs of 32
    // tokens.  The accumulator has features in lanes and tokens in columns; a
    // group turns a run around through shared memory, so that a token's features
    // leave in wide stores.  (Straight from the registers, 2 bytes per lane, a
    // tile of 192 tokens took 4300 cycles, more than its products.)
    const int group = (warp - kWarpEpi0) >> 2;
    const int quarter = warp & 3;                  // the TMEM lanes this warp may read
    const int bar = 1 + group;
    const int gtid = ((warp - kWarpEpi0) & 3) * 32 + lane;         // thread within the group
    uint8_t *ex = smem + p.ex_off + group * kExBytes;
    if (fuse) {
      griddep_wait();
      griddep_launch_dependents();
      const int tid = (warp - kWarpEpi0) * 32 + lane;
      if (p.x_f16)
        quantize_to_smem<ActF16, FMT>(p, smem + p.x_off, smem + p.fuse_sf_off, k_first, k_end, tid, kEpiWarps * 32);
      else
        quantize_to_smem<ActBf16, FMT>(p, smem + p.x_off, smem + p.fuse_sf_off, k_first, k_end, tid, kEpiWarps * 32);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&x_ready);
    }
    for (int j = 0; j < tiles; ++j) {
      const TileRec t = recs[j];
      const int buf = j & 1;
      debug_check(t.row >= 0 && t.row + t.valid <= p.rows && t.w0 >= 0 && t.e < p.groups, err);
      // the column of each of the tile's rows, where all rows of x are columns
      int col = 0;
      if (fuse && group == 0 && gtid < 32 && gtid < t.valid) {
        const int r = p.order ? __ldg(p.order + t.row + gtid) / p.fan : t.row + gtid;
        col = min(max(r, 0), kFuseRows - 1);
      }
      bool ok = mbar_wait(&acc_full[buf], (j >> 1) & 1, abort_flag, p.timeout_ns, err);
      ok = bar_and_group(bar, ok);
      if (!ok) break;
      if (fuse && group == 0 && gtid < 32) cols[gtid] = col;
      tc_fence_after();
      const uint32_t acc = tmem + buf * kTileTokens + (static_cast<uint32_t>(quarter) << 21);
      const int row_in_block = quarter * 32 + lane;
      // The tokens this CTA finishes.  A split tile: every CTA of the cluster lays its
      // partial sums out in shared memory (the stages' space: all of its products
      // are done), and adds all of them up, in rank order, for its share of the tokens.
      int first = 0, count = t.valid;
      float *part = reinterpret_cast<float *>(smem);
      if constexpr (MODE == SPLIT) {
        const int share = ceil_div(t.valid, split);
        first = min(t.valid, k_rank * share);
        count = min(t.valid, first + share) - first;
        for (int c0 = group * 32; c0 < t.n; c0 += 32 * kEpiGroups) {
          uint32_t r[2][16];
          tmem_ld16(acc + c0, r[0]);
          tmem_ld16(acc + c0 + 16, r[1]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < t.n) part[(c0 + c) * kSfRows + row_in_block] = __uint_as_float(r[c >> 4][c & 15]);
        }
        __syncwarp();
        if (lane < split) mbar_arrive_release_cluster(peer_address(&part_ready, lane));
        ok = mbar_wait_cluster(&part_ready, j & 1, abort_flag, p.timeout_ns, err);
        ok = bar_and_group(bar, ok);
        if (!ok) break;
      }
      const float alpha = p.x_scale * (p.w_scale ? __ldg(p.w_scale + t.e) : 1.0f);
      bool released = false;
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_cluster(leader_address(&acc_empty[buf]));
          else
            mbar_arrive(&acc_empty[buf]);
        }
        released = true;
      };
      for (int c0 = group * 32; c0 < count; c0 += 32 * kEpiGroups) {
        uint32_t r[2][16];
        if constexpr (MODE == SPLIT) {
#pragma unroll
          for (int c = 0; c < 32; ++c) r[c >> 4][c & 15] = 0;
          for (int q = 0; q < split; ++q) {
            const uint32_t from = peer_address(part + row_in_block, q);
            float v[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const int i = first + c0 + c;
              v[c] = c0 + c < count ? load_peer(from + (fuse ? cols[i] : i) * (kSfRows * 4)) : 0.0f;
            }
#pragma unroll
            for (int c = 0; c < 32; ++c)
              r[c >> 4][c & 15] = __float_as_uint(__uint_as_float(r[c >> 4][c & 15]) + v[c]);
          }
        } else {
          tmem_ld16(acc + c0, r[0]);
          tmem_ld16(acc + c0 + 16, r[1]);
          tmem_ld_wait();
        }
        if (c0 + 32 * kEpiGroups >= count) release();     // the warp's last look at the accumulator
        if (!SWIGLU && p.out_f32) {
          // 32 lanes store 128 contiguous bytes: no need to turn the run around
          const int n = t.w0 + row_in_block;
          float *out = static_cast<float *>(p.out) + static_cast<int64_t>(t.row + first + c0) * p.N + n;
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (c0 + c < count && n < p.N)
              out[static_cast<int64_t>(c) * p.N] = __uint_as_float(r[c >> 4][c & 15]) * alpha;
        } else if constexpr (!SWIGLU) {
          uint16_t *ex16 = reinterpret_cast<uint16_t *>(ex);
#pragma unroll
          for (int c = 0; c < 32; ++c)
            ex16[c * kYPitch + row_in_block] = A::store(__uint_as_float(r[c >> 4][c & 15]) * alpha);
          bar_sync_group(bar);
          store_rows(ex16, static_cast<uint16_t *>(p.out) + static_cast<int64_t>(t.row + first + c0) * p.N, p.N, t.w0,
                     min(32, count - c0), gtid, p.wide, fuse && MODE != SPLIT ? cols : nullptr);
          bar_sync_group(bar);
        } else {
          // lanes 0-15 hold gate rows, 16-31 the same features' up rows: a
          // swap across the half warps gives the lower half the even
          // tokens' pairs and the upper half the odd tokens'
          const bool upper = lane >= 16;
          float *dst = reinterpret_cast<float *>(ex) + (lane >> 4) * kHPitch + quarter * 16 + (lane & 15);
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float a = __uint_as_float(r[c >> 4][c & 15]) * alpha;
            const float b = __uint_as_float(r[c >> 4][(c & 15) + 1]) * alpha;
            const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
            const float g = upper ? other : a, u = upper ? b : other;
            dst[c * kHPitch] = g * sigmoid_fast(g) * u;
          }
          bar_sync_group(bar);
          // one token's 16 features per thread: the four loads go in an order
          // that keeps the eight threads of a phase on different banks
          const int tok = gtid >> 2, fq = gtid & 3;
          const int f0 = t.w0 / 2 + fq * 16;      // first feature
          const int I = p.N / 2;
          const bool have = c0 + tok < count;
          const float4 *src = reinterpret_cast<const float4 *>(
              reinterpret_cast<float *>(ex) + (fuse && MODE != SPLIT ? cols[tok] : tok) * kHPitch + fq * 16);
          float4 v[4];
          uint32_t amax = 0;
          const int rot = (fq >> 1) + 2 * (tok & 1);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = src[(i + rot) & 3];
            amax = max(max(amax, __float_as_uint(v[i].x) & 0x7FFFFFFFu), __float_as_uint(v[i].y) & 0x7FFFFFFFu);
            amax = max(max(amax, __float_as_uint(v[i].z) & 0x7FFFFFFFu), __float_as_uint(v[i].w) & 0x7FFFFFFFu);
          }
          if (FMT == FP4_MX) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          float inv;
          uint32_t byte = fp4_scale_of<FMT>(amax, p.hq, inv);
          const int tl = t.t0 + first + c0 + tok;       // token within the group
          if (have) {
            const int64_t blk = t.x_block - t.t0 / kSfRows + tl / kSfRows;
            const int j = f0 / Fp4<FMT>::kBlock;
            uint8_t *sc = p.h_scales + (blk * p.h_k_blocks + (j >> 2)) * kSfBytes + (tl & 31) * 16 + ((tl >> 5) & 3) * 4;
            if (f0 < I && (FMT == FP4_NV || (fq & 1) == 0)) {
              sc[j & 3] = static_cast<uint8_t>(byte);
              // the row's last scale: zeros to the end of its scale block
              if (f0 + Fp4<FMT>::kBlock >= I)
                for (int z = (j & 3) + 1; z < 4; ++z) sc[z] = 0;
            }
            if (f0 < I) {
              uint64_t codes = 0;
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                const float q8[8] = {v[i].x * inv,     v[i].y * inv,     v[i].z * inv,     v[i].w * inv,
                                     v[i + 1].x * inv, v[i + 1].y * inv, v[i + 1].z * inv, v[i + 1].w * inv};
                const uint32_t c8 = fp4_pack8(q8);
                codes |= static_cast<uint64_t>(c8 & 0xFFFFu) << (16 * ((i + rot) & 3));
                codes |= static_cast<uint64_t>(c8 >> 16) << (16 * ((i + 1 + rot) & 3));
              }
              const int64_t at = static_cast<int64_t>(t.row + first + c0 + tok);
              *reinterpret_cast<uint64_t *>(p.h_codes + at * (I / 2) + f0 / 2) = codes;
            }
          }
          bar_sync_group(bar);
        }
      }
      if (!released) release();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag && rank == 0) {
    // Given up: let the products and copies already issued finish before tensor and
    // shared memory go away, each wait with a limit.  (A pair's leader waits for
    // both CTAs'; the partner stays until it has.)
    if (warp == kWarpMma && elect_one()) {
      commit_to<PAIR>(&mma_done);
      mbar_wait_drain(&mma_done, 0, 100000000ull);
    }
    if (warp == 0 && lane < 4) {
      const int filled = fills[lane];
      for (int i = 0; i < S && i < filled; ++i) {
        const int last = i + ((filled - 1 - i) / S) * S;
        mbar_wait_drain(&full[i], (last / S) & 1, 100000000ull);
      }
    }
    __syncthreads();
  }
  if (MODE != LONE) cluster_sync();      // nothing of a partner's reaches this CTA any more
  tc_fence_after();
  if (warp == kWarpMma) tmem_free_all<PAIR>(tmem);
}

// -------------------------------------------------------------------- host --

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Codes [rows, K/2] bytes, boxes of 128 bytes by `box` rows, 128-byte swizzle.
bool encode_codes(CUtensorMap *map, const void *base, int64_t rows, int64_t K, int box) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t boxes[2] = {128, static_cast<cuuint32_t>(box)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tokens per group from which CTA pairs are taken.  Where the weights pass L2 pairs gain
// from there on, where they stay in it only from about 320 (us on pairs / on single CTAs,
// at 128, 192, 256, 320, 512 tokens per group; NV):
//   32 x 2048 x 4096    47.1/47.1  53.5/54.1  63.0/65.5  72.5/75.1  96.8/102.5
//   64 x 2048 x 2048    47.7/46.9  54.3/54.6  67.4/69.4  77.2/80.1  102.9/108.7
//    8 x 4096 x 7168    35.8/35.9  41.4/41.8  52.0/54.7  58.4/61.1  77.7/81.9
//   16 x 2048 x 2048    14.6/13.9  17.4/17.0  22.0/21.9  26.2/26.2  34.9/35.9
//    1 x 14336 x 4096   12.0/11.0  12.8/12.2  16.4/16.1  18.1/18.1  22.8/23.1
//    1 x 10240 x 2560    9.5/9.0   10.5/10.0  12.4/12.1  13.8/13.4  14.6/14.5
constexpr int kPairTokens = 192;
// Stages of K from which a tile is split.
constexpr int kSplitStages = 24;

constexpr int kSmemLimit = 227 * 1024 - 1024;   // less the static part

int align_up(int v, int a) { return (v + a - 1) / a * a; }

// Scale blocks [row blocks, k blocks] of 512 bytes as 128 words each; a box is a
// stage's blocks of `rows` row blocks.
bool encode_scales(CUtensorMap *map, const void *base, int64_t row_blocks, int64_t k_blocks, int per_stage, int rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {kSfBytes / 4, static_cast<cuuint64_t>(k_blocks), static_cast<cuuint64_t>(row_blocks)};
  const cuuint64_t strides[2] = {kSfBytes, static_cast<cuuint64_t>(k_blocks) * kSfBytes};
  const cuuint32_t boxes[3] = {kSfBytes / 4, static_cast<cuuint32_t>(per_stage), static_cast<cuuint32_t>(rows)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void *>(base), dims, strides, boxes, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class A, int FMT, bool SWIGLU, int MODE>
cudaError_t launch_gemm(const Fp4GemmArgs &a, GemmParams p, int num_sms, cudaStream_t stream, bool dependent) {
  constexpr int kSfPerStage = kStageK / Fp4<FMT>::kSfK;
  constexpr bool PAIR = MODE == PAIRED;
  auto *kernel = fp4_gemm_kernel<A, FMT, SWIGLU, MODE>;
  static std::once_flag once[64];
  static cudaError_t attr[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    attr[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  });
  if (attr[dev] != cudaSuccess) return attr[dev];

  // shared memory: x stages, weight stages, scale stages, exchange buffers,
  // tile records, group table
  const int ex = kEpiGroups * kExBytes;
  const int table = align_up(2 * (p.groups + 1) * 4, 16);
  // CTAs (pairs): one per SM (two SMs), no more than tiles can exist, and no more
  // tiles each than there are records
  const TilePlan plan = plan_tiles(most_tiles(p.rows, p.groups, p.bt, p.n_tiles), num_sms, PAIR ? 2 : p.split);
  if (plan.slots > (1 << 30)) return cudaErrorInvalidValue;
  p.recs = static_cast<int>(plan.recs);
  const int recs = p.recs * static_cast<int>(sizeof(TileRec));
  const bool fuse = p.x != nullptr;
  const int k_stages = ceil_div(p.K, kStageK);
  const int x_stage = fuse ? 0 : p.x_rows * 128, w_stage = kSfRows * 128;
  const int sf_stage = kSfPerStage * kSfBytes * (1 + (fuse ? 0 : p.x_sf));
  const int x_all = fuse ? k_stages * kFuseRows * 128 : 0, x_sf_all = fuse ? k_stages * kSfPerStage * kSfBytes : 0;
  const int fixed = 1024 + ex + recs + table + x_all + x_sf_all;
  int S = (kSmemLimit - fixed) / (x_stage + w_stage + sf_stage);
  if (S > kMaxStages) S = kMaxStages;
  if (S < 2) return cudaErrorInvalidValue;
  p.stages = S;
  p.x_off = 0;
  const int x_bytes = x_all + S * x_stage;
  p.w_off = align_up(x_bytes, 1024);
  p.sf_off = p.w_off + S * w_stage;
  p.fuse_sf_off = p.sf_off + S * sf_stage;
  p.ex_off = align_up(p.fuse_sf_off + x_sf_all, 128);
  p.rec_off = p.ex_off + ex;
  p.table_off = p.rec_off + recs;
  const int bytes = p.table_off + table + 1024;   // and the base's alignment
  if (bytes > kSmemLimit) return cudaErrorInvalidValue;

  GemmMaps maps;
  if (!encode_codes(&maps.w, a.w_codes, static_cast<int64_t>(p.groups) * p.N, p.K, kSfRows))
    return cudaErrorInvalidValue;
  maps.x = maps.w;
  if (!fuse && !encode_codes(&maps.x, a.x_codes, p.rows, p.K, p.x_rows)) return cudaErrorInvalidValue;
  maps.xb = maps.x;
  if (!fuse && p.x_box != p.x_rows && !encode_codes(&maps.xb, a.x_codes, p.rows, p.K, p.x_box))
    return cudaErrorInvalidValue;
  maps.sfw = maps.sfx = maps.x;
  if (PAIR) {
    const int64_t x_blocks = a.offsets ? ragged_row_block(p.rows, p.groups) : ceil_div(p.rows, kSfRows);
    if (!encode_scales(&maps.sfw, a.w_scales, static_cast<int64_t>(p.groups) * p.w_row_blocks, p.k_blocks, kSfPerStage,
                       1) ||
        !encode_scales(&maps.sfx, a.x_scales, x_blocks, p.k_blocks, kSfPerStage, p.x_sf))
      return cudaErrorInvalidValue;
  }
  const int unit = PAIR ? 2 : p.split;
  const int grid = static_cast<int>(plan.slots) * unit;
  if (p.split > 1 && p.bt * kSfRows * 4 > p.ex_off) return cudaErrorInvalidValue;   // the partial sums' space
  return launch_clusters(kernel, dim3(static_cast<unsigned>(grid)), unit, kThreads, static_cast<size_t>(bytes),
                         stream, dependent, p, maps);
}

template <int MODE>
cudaError_t dispatch_gemm(const Fp4GemmArgs &a, const GemmParams &p, int num_sms, cudaStream_t stream,
                          bool dependent) {
  const bool mx = a.fmt == FP4_MX;
  if (a.swiglu)
    return mx ? launch_gemm<ActBf16, FP4_MX, true, MODE>(a, p, num_sms, stream, dependent)
              : launch_gemm<ActBf16, FP4_NV, true, MODE>(a, p, num_sms, stream, dependent);
  if (a.act == ActF16::kId)
    return mx ? launch_gemm<ActF16, FP4_MX, false, MODE>(a, p, num_sms, stream, dependent)
              : launch_gemm<ActF16, FP4_NV, false, MODE>(a, p, num_sms, stream, dependent);
  return mx ? launch_gemm<ActBf16, FP4_MX, false, MODE>(a, p, num_sms, stream, dependent)
            : launch_gemm<ActBf16, FP4_NV, false, MODE>(a, p, num_sms, stream, dependent);
}

}  // namespace

// Whether every CTA quantises `rows` rows of x itself: one launch instead of two, as
// long as there is little of it (N = 8192: 1 x 2048 6.55 us against 6.94 with a launch
// of its own, 4 x 2048 6.78 and 6.95, 8 x 2048 7.20 and 6.94) and its codes and scales
// leave most of the shared memory to the weights' stages.
bool fp4_gemm_quantizes(int64_t rows, int64_t K, int fmt) {
  const int64_t stages = (K + kStageK - 1) / kStageK;
  const int64_t bytes = stages * (kFuseRows * 128 + kStageK / (4 * fp4_block(fmt)) * kSfBytes);
  return rows <= kFuseRows && rows * K <= kFuseElements && bytes <= 96 * 1024;
}

cudaError_t launch_fp4_gemm(const Fp4GemmArgs &a, int num_sms, uint64_t timeout_ns, cudaStream_t stream,
                            bool dependent) {
  if (num_sms <= 0) return cudaErrorInvalidDevice;
  GemmParams p = {};
  p.w_scales = a.w_scales;
  p.x_scales = a.x_scales;
  p.offsets = a.offsets;
  p.w_scale = a.w_scale;
  p.x_scale = a.x_scale;
  p.groups = a.groups;
  p.rows = static_cast<int>(a.rows);
  p.max_group = static_cast<int>(a.max_group < a.rows ? a.max_group : a.rows);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.k_blocks = static_cast<int>(fp4_k_blocks(a.K, a.fmt));
  p.w_row_blocks = ceil_div(p.N, kSfRows);
  p.bt = p.max_group >= kTileTokens ? kTileTokens : align_up(p.max_group, 16);
  p.x_sf = p.max_group > 128 ? 2 : 1;
  p.out = a.out;
  p.out_f32 = a.out_f32;
  p.wide = a.N % 8 == 0 && reinterpret_cast<uintptr_t>(a.out) % 16 == 0;
  p.h_codes = a.h_codes;
  p.h_scales = a.h_scales;
  p.h_k_blocks = a.swiglu ? static_cast<int>(fp4_k_blocks(a.N / 2, a.fmt)) : 0;
  p.hq = make_fp4_scale(a.h_scale);
  p.timeout_ns = timeout_ns;
  p.withhold = g_withhold.exchange(0, std::memory_order_relaxed);

  if (a.x) {
    p.x = a.x;
    p.xq = make_fp4_scale(a.x_scale);
    p.x_f16 = a.act == ActF16::kId;
    p.x_tokens = static_cast<int>(a.x_tokens);
    p.order = a.order;
    p.fan = a.fan;
  }

  // (group, token tile) pairs there can be at most
  const int64_t groups = p.groups < p.rows ? p.groups : p.rows;
  const int64_t tiles = most_tiles(p.rows, p.groups, p.bt, 1);

  // CTA pairs share a tile of 256 weight rows: each copies its own 128 rows and
  // half of the tokens, which leaves an SM a quarter less to copy per product.
  // With few tokens per group the weights are all there is to copy, and the tiles
  // are better spread over single CTAs.
  if (!p.x && p.rows / groups >= kPairTokens && tiles * ceil_div(p.N, 256) * 2 >= num_sms) {
    p.bt = align_up(p.bt, 32);
    p.x_rows = p.bt / 2;
    p.x_box = p.x_rows < 32 ? p.x_rows : 32;
    p.x_rows = align_up(p.x_rows, p.x_box);
    p.n_tiles = ceil_div(p.N, 2 * kSfRows);
    p.split = 1;
    return dispatch_gemm<PAIRED>(a, p, num_sms, stream, dependent);
  }

  p.x_box = p.bt < 64 ? p.bt : 64;
  p.x_rows = align_up(p.bt, p.x_box);
  p.n_tiles = ceil_div(p.N, kSfRows);

  // Few tiles and a long K: a cluster of 4 or 2 CTAs shares a tile's K.  A tile's time
  // is 4.5 us and 0.28 us per stage of its chain, the cluster's barriers and the
  // sum cost about 1.5 us, more with many tokens (N = 2048, M = 1: K = 8192 13.6 -> 10.6
  // us with 4, K = 4096 9.2 -> 9.0, K = 2048 7.2 -> 8.2; M = 128, K = 8192: 14.6 us,
  // with 2 13.7, with 4 14.9).  Clusters of 4 fill 128 of the SMs.
  p.split = 1;
  if (ceil_div(p.K, kStageK) >= kSplitStages) {
    if (p.bt <= 64 && tiles * p.n_tiles * 4 <= num_sms * 27 / 32)
      p.split = 4;
    else if (tiles * p.n_tiles * 2 <= num_sms)
      p.split = 2;
  }
  return p.split > 1 ? dispatch_gemm<SPLIT>(a, p, num_sms, stream, dependent)
                     : dispatch_gemm<LONE>(a, p, num_sms, stream, dependent);
}

void fp4_gemm_withhold_next() { g_withhold.store(1); }

// Read and clear the device error word of this translation unit's kernels.
cudaError_t fp4_gemm_take_errors(unsigned int *out) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp4_error, sizeof v);
  if (e != cudaSuccess) return e;
  if (v) {
    e = cudaMemcpyToSymbol(g_fp4_error, &zero, sizeof zero);
    if (e != cudaSuccess) return e;
  }
  *out = v;
  return cudaSuccess;
}

}  // namespace qsw
