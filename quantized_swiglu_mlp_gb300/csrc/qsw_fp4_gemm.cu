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
// without a second kernel.  Where the 128-row tiles would not fill the SMs, a tile
// is 64, 32 or 16 rows (`rt`): only those rows are copied, the MMA still reads 128
// -- the others hold whatever shared memory holds, and their accumulator lanes
// are never read.  The rows keep their place r mod 128, so that the scale block's
// lanes fit: the A descriptor starts that many rows before the copied ones.
//
// One persistent CTA per SM, 11 warps: warps 0 and 10 issue the weights' and the
// activations' copies (a ring of stages of 256 elements of K: 128-byte swizzled
// code tiles by TMA, scale blocks by bulk copies), warp 1 moves the scales into
// tensor memory and issues the MMAs, warps 2-9 run the epilogue.  Tensor memory: two accumulators of 192
// columns, so that a tile's epilogue runs under the next tile's products, and
// two scale buffers of 48 columns.
//
// Programmatic dependent launch: everything a CTA does before griddep_wait --
// the group table, the weights of its first stages -- reads only what was
// complete before the launch in front of this one began (each kernel of a chain
// lets the next one start only after its own wait).
#include <mutex>

#include "qsw_fp4.cuh"
#include "qsw_internal.h"

namespace qsw {
namespace {

__device__ unsigned int g_fp4_error;

constexpr int kTileTokens = 192;
constexpr int kMaxStages = 16;
constexpr int kEpiWarps = 8;
constexpr int kWarpW = 0, kWarpMma = 1, kWarpEpi0 = 2, kWarpX = kWarpEpi0 + kEpiWarps;
constexpr int kThreads = 32 * (kWarpX + 1);
constexpr int kStageK = 256;                 // elements of K per stage: one 128-byte swizzle row
constexpr int kSfCol = 2 * kTileTokens;      // first scale column of tensor memory
constexpr int kSfCols = 48;                  // per scale buffer: 16 weight, 32 token columns
constexpr int kXPitch = 80;                  // floats per token row of the epilogue's exchange buffer
constexpr int kXBytes = 32 * kXPitch * 4;    // one buffer: 32 tokens

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
  int n_tiles;              // weight tiles of `rt` rows per group
  int k_blocks;             // scale blocks along K
  int w_row_blocks;         // scale row blocks of a group's weights
  int rt, bt;               // weight rows and most tokens of a tile
  int x_box, x_rows;        // rows of the small TMA box of x, and of a stage (the large box)
  int x_sf;                 // scale row blocks of x in a stage
  int stages;
  int x_off, w_off, sf_off, ex_off, table_off;   // byte offsets in shared memory
  void *out;
  uint8_t *h_codes;
  uint8_t *h_scales;
  int h_k_blocks;
  Fp4Scale hq;
  uint64_t timeout_ns;
};

struct Tile {
  int e;        // group
  int off;      // its first row
  int t0;       // first token of the tile within the group
  int valid;    // tokens
  int n;        // valid rounded up to the MMA's step
  int w0;       // first weight row within the group
};

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Token tiles of a group of m rows; more than one tile: equal sizes, multiples
// of 64 (the scale lanes of a tile then start at column 0 or 2 of a block).
__device__ __forceinline__ int token_tiles(int m, int bt) { return ceil_div(m, bt); }

// Walks the CTA's tiles: tile ids count up, token tiles fastest, then weight
// tiles, then groups.
struct TileWalk {
  const int *off;     // [groups + 1] in shared memory
  const int *first;   // [groups + 1] first tile id of each group
  int id, e;
  __device__ __forceinline__ TileWalk(const int *table, const GemmParams &p)
      : off(table), first(table + p.groups + 1), id(static_cast<int>(blockIdx.x)), e(0) {}
  __device__ __forceinline__ bool get(const GemmParams &p, Tile &t) {
    if (id >= first[p.groups]) return false;
    while (id >= first[e + 1]) ++e;
    const int m = min(off[e + 1] - off[e], p.max_group);
    const int nt = token_tiles(m, p.bt);
    const int local = id - first[e];
    const int wt = local / nt, tt = local - wt * nt;
    const int size = nt > 1 ? (ceil_div(m, nt) + 63) & ~63 : m;
    t.e = e;
    t.off = off[e];
    t.t0 = tt * size;
    t.valid = min(size, m - t.t0);
    t.n = max(16, (t.valid + 15) & ~15);
    t.w0 = wt * p.rt;
    return true;
  }
  __device__ __forceinline__ void next() { id += static_cast<int>(gridDim.x); }
};

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
__device__ __forceinline__ void scales_to_tmem(uint32_t taddr, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// One thread of a converged warp.  The copies and products are issued by a
// thread chosen this way: the compiler then keeps their operands in uniform
// registers (chosen with `lane == 0`, each instruction took about 100 cycles).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

template <int FMT>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t accumulate) {
  if (FMT == FP4_MX)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}

// Instruction descriptor: e2m1 A and B, M = 128; N / 8 and the scale selectors
// are added per tile and per step.
template <int FMT>
__device__ __forceinline__ uint32_t fp4_idesc(int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (FMT == FP4_MX ? 1u << 23 : 0u) |   // E8M0 or E4M3 scales
         (8u << 24);                         // M / 16
}

// The copies and products of one stage: `nkb` scale blocks, `steps` products of 64
// elements of K.  One thread's copies and products run in the order of issue.
template <int FMT, int XSF>
__device__ __forceinline__ void issue_stage(uint32_t d, uint32_t idesc, uint64_t wd, uint64_t xd, uint32_t sf,
                                            uint64_t sfd, uint32_t x_col, int nkb, int steps, bool first) {
  constexpr int kSfPerStage = kStageK / Fp4<FMT>::kSfK;
#pragma unroll
  for (int kb = 0; kb < kSfPerStage; ++kb) {
    if (kb >= nkb) break;
    scales_to_tmem(sf + kb * 4, sfd + kb * (kSfBytes >> 4));
#pragma unroll
    for (int b = 0; b < XSF; ++b)
      scales_to_tmem(sf + 16 + kb * 8 + b * 4, sfd + (kSfPerStage * (1 + b) + kb) * (kSfBytes >> 4));
  }
#pragma unroll
  for (int kk = 0; kk < kStageK / 64; ++kk) {
    if (kk >= steps) break;
    const int kb = FMT == FP4_MX ? kk >> 1 : kk;
    // MX: an MMA takes two of a scale block's four scales
    const uint32_t sel = FMT == FP4_MX ? static_cast<uint32_t>(kk & 1) * 2u : 0u;
    umma_fp4<FMT>(d, wd + 2 * kk, xd + 2 * kk, idesc | (sel << 4) | (sel << 29), sf + kb * 4, sf + 16 + kb * 8 + x_col,
                  first && kk == 0 ? 0u : 1u);
  }
}

__device__ __forceinline__ void bar_sync_half(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(kEpiWarps * 16) : "memory");
}
// All threads of the half agree: every one's `ok`.
__device__ __forceinline__ bool bar_and_half(int id, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok ? 1u : 0u), "r"(id), "r"(kEpiWarps * 16)
      : "memory");
  return r != 0;
}

// ------------------------------------------------------------------ kernel --

template <class A, int FMT, bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ GemmParams p, const __grid_constant__ CUtensorMap tm_w,
                    const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_xb) {
  constexpr int kSfPerStage = kStageK / Fp4<FMT>::kSfK;   // scale blocks per stage: 2 (MX), 4 (NV)
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], mma_done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int *abort_flag = &abort_word;
  int *table = reinterpret_cast<int *>(smem + p.table_off);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  unsigned int *err = &g_fp4_error;
  const int S = p.stages;

  if constexpr (kDebugBounds) {
    debug_poison_smem(smem, static_cast<uint32_t>(p.table_off));
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 2);      // both producers
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    mbar_init(&mma_done, 1);
    abort_word = 0;
    fence_mbar_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
    prefetch_tensormap(&tm_xb);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  if (warp == kWarpEpi0) {
    // group table: offsets (clamped, so that no table of the caller leads
    // outside the buffers) and the first tile id of each group
    int *first = table + p.groups + 1;
    int total = 0;
    for (int e0 = 0; e0 < p.groups; e0 += 32) {
      const int e = e0 + lane;
      int lo = 0, hi = 0;
      if (e < p.groups) {
        hi = p.rows;
        if (p.offsets) ragged_range(p.offsets, e, p.rows, lo, hi);
      }
      int tiles = token_tiles(min(hi - lo, p.max_group), p.bt) * p.n_tiles;
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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  const int k_stages = ceil_div(p.K, kStageK);

  // Ring positions are counted, not divided: a division by the run-time stage
  // count in every iteration cost the issuing thread more than its products.
  if (warp == kWarpW || warp == kWarpX) {
    // --------------------------------------------------------- producers ----
    // One warp copies the weights' codes and scales, another the
    // activations': each stage's barrier gets one arrival from both.
    if (elect_one()) {
      const bool w_side = warp == kWarpW;
      const int stage = (w_side ? p.rt : p.x_rows) * 128;
      const int sf_stage = kSfPerStage * kSfBytes * (1 + p.x_sf);
      uint8_t *codes = smem + (w_side ? p.w_off : p.x_off);
      uint8_t *sf = smem + p.sf_off + (w_side ? 0 : kSfPerStage * kSfBytes);
      TileWalk walk(table, p);
      Tile t;
      int s = 0, filled = 0;
      uint32_t phase = 1;      // parity that a free slot's barrier shows: the first round passes at once
      bool ok = true, more = walk.get(p, t);
      // the weights' first stages go out before the wait
      if (!w_side) {
        griddep_wait();
        griddep_launch_dependents();
      }
      while (more && ok) {
        const int64_t block = w_side ? static_cast<int64_t>(t.e) * p.w_row_blocks + t.w0 / kSfRows
                                     : (p.offsets ? ragged_row_block(t.off, t.e) : 0) + t.t0 / kSfRows;
        const uint8_t *sf_src = (w_side ? p.w_scales : p.x_scales) + block * p.k_blocks * kSfBytes;
        const int64_t sf_row = static_cast<int64_t>(p.k_blocks) * kSfBytes;
        const int blocks = w_side ? 1 : ceil_div(t.t0 + t.n, kSfRows) - t.t0 / kSfRows;
        const int row = w_side ? t.e * p.N + t.w0 : t.off + t.t0;
        // x: one box of bt rows, or boxes of 64 where they come to less
        const int boxes = w_side || t.n > p.x_rows - p.x_box ? 1 : ceil_div(t.n, p.x_box);
        const bool whole = w_side || t.n > p.x_rows - p.x_box;
        const int bytes = whole ? stage : boxes * p.x_box * 128;
        const CUtensorMap *tm = w_side ? &tm_w : whole ? &tm_x : &tm_xb;
        debug_check(blocks <= p.x_sf && t.n * 128 <= (w_side ? kSfRows * 256 : bytes), err);
        for (int ks = 0; ks < k_stages; ++ks) {
          const int nkb = min(kSfPerStage, p.k_blocks - ks * kSfPerStage) * kSfBytes;
          if (!mbar_wait(&empty[s], phase, abort_flag, p.timeout_ns, err)) {
            ok = false;
            break;
          }
          uint64_t *bar = &full[s];
          mbar_arrive_expect_tx(bar, bytes + nkb * blocks);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(codes + s * stage + b * p.x_box * 128, tm, bar, ks * 128, row + b * p.x_box);
          for (int b = 0; b < blocks; ++b)
            bulk_load(sf + s * sf_stage + b * kSfPerStage * kSfBytes, sf_src + b * sf_row, nkb, bar);
          sf_src += kSfPerStage * kSfBytes;
          ++filled;
          if (++s == S) {
            s = 0;
            phase ^= 1;
          }
        }
        walk.next();
        more = walk.get(p, t);
      }
      if (!ok) {
        // let the copies already issued land before the CTA's memory goes away
        for (int i = 0; i < S && i < filled; ++i) {
          const int last = i + ((filled - 1 - i) / S) * S;
          mbar_wait_drain(&full[i], (last / S) & 1, 100000000ull);
        }
      }
    }
    __syncwarp();
  } else if (warp == kWarpMma) {
    // --------------------------------------------------------- MMA issuer ---
    // The whole warp walks the tiles and waits, one elected lane issues: with
    // control flow and operands the same in all lanes, descriptors and
    // addresses live in uniform registers, as these instructions want them.
    const bool issuer = elect_one();
    const uint32_t x_stage = p.x_rows * 128 >> 4, w_stage = p.rt * 128 >> 4;
    const uint32_t sf_stage = kSfPerStage * kSfBytes * (1 + p.x_sf) >> 4;
    TileWalk walk(table, p);
    Tile t;
    int s = 0, n_tile = 0;
    uint32_t phase = 0, it = 0;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.timeout_ns, err)) != 0;
    };
    for (; ok && walk.get(p, t); walk.next(), ++n_tile) {
      const int buf = n_tile & 1;
      ok = wait(&acc_empty[buf], ((n_tile >> 1) & 1) ^ 1u);
      if (!ok) break;
      const int n = __shfl_sync(0xffffffffu, t.n, 0), t0 = __shfl_sync(0xffffffffu, t.t0, 0);
      const int w0 = __shfl_sync(0xffffffffu, t.w0, 0);
      const uint32_t d = tmem + buf * kTileTokens;
      const uint32_t idesc = fp4_idesc<FMT>(n);
      const int shift = w0 & (kSfRows - 1);              // lane of the tile's first weight row
      const uint32_t x_col = (t0 & 64) ? 2u : 0u;        // scale column of the tile's first token
      const int x_sf = ceil_div(t0 + n, kSfRows) - t0 / kSfRows;
      const uint64_t wd0 = umma_desc_sw128(smem_u32(smem + p.w_off) - shift * 128);
      const uint64_t xd0 = umma_desc_sw128(smem_u32(smem + p.x_off));
      const uint64_t sfd0 = scales_desc(smem_u32(smem + p.sf_off));
      int kb_left = p.k_blocks, steps_left = ceil_div(p.K, 64);
      for (int ks = 0; ks < k_stages; ++ks) {
        ok = wait(&full[s], phase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sf = tmem + kSfCol + (it & 1) * kSfCols;
        const uint64_t wd = wd0 + s * w_stage, xd = xd0 + s * x_stage, sfd = sfd0 + s * sf_stage;
        if (issuer) {
          if (x_sf == 1)
            issue_stage<FMT, 1>(d, idesc, wd, xd, sf, sfd, x_col, kb_left, steps_left, ks == 0);
          else
            issue_stage<FMT, 2>(d, idesc, wd, xd, sf, sfd, x_col, kb_left, steps_left, ks == 0);
          umma_commit(&empty[s]);
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
      if (ok && issuer) umma_commit(&acc_full[buf]);
    }
    if (!ok && issuer) {
      umma_commit(&mma_done);
      mbar_wait_drain(&mma_done, 0, 100000000ull);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue --
    // Two halves of four warps (one per lane quarter) take alternate runs of
    // 32 tokens.
    const int ew = warp - kWarpEpi0, half = ew >> 2;
    const int quarter = warp & 3;                  // the TMEM lanes this warp may read
    const int bar = 1 + half;
    const int htid = (ew & 3) * 32 + lane;         // thread within the half
    float *ex = reinterpret_cast<float *>(smem + p.ex_off + half * kXBytes);
    TileWalk walk(table, p);
    Tile t;
    int n_tile = 0;
    for (; walk.get(p, t); walk.next(), ++n_tile) {
      const int buf = n_tile & 1;
      bool ok = mbar_wait(&acc_full[buf], (n_tile >> 1) & 1, abort_flag, p.timeout_ns, err);
      ok = SWIGLU ? bar_and_half(bar, ok) : __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * kTileTokens + (static_cast<uint32_t>(quarter) << 21);
      const float alpha = p.x_scale * (p.w_scale ? __ldg(p.w_scale + t.e) : 1.0f);
      const int lane0 = t.w0 & (kSfRows - 1);      // the tile's lanes: [lane0, lane0 + rt)
      const int row_in_block = quarter * 32 + lane;
      const bool mine = row_in_block >= lane0 && row_in_block < lane0 + p.rt;
      const bool warp_mine = quarter * 32 < lane0 + p.rt && quarter * 32 + 32 > lane0;
      for (int c0 = half * 32; c0 < t.valid; c0 += 64) {
        uint32_t r[2][16];
        if (warp_mine) {
          tmem_ld16(acc + c0, r[0]);
          tmem_ld16(acc + c0 + 16, r[1]);
          tmem_ld_wait();
        }
        if constexpr (!SWIGLU) {
          const int64_t n = (t.w0 & ~(kSfRows - 1)) + row_in_block;
          if (mine && n < p.N) {
            uint16_t *out = static_cast<uint16_t *>(p.out) + static_cast<int64_t>(t.off + t.t0 + c0) * p.N + n;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (c0 + c < t.valid) out[static_cast<int64_t>(c) * p.N] = A::store(__uint_as_float(r[c >> 4][c & 15]) * alpha);
          }
        } else {
          if (warp_mine) {
            // lanes 0-15 hold gate rows, 16-31 the same features' up rows: a
            // swap across the half warps gives the lower half the even
            // tokens' pairs and the upper half the odd tokens'
            const bool upper = lane >= 16;
            float *dst = ex + (lane >> 4) * kXPitch + quarter * 16 + (lane & 15);
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float a = __uint_as_float(r[c >> 4][c & 15]) * alpha;
              const float b = __uint_as_float(r[c >> 4][(c & 15) + 1]) * alpha;
              const float other = __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
              const float g = upper ? other : a, u = upper ? b : other;
              dst[c * kXPitch] = g * sigmoid_fast(g) * u;
            }
          }
          bar_sync_half(bar);
          // one token's 16 features per thread: the four loads go in an order
          // that keeps the eight threads of a phase on different banks
          const int tok = htid >> 2, fq = htid & 3;
          const int f0 = (t.w0 & ~(kSfRows - 1)) / 2 + fq * 16;      // first feature
          const int I = p.N / 2;
          const bool in_tile = fq * 32 >= lane0 && fq * 32 < lane0 + p.rt;
          const bool have = in_tile && c0 + tok < t.valid;
          const float4 *src = reinterpret_cast<const float4 *>(ex + tok * kXPitch + fq * 16);
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
          const int tl = t.t0 + c0 + tok;       // token within the group
          if (have) {
            const int64_t blk = (p.offsets ? ragged_row_block(t.off, t.e) : 0) + tl / kSfRows;
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
              *reinterpret_cast<uint64_t *>(p.h_codes + static_cast<int64_t>(t.off + tl) * (I / 2) + f0 / 2) = codes;
            }
          }
          bar_sync_half(bar);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
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

constexpr int kSmemLimit = 227 * 1024 - 1024;   // less the static part

int align_up(int v, int a) { return (v + a - 1) / a * a; }

template <class A, int FMT, bool SWIGLU>
cudaError_t launch_gemm(const Fp4GemmArgs &a, GemmParams p, int num_sms, cudaStream_t stream, bool dependent) {
  constexpr int kSfPerStage = kStageK / Fp4<FMT>::kSfK;
  auto *kernel = fp4_gemm_kernel<A, FMT, SWIGLU>;
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
  // group table; around the weight stages at least the 128 - rt rows that an
  // MMA reads beyond a short tile
  const int slack = (kSfRows - p.rt) * 128;
  const int ex = SWIGLU ? 2 * kXBytes : 0;
  const int table = align_up(2 * (p.groups + 1) * 4, 16);
  const int x_stage = p.x_rows * 128, w_stage = p.rt * 128, sf_stage = kSfPerStage * kSfBytes * (1 + p.x_sf);
  const int fixed = 1024 + 2 * slack + ex + table;
  int S = (kSmemLimit - fixed) / (x_stage + w_stage + sf_stage);
  if (S > kMaxStages) S = kMaxStages;
  if (S < 2) return cudaErrorInvalidValue;
  p.stages = S;
  p.x_off = 0;
  p.w_off = align_up(S * x_stage < slack ? slack : S * x_stage, 1024);
  p.sf_off = p.w_off + S * w_stage;
  p.ex_off = align_up(p.sf_off + S * sf_stage, 128);
  p.table_off = p.ex_off + ex;
  int bytes = p.table_off + table;
  if (bytes < p.sf_off + slack) bytes = p.sf_off + slack;
  bytes += 1024;   // base alignment
  if (bytes > kSmemLimit) return cudaErrorInvalidValue;

  CUtensorMap tm_w, tm_x, tm_xb;
  if (!encode_codes(&tm_w, a.w_codes, static_cast<int64_t>(p.groups) * p.N, p.K, p.rt) ||
      !encode_codes(&tm_x, a.x_codes, p.rows, p.K, p.x_rows))
    return cudaErrorInvalidValue;
  tm_xb = tm_x;
  if (p.x_box != p.x_rows && !encode_codes(&tm_xb, a.x_codes, p.rows, p.K, p.x_box)) return cudaErrorInvalidValue;
  // no more CTAs than tiles can exist
  const int64_t token_tiles_max = static_cast<int64_t>(p.rows) / p.bt + (p.groups < p.rows ? p.groups : p.rows);
  const int64_t most = token_tiles_max * p.n_tiles;
  const int grid = static_cast<int>(most < num_sms ? most : num_sms);
  return launch_on(kernel, dim3(static_cast<unsigned>(grid)), kThreads, static_cast<size_t>(bytes), stream, dependent,
                   p, tm_w, tm_x, tm_xb);
}

}  // namespace

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
  p.x_box = p.bt < 64 ? p.bt : 64;
  p.x_rows = align_up(p.bt, p.x_box);
  p.x_sf = p.max_group > 128 ? 2 : 1;
  p.out = a.out;
  p.h_codes = a.h_codes;
  p.h_scales = a.h_scales;
  p.h_k_blocks = a.swiglu ? static_cast<int>(fp4_k_blocks(a.N / 2, a.fmt)) : 0;
  p.hq = make_fp4_scale(a.h_scale);
  p.timeout_ns = timeout_ns;

  // Rows of a weight tile: the fewest rounds of the SMs, counted in rows plus a
  // fixed cost per tile, over the most (group, token tile) pairs there can be.
  const int64_t pairs = static_cast<int64_t>(p.rows) / p.bt + (p.groups < p.rows ? p.groups : p.rows);
  const int least = !a.swiglu ? 16 : a.fmt == FP4_MX ? 64 : 32;   // a hidden block's features within one tile
  int64_t best = -1;
  p.rt = kSfRows;
  for (int rt = kSfRows; rt >= least; rt /= 2) {
    const int64_t rounds = (pairs * ceil_div(p.N, rt) + num_sms - 1) / num_sms;
    const int64_t cost = rounds * (rt + 16);
    if (best < 0 || cost < best) {
      best = cost;
      p.rt = rt;
    }
  }
  p.n_tiles = ceil_div(p.N, p.rt);

  if (a.swiglu)
    return a.fmt == FP4_MX ? launch_gemm<ActBf16, FP4_MX, true>(a, p, num_sms, stream, dependent)
                           : launch_gemm<ActBf16, FP4_NV, true>(a, p, num_sms, stream, dependent);
  if (a.act == ActF16::kId)
    return a.fmt == FP4_MX ? launch_gemm<ActF16, FP4_MX, false>(a, p, num_sms, stream, dependent)
                           : launch_gemm<ActF16, FP4_NV, false>(a, p, num_sms, stream, dependent);
  return a.fmt == FP4_MX ? launch_gemm<ActBf16, FP4_MX, false>(a, p, num_sms, stream, dependent)
                         : launch_gemm<ActBf16, FP4_NV, false>(a, p, num_sms, stream, dependent);
}

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
