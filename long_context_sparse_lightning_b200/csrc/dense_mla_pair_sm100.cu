// Dense latent attention in the absorbed form for many query rows: a CTA pair
// per item of 128 rows (heads of a token, or of several), tcgen05 cta_group::2.
//
//     S [128 x 64]   = Q [128 x 576] . C^T            (M = 128, N = 64,  K = 576)
//     O [128 x 512] += P [128 x 64] . C[:, 0:512]     (M = 128, N = 256 twice, K = 64)
//
// Each CTA holds 64 of the rows (all of Q, P and its half of the accumulators),
// so softmax needs no exchange, and half of every B operand, which the tensor
// cores of both read: for S the keys [32 r, 32 r + 32) of a tile with all 576
// dims, for O the dims [256 r, 256 r + 256) with all 64 keys.  An M = 128 product of a
// pair runs at the full rate (measured: 65 cycles for N = 256, K = 16; one CTA with 64
// rows gets half of that), where the transposed form of the one-CTA kernel
// pays 34 + 48 cycles for the same work (64 x 16K-32K at 128 heads 771 -> 430 us).
//
// A tile of 64 keys takes ~1600 cycles where the cache is in L2.  Its MMAs take 1456 by their
// measured rates (36 x 26 + 8 x 65); their operands (Q is read again for every tile) and the
// tile's arrival are ~212 KB of shared-memory traffic, ~1660 cycles at 128 bytes each.  64 x 16K-32K at
// 128 heads: 409 us cold (4.5 TB/s, 1.07 PFLOP/s), ~500 under the power limit (~1.3 GHz).
//
// A descriptor of a pair names one offset for both CTAs, which ties the two
// uses of a tile together: block d of a tile's stage holds this CTA's own keys
// at dims [64 d, 64 d + 64) while S reads it.  Then the four blocks of the other
// CTA's dims are no longer needed, and the keys of the other CTA at this CTA's own
// dims are loaded over them: blocks 0-3 become the keys 0-31 and blocks 4-7 the keys
// 32-63, each CTA's own dims, at the same offsets in both.  A tile costs 9 + 4
// blocks of 4 KB per CTA and four tiles fit beside Q (with the second four in
// blocks of their own it would be three, and a wait between S and O is
// covered by the next tile's S anyway).
//
// Tensor memory of one CTA (M = 128 over a pair: lanes 0-63 hold the rows'
// first N / 2 columns, lanes 64-127 the others): O at [0, 256), three score
// buffers of 32 columns behind it (S runs two tiles ahead of O).
//
// Roles per CTA: warp 0 items and TMA of the keys, warp 1 MMAs (rank 0), warp 2
// TMA of the second half, warps 4-7 and 8-11 softmax of every other tile and epilogue
// (thread = one row's 32 keys of a tile, or 128 of its output dims).  Row references as in the one-CTA kernel.
#include <atomic>

#include "dense_mla.cuh"

namespace dsa {
namespace {

using namespace dense;

constexpr int kN = 128;                   // rows per item
constexpr int kThreads = 384;
constexpr int kSoftThreads = 256;         // two softmax warpgroups
constexpr int kBlk = 32 * 128;            // [32 keys x 64 dims]
constexpr int kStage = 9 * kBlk;
constexpr int kStages = 4;
constexpr int kQBlk = 64 * 128;           // [64 rows x 64 dims]
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 256;            // + 32 * buffer

constexpr int OFF_Q = 0;
constexpr int kSBufs = 3;
constexpr int kPBlk = 64 * 64;            // [64 rows x 32 keys] bf16, 64-byte swizzle
constexpr int kPrefetch = 4;              // tiles that L2 is asked for ahead of the load

constexpr int OFF_P = 9 * kQBlk;          // 2 x the first half of P; the second lies in the stage's block 8
constexpr int OFF_KV = OFF_P + 2 * kPBlk;
constexpr int OFF_AUX = OFF_KV + kStages * kStage;
constexpr int kSmem = OFF_AUX + 2048 + 1024;
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(OFF_KV % 1024 == 0 && kStage % 1024 == 0, "swizzle atoms");

struct Aux {
  uint64_t q_full, q_free;
  uint64_t full[kStages], empty[kStages];   // keys landed in both CTAs (rank 0's) / tile done (both)
  uint64_t rows_set[kStages];               // this stage's cache row is known (for warp 2)
  uint64_t v_full[kStages];                 // the other CTA's keys landed here
  uint64_t s_full[kSBufs], s_free[kSBufs];
  uint64_t p_full[2];
  uint64_t ref_set[2];                      // tile parity: the rows' references with the tile are known
  uint64_t o_full, o_free;
  uint64_t item_full[2], item_free[2];
  uint64_t drain;
  Item item[2];
  int32_t row[kStages];                     // cache row of the tile's position 0, -1: a page outside the pool
  uint32_t tmem;
  union {
    ShareScratch share;
    float mx[2][2][64];                     // per warpgroup and half of a tile's keys: row maxima / row sums
  };
  float ref[64];                            // the rows' references
  int32_t lost[2];                          // by turns of the items with tiles: number (from 1) of one that hidden
                                            // values were cleaned out of
};
static_assert(sizeof(Aux) <= 2048, "");

// Four neighbouring lanes hold four pieces of 8 words each: piece q of lane j goes to
// lane q as its piece j.
__device__ __forceinline__ void exchange_4(uint32_t (&v)[32], uint32_t lane) {
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q & bit) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t &lo = v[8 * q + e], &hi = v[8 * (q | bit) + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
        if (up) {
          lo = got;
        } else {
          hi = got;
        }
      }
    }
  }
}

// Keys that some row must not see: 0 x a non-finite value would reach that row, so
// such values become 0 in the tile.  A row that does see the key has its NaN from
// the score, or where that is -inf from the epilogue: *lost is set to `tag` in both CTAs, whose
// rows take this CTA's dims.  By the 128 threads of a warpgroup; not inlined: its code between a
// tile's softmax and the next costs the tiles that have no border (16K samples prefix 253 us, so 245).
__device__ __noinline__ void clean_values(uint8_t* stage, int pos0, int lo, int min_lim, int last, int32_t* lost, int tag,
                                          int st) {
  bool seen = false;
#pragma unroll 1
  for (int u0 = st; u0 < 8 * kBlk / 16; u0 += 8 * 128) {      // (four loads' latency at once)
    uint4* w = reinterpret_cast<uint4*>(stage) + u0;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int pos = pos0 + 32 * (u0 >> 10) + ((u0 >> 3) & 15) + 16 * g;
      if (pos >= lo && pos <= min_lim) continue;
      uint4 a[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) a[q] = w[256 * q + 128 * g];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (any_not_finite(a[q])) {
          w[256 * q + 128 * g] = finite_or_zero(a[q]);
          seen |= pos >= lo && pos <= last;
        }
    }
  }
  if (seen) {
    const uint32_t at = smem_u32(lost);
    for (uint32_t r = 0; r < 2; ++r)
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(mapa_shared(at, r)), "r"(tag) : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    dense_pair_kernel(const DenseMlaParams p, const __grid_constant__ DenseMaps maps) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Aux* ax = reinterpret_cast<Aux*>(sm + OFF_AUX);
  const uint32_t rank = cluster_ctarank();
  const int unit = static_cast<int>(blockIdx.x >> 1), n_units = static_cast<int>(gridDim.x >> 1);
  const uint32_t warp = warp_id(), lane = lane_id();
  const int tid = threadIdx.x;
  const int H = p.n_heads;
  const RawEntry first = read_entry(p, tid);      // in flight during the set-up

  if (tid == 0) {
    mbar_init(&ax->q_full, 1);
    mbar_init(&ax->q_free, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ax->full[i], 1);
      mbar_init(&ax->empty[i], 1);
      mbar_init(&ax->rows_set[i], 1);
      mbar_init(&ax->v_full[i], 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(&ax->s_full[i], 1);
      mbar_init(&ax->s_free[i], 8);                    // a softmax warpgroup of both CTAs
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ax->p_full[i], 8);
      mbar_init(&ax->item_full[i], 1);
      mbar_init(&ax->ref_set[i], 4);
      mbar_init(&ax->item_free[i], rank == 0 ? 10 : 9); // softmax warps, warp 2, rank 0's MMA thread
    }
    mbar_init(&ax->drain, 1);
    mbar_init(&ax->o_full, 1);
    mbar_init(&ax->o_free, 16);
    ax->lost[0] = ax->lost[1] = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.c);
    prefetch_tmap(&maps.v);
  }
  if (warp == 1) tmem_alloc_pair(&ax->tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Share share = find_share<kN, kThreads>(p, ax->share, first, unit, n_units);
  cluster_sync();                                      // the other CTA's barriers exist
  const uint32_t tmem = ax->tmem;

  if (warp == 0) {
    // ------------------------------------------- items, rows and keys by TMA --
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity, uint32_t site) {
      if (ok && !mbar_wait(b, parity, p.budget)) {
        if (lane == 0) report_error(p.err, kDevErrTimeout, site, blockIdx.x);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
    };
    int k = 0, n_q = 0, t = 0;
    auto publish = [&](const Item& it) {
      if (k >= 2) wait(&ax->item_free[k & 1], ((k >> 1) + 1) & 1, 550);
      if (ok && lane == 0) {
        ax->item[k & 1] = it;
        mbar_arrive(&ax->item_full[k & 1]);
      }
      __syncwarp();
      ++k;
    };
    const uint32_t q_full = mapa_shared(smem_u32(&ax->q_full), 0);
    Walk<kN> walk(p, share, unit);
    Item it;
    while (ok && walk.next(it)) {
      const int64_t kstart = walk.e.kstart;
      // Cache rows of 32 tiles, one per lane (a tile lies in one page), and of the 32 after them.
      auto tile_row = [&](int i) -> int {
        if (i >= it.n_tiles) return -1;
        const int64_t r = cache_row(p.pt, walk.e.b, kstart, (it.tile0 + i) * kTile);
        if (r < 0 && rank == 0) report_error(p.err, kDevErrBounds, 504, walk.e.b);
        return r < 0 ? -1 : static_cast<int>(r);
      };
      publish(it);
      if (!ok || it.n_tiles == 0) continue;
      int my_row = tile_row(static_cast<int>(lane)), my_next = tile_row(32 + static_cast<int>(lane));
      if (n_q > 0) wait(&ax->q_free, (n_q - 1) & 1, 551);
      if (!ok) break;
      ++n_q;
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(&ax->q_full, 2 * 9 * kQBlk);
        tma_load_3d_pair(sm + OFF_Q, &maps.q, q_full, 0, it.row0 + 64 * static_cast<int>(rank), 0);
      }
      __syncwarp();
      for (int i = 0; ok && i < it.n_tiles; ++i, ++t) {
        if (i > 0 && (i & 31) == 0) {
          my_row = my_next;
          my_next = tile_row(i + 32 + static_cast<int>(lane));
        }
        const int row = __shfl_sync(0xffffffffu, my_row, i & 31);
        const int ahead_a = __shfl_sync(0xffffffffu, my_row, (i + kPrefetch) & 31);
        const int ahead_b = __shfl_sync(0xffffffffu, my_next, (i + kPrefetch) & 31);
        const int s = t % kStages;
        if (t >= kStages) wait(&ax->empty[s], ((t / kStages) + 1) & 1, 552);
        if (!ok) break;
        if (lane == 0) {
          ax->row[s] = row;
          mbar_arrive(&ax->rows_set[s]);
          if (rank == 0) mbar_arrive_expect_tx(&ax->full[s], 2 * kStage);
          const uint32_t full = mapa_shared(smem_u32(&ax->full[s]), 0);
          // a tile of a page outside the pool lies behind the cache: zeros arrive, no row is read
          const int y = row < 0 ? static_cast<int>(p.total_keys) : row + 32 * static_cast<int>(rank);
          tma_load_3d_pair(sm + OFF_KV + s * kStage, &maps.c, full, 0, y, 0);
        }
        // this CTA's keys of a later tile: 288 lines of one run of the cache, nine per lane
        const int ahead = (i & 31) + kPrefetch < 32 ? ahead_a : ahead_b;
        const int64_t y1 = static_cast<int64_t>(ahead) + 32 * static_cast<int>(rank);
        if (ahead >= 0 && y1 + 32 <= p.total_keys) {
          const uint8_t* at = reinterpret_cast<const uint8_t*>(p.kv) + y1 * 1152 + lane * 128;
#pragma unroll
          for (int c = 0; c < 9; ++c) asm volatile("prefetch.global.L2 [%0];" ::"l"(at + c * 4096));
        }
        __syncwarp();
      }
    }
    if (ok) {
      Item end;
      end.n_tiles = -1;
      publish(end);
    }
    // All copies land before the blocks end, also those that nothing waits for any more because a
    // wait has run out, here or in another role.  Rank 0's barriers count both CTAs'; what rank 1
    // has issued beyond rank 0 lands within its pause.
    bool landed = rank == 0;
    if (landed && n_q > 0) landed = mbar_wait(&ax->q_full, (n_q - 1) & 1, kDrainCycles);
    for (int i = max(0, t - kStages); landed && i < t; ++i)
      landed = mbar_wait(&ax->full[i % kStages], (i / kStages) & 1, kDrainCycles);
    if (!ok && rank != 0) drain_pause();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs --
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc_s = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 64, 0, 0);     // Q, C K-major
      constexpr uint32_t idesc_o = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 256, 0, 1);    // P K-major, C MN-major
      const uint32_t q_addr = smem_u32(sm + OFF_Q), p_addr = smem_u32(sm + OFF_P), kv_addr = smem_u32(sm + OFF_KV);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity, uint32_t site) {
        if (ok && !mbar_wait(b, parity, p.budget)) {
          report_error(p.err, kDevErrTimeout, site, blockIdx.x);
          ok = false;
        }
        return ok;
      };
      int n_q = 0, t_s = 0, t_o = 0, n_o = 0;
      auto score = [&](bool last) {
        const int s = t_s % kStages, sb = t_s % kSBufs;
        if (t_s >= kSBufs && !wait(&ax->s_free[sb], ((t_s / kSBufs) + 1) & 1, 561)) return;
        if (!wait(&ax->full[s], (t_s / kStages) & 1, 562)) return;
        tc_fence_after();
#pragma unroll
        for (int d = 0; d < 9; ++d)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16_ss_pair(tmem + TM_S + 32 * sb, smem_desc(q_addr + d * kQBlk + kk * 32, 16, 1024, kSwizzle128B),
                             smem_desc(kv_addr + s * kStage + d * kBlk + kk * 32, 16, 1024, kSwizzle128B), idesc_s,
                             (d | kk) ? 1u : 0u);
        umma_commit_pair(&ax->s_full[sb]);
        if (last) umma_commit_pair(&ax->q_free);
        ++t_s;
      };
      for (int k = 0; ok; ++k) {
        if (!wait(&ax->item_full[k & 1], (k >> 1) & 1, 560)) break;
        const int nt = ax->item[k & 1].n_tiles;
        mbar_arrive(&ax->item_free[k & 1]);
        if (nt < 0) break;
        if (nt == 0) continue;
        if (!wait(&ax->q_full, n_q & 1, 563)) break;
        ++n_q;
        // scores run two tiles ahead, so that neither the softmax of a tile nor the
        // load of its second half is waited for while there are scores to compute
        score(nt == 1);
        if (ok && nt > 1) score(nt == 2);
        for (int i = 0; ok && i < nt; ++i) {
          if (i + 2 < nt) score(i + 3 == nt);
          const int s = t_o % kStages;
          if (!ok || !wait(&ax->p_full[t_o & 1], (t_o >> 1) & 1, 564)) break;       // P written, and all keys at each CTA's dims landed
          if (i == 0 && n_o > 0 && !wait(&ax->o_free, (n_o - 1) & 1, 565)) break;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < 2; ++g)
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                umma_f16_ss_pair(tmem + 128 * j,
                                 smem_desc((g == 0 ? p_addr + (t_o & 1) * kPBlk : kv_addr + s * kStage + 8 * kBlk) + kk * 32,
                                           16, 512, kSwizzle64B),
                                 smem_desc(kv_addr + s * kStage + (4 * g + 2 * j) * kBlk + kk * 2048, kBlk, 1024,
                                           kSwizzle128B),
                                 idesc_o, (i | g | kk) ? 1u : 0u);
          umma_commit_pair(&ax->empty[s]);
          ++t_o;
          if (i + 1 == nt) umma_commit_pair(&ax->o_full);
        }
        ++n_o;
      }
      // the MMAs in flight end before their memory goes, whichever role has given up
      umma_commit_pair_here(&ax->drain);
      mbar_wait(&ax->drain, 0, kDrainCycles);
    }
  } else if (warp == 2) {
    // ------------------------- the other CTA's keys at this CTA's dims by TMA --
    bool ok = true;
    int n_own = 0;          // loads issued
    auto wait = [&](uint64_t* b, uint32_t parity, uint32_t site) {
      if (ok && !mbar_wait(b, parity, p.budget)) {
        if (lane == 0) report_error(p.err, kDevErrTimeout, site, blockIdx.x);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
    };
    for (int k = 0; ok; ++k) {
      wait(&ax->item_full[k & 1], (k >> 1) & 1, 570);
      if (!ok) break;
      const Item it = ax->item[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ax->item_free[k & 1]);
      if (it.n_tiles < 0) break;
      const int min_lim = it.prefix ? it.last : it.base + (it.row0 - it.seq_row0) / H;
      for (int i = 0; ok && i < it.n_tiles; ++i, ++n_own) {
        const int s = n_own % kStages, pos0 = (it.tile0 + i) * kTile;
        wait(&ax->rows_set[s], (n_own / kStages) & 1, 571);
        wait(&ax->s_full[n_own % kSBufs], (n_own / kSBufs) & 1, 572);     // S has read the tile
        if (!ok) break;
        if (lane == 0) {
          const int row = ax->row[s], none = static_cast<int>(p.total_keys);
          const bool border = row < 0 || pos0 < it.lo || pos0 + kTile - 1 > min_lim;
          uint8_t* st = sm + OFF_KV + s * kStage;
          // On the border the softmax warps rewrite values (below): there both
          // halves come anew, so that this barrier covers all they touch.
          mbar_arrive_expect_tx(&ax->v_full[s], (border ? 8 : 4) * kBlk);
          for (int g = 0; g < 2; ++g) {
            if (!border && g == static_cast<int>(rank)) continue;
            tma_load_3d(st + 4 * g * kBlk, &maps.v, &ax->v_full[s], 0, row < 0 ? none : row + 32 * g,
                        4 * static_cast<int>(rank));
          }
        }
        __syncwarp();
      }
    }
    bool landed = true;
    for (int i = max(0, n_own - kStages); landed && i < n_own; ++i)
      landed = mbar_wait(&ax->v_full[i % kStages], (i / kStages) & 1, kDrainCycles);
  } else if (warp >= 4) {
    // ---------------------------------------------------- softmax, epilogue --
    // The two warpgroups take turns at the tiles: one alone, a warp per scheduler,
    // shows every latency of its chain (~1800 cycles a tile against ~1400 of MMAs).
    // A row's reference passes from tile to tile through shared memory.
    const int wg = static_cast<int>(warp >> 2) - 1;
    const int qd = static_cast<int>(warp & 3u);
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(qd * 32) << 16);
    const int half = qd >> 1;                                      // keys 32 half .. of a tile, dims 256 half ..
    const int r = (qd & 1) * 32 + static_cast<int>(lane);          // row of this CTA
    const int n = 64 * static_cast<int>(rank) + r;                 // row of the item
    const int st = tid & 127;
    const uint32_t wg_bar = 2 + wg;
    const float NEG_INF = __int_as_float(0xff800000);
    const float scale = p.scale_log2;
    const uint32_t p_row = smem_u32(sm + (half == 0 ? OFF_P : OFF_KV + 8 * kBlk)) + r * 64;
    const uint32_t s_free0 = mapa_shared(smem_u32(&ax->s_free[0]), 0), p_full0 = mapa_shared(smem_u32(&ax->p_full[0]), 0);
    const uint32_t o_free = mapa_shared(smem_u32(&ax->o_free), 0);
    bool ok = true;
    // Once a wait has run out nothing waits any more: the warps go on to the
    // end in step (their barriers keep matching) and the error word tells.
    auto wait = [&](uint64_t* b, uint32_t parity, uint32_t site) {
      if (ok && !mbar_wait(b, parity, p.budget)) {
        report_error(p.err, kDevErrTimeout, site, blockIdx.x);
        ok = false;
      }
      __syncwarp();
    };
    int t0 = 0, n_o = 0;              // tiles before this item, items with tiles
    for (int k = 0;; ++k) {
      wait(&ax->item_full[k & 1], (k >> 1) & 1, 580);
      if (bar_any(!ok, 1, kSoftThreads)) break;       // a warp that gave up must not leave the others at a barrier
      const Item it = ax->item[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ax->item_free[k & 1]);
      if (it.n_tiles < 0) break;
      const int min_lim = it.prefix ? it.last : it.base + (it.row0 - it.seq_row0) / H;
      const int lim = n >= it.rows ? -1 : (it.prefix ? it.last : it.base + (it.row0 + n - it.seq_row0) / H);
      float m = NEG_INF, l = 0.f;     // reference and this thread's share of the row's sum in its units
      for (int i = (t0 ^ wg) & 1; i < it.n_tiles; i += 2) {
        const int t = t0 + i, sb = t % kSBufs, s = t % kStages, pos0 = (it.tile0 + i) * kTile;
        uint32_t x[32];
        wait(&ax->s_full[sb], (t / kSBufs) & 1, 581);
        tc_fence_after();
        tmem_ld32(t_lane + TM_S + 32 * sb, x);
        tmem_ld_wait();
        tc_fence_before();
        wait(&ax->rows_set[s], (t / kStages) & 1, 586);
        const bool skip = ax->row[s] < 0;
        if (lane == 0) mbar_arrive_remote(s_free0 + 8 * sb);
        const bool border = skip || pos0 < it.lo || pos0 + kTile - 1 > min_lim;
        if (border) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int pos = pos0 + 32 * half + j;
            if (skip || pos < it.lo || pos > lim) x[j] = __float_as_uint(NEG_INF);
          }
        }
        float m4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m4[j] = __uint_as_float(x[j]);
#pragma unroll
        for (int j = 4; j < 32; ++j) m4[j & 3] = fmaxf(m4[j & 3], __uint_as_float(x[j]));
        const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * scale;
        float now = NEG_INF;          // the row's reference before this tile
        if (i > 0) {
          wait(&ax->ref_set[(t - 1) & 1], ((t - 1) >> 1) & 1, 587);
          now = ax->ref[r];
        }
        // reference -inf: any finite score grows it, a masked one (NaN here) does not
        const bool grow = bar_any(mx - now > kGrow, wg_bar, 128);
        float f = 1.f;
        if (grow) {
          ax->mx[wg][half][r] = mx;
          bar_sync(wg_bar, 128);
          const float top = fmaxf(ax->mx[wg][0][r], ax->mx[wg][1][r]);
          if (top > now) {
            f = exp2_approx(now - top);
            now = top;
          }
        }
        if ((grow || i == 0) && half == 0) ax->ref[r] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ax->ref_set[t & 1]);
        if (now != m) {
          l *= exp2_approx(m - now);
          m = now;
        }
        if (grow && i > 0) {
          // O is idle once the previous tile's product is done
          wait(&ax->empty[(t - 1) % kStages], ((t - 1) / kStages) & 1, 582);
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 256; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_lane + c, o);
            tmem_ld_wait();
            uint32_t a[16], b[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              a[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              b[j] = __float_as_uint(__uint_as_float(o[16 + j]) * f);
            }
            tmem_st16(t_lane + c, a);
            tmem_st16(t_lane + c + 16, b);
          }
          tmem_st_wait();
          tc_fence_before();
        }
        const float ref = m == NEG_INF ? 0.f : -m;
        uint32_t pk[16];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float a = exp2_approx(fmaf(__uint_as_float(x[2 * j]), scale, ref));
          const float b = exp2_approx(fmaf(__uint_as_float(x[2 * j + 1]), scale, ref));
          sum += a + b;
          pk[j] = pack_bf16(a, b);
        }
        l += sum;
        // the first half's buffer is read by the product before last until that is
        // done; the second half takes the place of the tile's RoPE dims, which S has read
        if (t > 1) wait(&ax->empty[(t - 2) % kStages], ((t - 2) / kStages) & 1, 583);
        const uint32_t p_at = p_row + (half == 0 ? (t & 1) * kPBlk : s * kStage);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p_at + ((u ^ ((r >> 1) & 3)) << 4)),
                       "r"(pk[4 * u]), "r"(pk[4 * u + 1]), "r"(pk[4 * u + 2]), "r"(pk[4 * u + 3])
                       : "memory");
        wait(&ax->v_full[s], (t / kStages) & 1, 584);
        if (border) clean_values(sm + OFF_KV + s * kStage, pos0, it.lo, min_lim, it.last, &ax->lost[n_o & 1], n_o + 1, st);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(p_full0 + 8 * (t & 1));
      }
      t0 += it.n_tiles;

      // ---- the row's sum over both halves of the keys and both warpgroups ----
      float last = NEG_INF;
      if (it.n_tiles > 0) {
        wait(&ax->ref_set[(t0 - 1) & 1], ((t0 - 1) >> 1) & 1, 588);
        last = ax->ref[r];
        if (last != m) l *= exp2_approx(m - last);
      }
      bar_sync(wg_bar, 128);          // the last tile's maxima have been read
      ax->mx[wg][half][r] = l;
      bar_sync(1, kSoftThreads);
      const float sum = (ax->mx[0][0][r] + ax->mx[0][1][r]) + (ax->mx[1][0][r] + ax->mx[1][1][r]);
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      if (wg == 0 && half == 0 && n < it.rows) store_lse(p, it, kN, n, sum == 0.f ? NEG_INF : last + log2f(sum));
      if (it.n_tiles > 0) {
        wait(&ax->o_full, n_o & 1, 585);
        ++n_o;
        tc_fence_after();
      }
      // read before o_free, which the next item's products wait for, and so the one after it, whose flag this will be
      const bool lost = it.n_tiles > 0 && *static_cast<volatile int32_t*>(&ax->lost[(n_o - 1) & 1]) == n_o;
      float* dst32 = fp32_rows(p, it, kN);
      // 64 dims at a time.  A thread has a row's, which would go out as 32 rows' sectors an
      // instruction; four lanes exchange theirs first, so that each row gets whole lines (16K
      // samples prefix 249 -> 245 us; the piece of one short item still takes ~5700 cycles, 128
      // KB out of one SM).
      const int row4 = n & ~3;                 // the first of the four lanes' rows
      const int piece = 8 * static_cast<int>(lane & 3u);
#pragma unroll 1
      for (int c = 128 * wg; c < 128 * wg + 128; c += 64) {
        uint32_t o[2][32];
        if (it.n_tiles > 0) {
          tmem_ld32(t_lane + c, o[0]);
          tmem_ld32(t_lane + c + 32, o[1]);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int j = 0; j < 64; ++j) o[j >> 5][j & 31] = 0u;
        }
        const int d = 256 * half + c;
        if (dst32 != nullptr) {
          if (it.n_tiles > 0) {                // an empty piece has lse = -inf, its output is not read
#pragma unroll
            for (int g = 0; g < 2; ++g) {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[g][j] = __float_as_uint(__uint_as_float(o[g][j]) * inv);
              exchange_4(o[g], lane);
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (row4 + q < it.rows)
                  store_32(dst32 + static_cast<int64_t>(row4 + q) * 512 + d + 32 * g + piece, &o[g][8 * q]);
            }
          }
        } else {
          uint32_t v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j)
            v[j] = pack_bf16(__uint_as_float(o[j >> 4][2 * (j & 15)]) * inv, __uint_as_float(o[j >> 4][2 * (j & 15) + 1]) * inv);
          exchange_4(v, lane);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (row4 + q < it.rows)
              store_32(p.out + static_cast<int64_t>(it.row0 + row4 + q) * 512 + d + 2 * piece, &v[8 * q]);
        }
        __syncwarp();
      }
      if (it.n_tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !(unit == 0 && n_o - 1 == p.skip_arrival)) mbar_arrive_remote(o_free);
      }
      // the outputs are written, mx and ref may be rewritten
      if (bar_any(lost, 1, kSoftThreads)) {
        // this CTA's rows of the item, of all dims
        const int r0 = 64 * static_cast<int>(rank);
        write_nan(p.pt, p.kv, it.b, it.kstart, hidden(it, min_lim), min(it.rows - r0, 64), it.base,
                  it.row0 + r0 - it.seq_row0, H, dst32 == nullptr ? nullptr : dst32 + r0 * 512,
                  p.out + static_cast<int64_t>(it.row0 + r0) * 512, tid - 128, kSoftThreads);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                     // the other CTA no longer touches this one's memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// CTA pairs that can be resident at once (cached per device): every pair takes an
// equal share, so one that waited for a free slot would double the time.
int resident_pairs() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  const int v = cache[dev].load(std::memory_order_relaxed);
  if (v != 0) return v - 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(kSmem);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, dense_pair_kernel, &cfg) != cudaSuccess) n = 0;
  cudaGetLastError();   // a refused query leaves no sticky error behind
  cache[dev].store(n + 1, std::memory_order_relaxed);
  return n;
}

}  // namespace

cudaError_t launch_dense_pair(const DenseMlaParams& p, const DenseMaps& maps, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(dense_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  int pairs = resident_pairs();
  if (pairs < 1) pairs = sm_count() / 2;
  if (pairs < 1 || pairs > kDenseMaxCtas / 2) pairs = kDenseMaxCtas / 2;
  if (pairs < p.gang) return cudaErrorInvalidConfiguration;
  pairs = pairs / p.gang * p.gang;
  dense_pair_kernel<<<2 * pairs, kThreads, kSmem, stream>>>(p, maps);
  return cudaGetLastError();
}

}  // namespace dsa
