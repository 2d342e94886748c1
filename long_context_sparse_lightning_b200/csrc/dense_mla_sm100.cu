// Dense latent attention in the absorbed form on sm_100a, and the same for a
// batch that shares a prefix.
//
//     o[h] = sum_{s <= t} softmax_s(sm_scale * q[h] . c[s]) * c[s][0:512]
//
// over the 576-d latent rows c of every position up to the token's own (MQA
// mode: all heads of a token attend the same rows).
//
// This kernel: items of up to N = 16 or 32 query rows, one CTA each (a rank's heads
// in decode); dense_mla_pair_sm100.cu has the one for more rows, dense_mla.cuh what
// both share.  Both products are computed transposed.  An item is a few query rows
// (heads of one token, or of a few tokens of one sequence) and a range of 64-key
// tiles; per tile
//     S^T [64 keys x N]  = C [64 x 576] . Q^T        (M = 64,  K = 576)
//     O^T [512 x N]     += C[:, 0:512]^T . P^T        (4 x M = 128, K = 64)
// so that the cache tile, as it lands by TMA, is the M-side operand of both
// (K-major, then MN-major) and the few query rows are the N side: with the rows on
// the M side a 16-head rank would pay for 128 rows of tensor work, and their 512
// output dims would fill tensor memory.
//
// A CTA reads 72 KB per tile.  At the measured copy bandwidth (6.46 TB/s) an SM
// gets that in ~3100 cycles; the tensor work of a tile is ~1600 (36 x 27 and 16 x 39
// cycles measured, N = 16), so decode is bound by the cache read: 64 sequences of
// 1K-32K positions at 16 heads 236 us, 5.4 TB/s, 83 % of the copy rate.
//
// Work split: the (sequence, row tiles) items of a launch are laid end to end
// by their tile counts (plus a constant for an item's prologue and epilogue), and
// every group of W CTAs takes an equal share of that line; the W CTAs of a group
// take neighbouring row tiles over the same keys, so that the rows a second CTA
// needs are in L2.  W is one number for the launch, from the average rows of a sequence: where
// sequences differ in their numbers of tokens, members of a group without a row tile of the shorter
// ones idle over those (see dense_plan).  An item cut by a share's border leaves normalised partial
// outputs and log-sum-exps, at most two per CTA, which dense_merge_kernel joins.
// Lengths are read on the device: uneven contexts balance without host knowledge.
//
// Roles: warp 0 walks the items and issues TMA; warp 1 issues the MMAs; warps
// 2-5 do softmax and epilogue.  Scores are read with the .16x256b shape (a thread holds
// 2 keys x N/4 rows), so row maxima are needed across lanes: instead of a
// running maximum per tile, a reference per row is taken from the first tile that
// shows the row a key and kept while no score exceeds it by 2^24 (fp32 sums and
// bf16 probabilities keep their relative precision over that range); one
// barrier with an OR per tile decides.  Probabilities are rounded to bf16 for the
// second product, whose other operand is the bf16 cache tile itself; row sums
// are taken in fp32 before that rounding.
#include "dense_mla.cuh"

namespace dsa {
namespace {

using namespace dense;

constexpr int kKeys = kTile;
constexpr int kBlk = kKeys * 128;         // one [64 keys x 64 dims] block, 128-byte swizzle
constexpr int kPair = 2 * kBlk;           // 128 value dims: one M block of the second product
constexpr int kWarps = 6;
constexpr int kThreads = kWarps * 32;
constexpr int kSoftThreads = 128;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 256;            // two score buffers of 64 columns; O^T block m at column m * N

template <int N>
struct Cfg {
  // Scores run one tile ahead of the second product, which holds its tile's four
  // pairs until it is done: eight pair slots at least.
  static constexpr int ROPE_SLOTS = 2;
  static constexpr int PAIR_SLOTS = N == 32 ? 9 : 10;
  static_assert(PAIR_SLOTS >= 8, "two tiles in flight");
  static constexpr int OFF_Q = 0;                                    // 9 blocks of [N rows x 64 dims]
  static constexpr int OFF_P = 9 * N * 128;                          // 2 x [64 keys x 64 rows] bf16
  static constexpr int OFF_ROPE = OFF_P + 2 * kBlk;
  static constexpr int OFF_PAIR = OFF_ROPE + ROPE_SLOTS * kBlk;
  static constexpr int OFF_AUX = OFF_PAIR + PAIR_SLOTS * kPair;
  static constexpr int SMEM = OFF_AUX + 2048 + 1024;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
  static_assert(OFF_P % 1024 == 0, "swizzle atoms");
};

struct Aux {
  uint64_t q_full, q_free;
  uint64_t rope_full[2], rope_empty[2];
  uint64_t pair_full[10], pair_empty[10];
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], p_empty[2];
  uint64_t o_full, o_empty;
  uint64_t item_full[2], item_free[2];
  uint64_t drain;
  Item item[2];
  int32_t skip[10];         // the tile whose first pair has this slot lies on a page outside the pool
  uint32_t tmem;
  union {
    ShareScratch share;
    float mx[4][32];        // per softmax warp: row maxima / row sums
  };
  float fac[32];            // rescaling factors, inverse row sums
  float ref[32];            // the rows' references, at the end of an item
  int32_t lim[32];          // last position each row sees
  int32_t lost;             // hidden values of the item that are not finite were cleaned
};
static_assert(sizeof(Aux) <= 2048, "");

// 16 TMEM lanes x N columns, the layout of tmem_ld_16x256b_x8
__device__ __forceinline__ void ld_scores(uint32_t t, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}
__device__ __forceinline__ void ld_scores(uint32_t t, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(t));
}
// 32 lanes x 16 consecutive columns
__device__ __forceinline__ void ld_cols16(uint32_t t, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}

// Keys that some row must not see: 0 x a non-finite value would reach that row, so
// such values become 0 in the tile (its pairs are slots n, n + 1, n + 2, n + 3 of the ring).
// A row that does see the key has its NaN from the score, or where that is -inf from the
// epilogue (*lost is set).  By 128 threads; not inlined, to stay out of the tiles that have no border.
template <int SLOTS>
__device__ __noinline__ void clean_values(uint8_t* pairs, int n, int pos0, int lo, int min_lim, int last, int32_t* lost,
                                          int st) {
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {                // key st / 8 + 16 g, eight units of it
    const int pos = pos0 + (st >> 3) + 16 * g;
    if (pos >= lo && pos <= min_lim) continue;
    uint4 a[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      a[q] = reinterpret_cast<const uint4*>(pairs + (n + (q >> 1)) % SLOTS * kPair + (q & 1) * kBlk)[st + 128 * g];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (any_not_finite(a[q])) {
        reinterpret_cast<uint4*>(pairs + (n + (q >> 1)) % SLOTS * kPair + (q & 1) * kBlk)[st + 128 * g] =
            finite_or_zero(a[q]);
        if (pos >= lo && pos <= last) *lost = 1;
      }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
    dense_mla_kernel(const DenseMlaParams p, const __grid_constant__ DenseMaps maps) {
  using C = Cfg<N>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Aux* ax = reinterpret_cast<Aux*>(sm + C::OFF_AUX);
  const uint32_t warp = warp_id(), lane = lane_id();
  const int tid = threadIdx.x;
  const int H = p.n_heads;
  const RawEntry first = read_entry(p, tid);      // in flight during the set-up

  if (tid == 0) {
    mbar_init(&ax->q_full, 1);
    mbar_init(&ax->q_free, 1);
    for (int i = 0; i < C::ROPE_SLOTS; ++i) {
      mbar_init(&ax->rope_full[i], 1);
      mbar_init(&ax->rope_empty[i], 1);
    }
    for (int i = 0; i < C::PAIR_SLOTS; ++i) {
      mbar_init(&ax->pair_full[i], 1);
      mbar_init(&ax->pair_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ax->s_full[i], 1);
      mbar_init(&ax->s_empty[i], 4);
      mbar_init(&ax->p_full[i], 4);
      mbar_init(&ax->p_empty[i], 1);
      mbar_init(&ax->item_full[i], 1);
      mbar_init(&ax->item_free[i], 5);      // the MMA thread and the softmax warps
    }
    mbar_init(&ax->drain, 1);
    mbar_init(&ax->o_full, 1);
    mbar_init(&ax->o_empty, 4);
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.c);
    prefetch_tmap(&maps.v);
  }
  if (warp == 1) {
    tmem_alloc(&ax->tmem, kTmemCols);
    tmem_relinquish();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Share share = find_share<N, kThreads>(p, ax->share, first, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
  const uint32_t tmem = ax->tmem;

  if (warp == 0) {
    // --------------------------------------------------- items and TMA loads --
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity, uint32_t site) {
      if (ok && !mbar_wait(b, parity, p.budget)) {
        if (lane == 0) report_error(p.err, kDevErrTimeout, site, blockIdx.x);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
    };
    int k = 0, n_q = 0, n_rope = 0, n_pair = 0;
    auto publish = [&](const Item& it) {
      if (k >= 2) wait(&ax->item_free[k & 1], ((k >> 1) + 1) & 1, 510);
      __syncwarp();      // every lane has its copy of the share, whose memory the softmax warps write from here on
      if (ok && lane == 0) {
        ax->item[k & 1] = it;
        mbar_arrive(&ax->item_full[k & 1]);
      }
      __syncwarp();
      ++k;
    };
    Walk<N> walk(p, share, static_cast<int>(blockIdx.x));
    Item it;
    while (ok && walk.next(it)) {
      // Cache rows of 32 tiles, one per lane (a tile lies in one page), and of the 32 after them.
      auto tile_row = [&](int i) -> int {
        if (i >= it.n_tiles) return -1;
        const int64_t r = cache_row(p.pt, walk.e.b, walk.e.kstart, (it.tile0 + i) * kKeys);
        if (r < 0) report_error(p.err, kDevErrBounds, 504, walk.e.b);
        return r < 0 ? -1 : static_cast<int>(r);
      };
      int my_row = tile_row(static_cast<int>(lane)), my_next = tile_row(32 + static_cast<int>(lane));
      publish(it);
      if (!ok || it.n_tiles == 0) continue;
      if (n_q > 0) wait(&ax->q_free, (n_q - 1) & 1, 511);
      if (!ok) break;
      ++n_q;
      if (lane == 0) {
        mbar_arrive_expect_tx(&ax->q_full, 9 * N * 128);
        tma_load_3d(sm + C::OFF_Q, &maps.q, &ax->q_full, 0, it.row0, 0);
      }
      __syncwarp();
      for (int i = 0; ok && i < it.n_tiles; ++i) {
        if (i > 0 && (i & 31) == 0) {
          my_row = my_next;
          my_next = tile_row(i + 32 + static_cast<int>(lane));
        }
        int row = __shfl_sync(0xffffffffu, my_row, i & 31);
        const int skip = row < 0 ? 1 : 0;
        if (skip) row = static_cast<int>(p.total_keys);      // past the pool: zeros arrive, no row is read
        const int rs = n_rope % C::ROPE_SLOTS;
        if (n_rope >= C::ROPE_SLOTS) wait(&ax->rope_empty[rs], ((n_rope / C::ROPE_SLOTS) + 1) & 1, 512);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&ax->rope_full[rs], kBlk);
          tma_load_3d(sm + C::OFF_ROPE + rs * kBlk, &maps.v, &ax->rope_full[rs], 0, row, 8);
        }
        ++n_rope;
        for (int m = 0; ok && m < 4; ++m) {
          const int ps = n_pair % C::PAIR_SLOTS;
          if (n_pair >= C::PAIR_SLOTS) wait(&ax->pair_empty[ps], ((n_pair / C::PAIR_SLOTS) + 1) & 1, 513);
          if (!ok) break;
          if (lane == 0) {
            uint8_t* dst = sm + C::OFF_PAIR + ps * kPair;
            if (m == 0) ax->skip[ps] = skip;
            mbar_arrive_expect_tx(&ax->pair_full[ps], kPair);
            tma_load_3d(dst, &maps.c, &ax->pair_full[ps], 0, row, 2 * m);
          }
          ++n_pair;
        }
      }
    }
    if (ok) {
      Item end;
      end.n_tiles = -1;
      publish(end);
    }
    // All copies land before the block ends, also those that nothing waits for any more because
    // a wait has run out, here or in another role.
    bool landed = true;
    if (n_q > 0) landed = mbar_wait(&ax->q_full, (n_q - 1) & 1, kDrainCycles);
    for (int i = max(0, n_rope - C::ROPE_SLOTS); landed && i < n_rope; ++i)
      landed = mbar_wait(&ax->rope_full[i % C::ROPE_SLOTS], (i / C::ROPE_SLOTS) & 1, kDrainCycles);
    for (int i = max(0, n_pair - C::PAIR_SLOTS); landed && i < n_pair; ++i)
      landed = mbar_wait(&ax->pair_full[i % C::PAIR_SLOTS], (i / C::PAIR_SLOTS) & 1, kDrainCycles);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMAs --
    if (elect_one()) {
      constexpr uint32_t idesc_s = idesc_f32acc(kFmtBF16, kFmtBF16, 64, N, 0, 0);    // C and Q K-major
      constexpr uint32_t idesc_o = idesc_f32acc(kFmtBF16, kFmtBF16, 128, N, 1, 1);   // C^T and P^T MN-major
      const uint32_t q_addr = smem_u32(sm + C::OFF_Q), p_addr = smem_u32(sm + C::OFF_P);
      const uint32_t rope_addr = smem_u32(sm + C::OFF_ROPE), pair_addr = smem_u32(sm + C::OFF_PAIR);
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity, uint32_t site) {
        if (ok && !mbar_wait(b, parity, p.budget)) {
          report_error(p.err, kDevErrTimeout, site, blockIdx.x);
          ok = false;
        }
        return ok;
      };
      int n_q = 0, t_s = 0, t_o = 0, n_o = 0;      // Q tiles, tiles scored, tiles accumulated, items accumulated
      auto score = [&](bool last) {
        const int rs = t_s % C::ROPE_SLOTS, sb = t_s & 1;
        const uint32_t d = tmem + TM_S + sb * 64;
        if (t_s >= 2 && !wait(&ax->s_empty[sb], ((t_s >> 1) + 1) & 1, 521)) return;
        if (!wait(&ax->rope_full[rs], (t_s / C::ROPE_SLOTS) & 1, 522)) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ss(d, smem_desc(rope_addr + rs * kBlk + kk * 32, 16, 1024, kSwizzle128B),
                      smem_desc(q_addr + 8 * N * 128 + kk * 32, 16, 1024, kSwizzle128B), idesc_s, kk ? 1u : 0u);
        umma_commit(&ax->rope_empty[rs]);
        for (int m = 0; m < 4; ++m) {
          const int n = 4 * t_s + m, ps = n % C::PAIR_SLOTS;
          if (!wait(&ax->pair_full[ps], (n / C::PAIR_SLOTS) & 1, 523)) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_f16_ss(d, smem_desc(pair_addr + ps * kPair + (kk >> 2) * kBlk + (kk & 3) * 32, 16, 1024, kSwizzle128B),
                        smem_desc(q_addr + (2 * m + (kk >> 2)) * N * 128 + (kk & 3) * 32, 16, 1024, kSwizzle128B),
                        idesc_s, 1u);
        }
        umma_commit(&ax->s_full[sb]);
        if (last) umma_commit(&ax->q_free);
        ++t_s;
      };
      for (int k = 0; ok; ++k) {
        if (!wait(&ax->item_full[k & 1], (k >> 1) & 1, 520)) break;
        const int nt = ax->item[k & 1].n_tiles;
        mbar_arrive(&ax->item_free[k & 1]);
        if (nt < 0) break;
        if (nt == 0) continue;
        if (!wait(&ax->q_full, n_q & 1, 524)) break;
        ++n_q;
        score(nt == 1);
        for (int i = 0; ok && i < nt; ++i) {
          if (i + 1 < nt) score(i + 2 == nt);
          const int pb = t_o & 1;
          if (!ok || !wait(&ax->p_full[pb], (t_o >> 1) & 1, 525)) break;
          if (i == 0 && n_o > 0 && !wait(&ax->o_empty, (n_o - 1) & 1, 526)) break;
          tc_fence_after();
          for (int m = 0; m < 4; ++m) {
            const int ps = (4 * t_o + m) % C::PAIR_SLOTS;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ss(tmem + m * N, smem_desc(pair_addr + ps * kPair + kk * 2048, kBlk, 1024, kSwizzle128B),
                          smem_desc(p_addr + pb * kBlk + kk * 2048, kBlk, 1024, kSwizzle128B), idesc_o,
                          (i | kk) ? 1u : 0u);
            umma_commit(&ax->pair_empty[ps]);
          }
          umma_commit(&ax->p_empty[pb]);
          ++t_o;
          if (i + 1 == nt) umma_commit(&ax->o_full);
        }
        ++n_o;
      }
      // the MMAs in flight end before their memory goes, whichever role has given up
      umma_commit(&ax->drain);
      mbar_wait(&ax->drain, 0, kDrainCycles);
    }
  } else {
    // ---------------------------------------------------- softmax, epilogue --
    // Warp of lane quarter qd holds keys 16 qd .. 16 qd + 15 of a tile (an M = 64
    // accumulator occupies the first 16 lanes of each quarter).
    constexpr int KC = N / 8;
    const int qd = static_cast<int>(warp & 3u);
    const uint32_t lane_base = static_cast<uint32_t>(qd * 32) << 16;
    const int key0 = 16 * qd + static_cast<int>(lane >> 2);        // and key0 + 8
    const int col0 = 2 * static_cast<int>(lane & 3u);              // columns 8 kc + col0 + {0, 1}
    const int st = tid - 64;                                       // 0 .. 127
    const float NEG_INF = __int_as_float(0xff800000);
    const float scale = p.scale_log2;
    const uint32_t p_base = smem_u32(sm + C::OFF_P);
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
    int t = 0, n_o = 0;       // tiles and items so far
    for (int k = 0;; ++k) {
      wait(&ax->item_full[k & 1], (k >> 1) & 1, 530);
      // a warp that gave up must not leave the others at a barrier
      if (bar_any(!ok, 1, kSoftThreads)) break;
      const Item it = ax->item[k & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&ax->item_free[k & 1]);
      if (it.n_tiles < 0) break;
      if (st < N)
        ax->lim[st] = st >= it.rows ? -1 : (it.prefix ? it.last : it.base + (it.row0 + st - it.seq_row0) / H);
      if (st == 0) ax->lost = 0;
      bar_sync(1, kSoftThreads);
      const int min_lim = ax->lim[0];       // row 0 is the earliest token's
      float mr[2 * KC], l[2 * KC];
#pragma unroll
      for (int c = 0; c < 2 * KC; ++c) {
        mr[c] = NEG_INF;
        l[c] = 0.f;
      }
      for (int i = 0; i < it.n_tiles; ++i, ++t) {
        const int sb = t & 1, pos0 = (it.tile0 + i) * kKeys;
        uint32_t s[4 * KC];
        wait(&ax->s_full[sb], (t >> 1) & 1, 531);
        tc_fence_after();
        ld_scores(tmem + lane_base + TM_S + sb * 64, s);
        tmem_ld_wait();
        tc_fence_before();
        // the first pair's barrier, long complete, shows what the loading warp has noted for the slot
        wait(&ax->pair_full[4 * t % C::PAIR_SLOTS], (4 * t / C::PAIR_SLOTS) & 1, 534);
        const int skip = ax->skip[4 * t % C::PAIR_SLOTS];   // kept until the slot is refilled, after this tile's product
        __syncwarp();
        if (lane == 0) mbar_arrive(&ax->s_empty[sb]);
        const bool border = skip != 0 || pos0 < it.lo || pos0 + kKeys - 1 > min_lim;
        if (border) {
#pragma unroll
          for (int kc = 0; kc < KC; ++kc)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int pos = pos0 + key0 + (e >> 1) * 8;
              if (skip || pos < it.lo || pos > ax->lim[8 * kc + col0 + (e & 1)]) s[4 * kc + e] = __float_as_uint(NEG_INF);
            }
        }
        bool grow = false;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            // reference -inf: any finite score grows it, a masked one (NaN here) does not
            grow |= fmaf(__uint_as_float(s[4 * kc + e]), scale, -mr[2 * kc + (e & 1)]) > kGrow;
        if (bar_any(grow, 1, kSoftThreads)) {
          // new references: the tile's row maxima where they exceed the old ones
#pragma unroll
          for (int c = 0; c < 2 * KC; ++c) {
            float m = fmaxf(__uint_as_float(s[4 * (c >> 1) + (c & 1)]), __uint_as_float(s[4 * (c >> 1) + 2 + (c & 1)]));
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane < 4) ax->mx[qd][8 * (c >> 1) + col0 + (c & 1)] = m;
          }
          bar_sync(1, kSoftThreads);
#pragma unroll
          for (int c = 0; c < 2 * KC; ++c) {
            const int n = 8 * (c >> 1) + col0 + (c & 1);
            const float m = fmaxf(fmaxf(ax->mx[0][n], ax->mx[1][n]), fmaxf(ax->mx[2][n], ax->mx[3][n])) * scale;
            const float f = m > mr[c] ? exp2_approx(mr[c] - m) : 1.f;
            mr[c] = fmaxf(mr[c], m);
            l[c] *= f;
            if (qd == 0 && (lane >> 2) == 0) ax->fac[n] = f;
          }
          bar_sync(1, kSoftThreads);
          if (i > 0) {
            // O^T is idle once the previous tile's product is done
            wait(&ax->p_empty[(t - 1) & 1], ((t - 1) >> 1) & 1, 532);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4 * N; c += 16) {
              uint32_t o[16];
              ld_cols16(tmem + lane_base + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * ax->fac[(c + j) % N]);
              tmem_st16(tmem + lane_base + c, o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        if (t >= 2) wait(&ax->p_empty[t & 1], ((t >> 1) + 1) & 1, 533);
        const uint32_t pbuf = p_base + (t & 1) * kBlk;
#pragma unroll
        for (int kc = 0; kc < KC; ++kc) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float m = mr[2 * kc + (e & 1)];
            x[e] = exp2_approx(fmaf(__uint_as_float(s[4 * kc + e]), scale, m == NEG_INF ? 0.f : -m));
          }
          l[2 * kc] += x[0] + x[2];
          l[2 * kc + 1] += x[1] + x[3];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int key = key0 + 8 * r;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(pbuf + key * 128 + ((kc ^ (key & 7)) << 4) + col0 * 2),
                         "r"(pack_bf16(x[2 * r], x[2 * r + 1]))
                         : "memory");
          }
        }
        if (border) {
#pragma unroll 1
          for (int m = 0; m < 4; ++m)
            wait(&ax->pair_full[(4 * t + m) % C::PAIR_SLOTS], ((4 * t + m) / C::PAIR_SLOTS) & 1, 534);
          clean_values<C::PAIR_SLOTS>(sm + C::OFF_PAIR, 4 * t, pos0, it.lo, min_lim, it.last, &ax->lost, st);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ax->p_full[t & 1]);
      }

      // ---- row sums over the tile's keys: 8 lanes, then 4 warps ----
#pragma unroll
      for (int c = 0; c < 2 * KC; ++c) {
        float v = l[c];
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane < 4) ax->mx[qd][8 * (c >> 1) + col0 + (c & 1)] = v;
      }
      bar_sync(1, kSoftThreads);
      float row_sum = 0.f;               // threads 0 .. N-1: row st's
      if (st < N) {
        row_sum = (ax->mx[0][st] + ax->mx[1][st]) + (ax->mx[2][st] + ax->mx[3][st]);
        ax->fac[st] = row_sum == 0.f ? 0.f : 1.f / row_sum;
      }
      // the row's reference lies with the threads of its column
      if (qd == 0 && lane < 4) {
#pragma unroll
        for (int c = 0; c < 2 * KC; ++c) ax->ref[8 * (c >> 1) + col0 + (c & 1)] = mr[c];
      }
      bar_sync(1, kSoftThreads);
      if (st < it.rows) store_lse(p, it, N, st, row_sum == 0.f ? NEG_INF : ax->ref[st] + log2f(row_sum));
      if (it.n_tiles > 0) {
        wait(&ax->o_full, n_o & 1, 535);
        ++n_o;
        tc_fence_after();
      }
      const int d0 = qd * 32 + static_cast<int>(lane);
      float* dst32 = fp32_rows(p, it, N);
      // four chunks of 16 columns at a time (the loads' latency once)
#pragma unroll 1
      for (int c0 = 0; c0 < 4 * N; c0 += 64) {
        uint32_t o[4][16];
        if (it.n_tiles > 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) ld_cols16(tmem + lane_base + c0 + 16 * q, o[q]);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 16; ++j) o[q][j] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c = c0 + 16 * q, n0 = c % N, d = (c / N) * 128 + d0;
          if (dst32 != nullptr) {
            if (it.n_tiles > 0) {          // an empty piece has lse = -inf, its output is not read
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (n0 + j < it.rows)
                  dst32[static_cast<int64_t>(n0 + j) * 512 + d] = __uint_as_float(o[q][j]) * ax->fac[n0 + j];
            }
          } else {
            // lane pairs exchange so that each stores two neighbouring dims of one row
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const float a = __uint_as_float(o[q][j]) * ax->fac[n0 + j];
              const float b = __uint_as_float(o[q][j + 1]) * ax->fac[n0 + j + 1];
              const bool odd = (lane & 1u) != 0;
              const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
              const uint32_t w = odd ? pack_bf16(got, b) : pack_bf16(a, got);
              const int n = n0 + j + (odd ? 1 : 0);
              if (n < it.rows)
                *reinterpret_cast<uint32_t*>(p.out + static_cast<int64_t>(it.row0 + n) * 512 + (d & ~1)) = w;
            }
          }
        }
      }
      if (it.n_tiles > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && !(blockIdx.x == 0 && n_o - 1 == p.skip_arrival)) mbar_arrive(&ax->o_empty);
      }
      if (ax->lost != 0) {
        bar_sync(1, kSoftThreads);        // the outputs are written
        write_nan(p.pt, p.kv, it.b, it.kstart, hidden(it, min_lim), it.rows, it.base, it.row0 - it.seq_row0, H, dst32,
                  p.out + static_cast<int64_t>(it.row0) * 512, st, kSoftThreads);
      }
      bar_sync(1, kSoftThreads);          // fac and lim may be rewritten
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// One row's pieces: log-sum-exps and outputs of the partial slots (or the one
// whole result), joined with weights 2^(lse_i - max).
struct RowPieces {
  const float* lse;
  const float* o;
  int64_t lse_step, o_step, lse_first, o_first;    // piece 0 at offset 0, piece i > 0 at first + (i - 1) * step
  int n;
};

__device__ __forceinline__ RowPieces row_pieces(const DenseMlaParams& p, int rec_half, int64_t row, int N, int n_slots) {
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.n_heads;
  const int4 r = p.rec[rec_half * rows + row];
  RowPieces x;
  x.lse_step = x.o_step = x.lse_first = x.o_first = 0;
  x.n = 0;
  if (r.x < 0) {                           // whole (shared prefix) or out of range (no pieces)
    if (p.shared && r.y > 0) {
      x.n = 1;
      x.lse = p.row_lse + rec_half * rows + row;
      x.o = p.row_o + (rec_half * rows + row) * 512;
    }
    return x;
  }
  // pieces: slot r.x, then slot 0 of every following group's member
  const int64_t last = static_cast<int64_t>(r.x >> 1) + static_cast<int64_t>(r.y - 1) * r.w;
  if (r.y < 1 || r.z < 0 || r.z >= N || r.w < 1 || last * 2 + 1 >= n_slots) return x;      // not a record of this launch
  x.n = r.y;
  x.lse = p.part_lse + static_cast<int64_t>(r.x) * N + r.z;
  x.o = p.part_o + (static_cast<int64_t>(r.x) * N + r.z) * 512;
  const int64_t step = 2 * static_cast<int64_t>(r.w);
  x.lse_step = step * N;
  x.o_step = step * N * 512;
  x.lse_first = (step - 1) * N;            // slot 2c + 1 -> slot 2(c + W)
  x.o_first = (step - 1) * N * 512;
  return x;
}

// WARPS warps per row, 4 x 4 dims a lane: one where there are many rows (their
// loads overlap), the whole block where there are few, whose pieces it splits.
template <int WARPS>
__global__ void __launch_bounds__(256) dense_merge_kernel(const DenseMlaParams p, int N, int n_slots) {
  __shared__ float4 part[WARPS > 1 ? WARPS : 1][128];
  __shared__ float part_sum[WARPS];
  const float NEG_INF = __int_as_float(0xff800000);
  const int64_t rows = static_cast<int64_t>(min(max(__ldg(&p.cu_q[p.num_seqs]), 0), p.total_q)) * p.n_heads;
  const int64_t most = static_cast<int64_t>(p.total_q) * p.n_heads;      // records are read before `rows` is known
  const int lane = static_cast<int>(threadIdx.x & 31u), warp = static_cast<int>(threadIdx.x >> 5);
  constexpr int ROWS = 8 / WARPS;
  const int w0 = warp % WARPS;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + warp / WARPS; row < most;
       row += static_cast<int64_t>(gridDim.x) * ROWS) {
    RowPieces a = row_pieces(p, 0, row, N, n_slots), b;
    b.n = 0;
    if (p.shared) {
      b = row_pieces(p, 1, row, N, n_slots);
      if (p.prefix_len == 0 || b.n == 0) a.n = 0;      // b.n = 0: the row's sequence is out of range
    }
    // Pieces: a's and then b's.  A warp's first output is asked for before the log-sum-exps
    // are known, even an empty piece's (not written, any bits); with more of them ahead
    // fewer blocks fit an SM (640 rows: 5.5 us with one, 6.9 with two, 6.5 with none).
    const int n = a.n + b.n;
    auto lse_of = [&](int j) {
      const RowPieces& x = j < a.n ? a : b;
      const int i = j < a.n ? j : j - a.n;
      return x.lse[i == 0 ? 0 : x.lse_first + (i - 1) * x.lse_step];
    };
    float4 v[4];
    auto load = [&](int j) {
      const RowPieces& x = j < a.n ? a : b;
      const int i = j < a.n ? j : j - a.n;
      const float4* o = reinterpret_cast<const float4*>(x.o + (i == 0 ? 0 : x.o_first + (i - 1) * x.o_step)) + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = __ldcg(o + 32 * c);
    };
    if (w0 < n) load(w0);
    const float mine = lane < n ? lse_of(lane) : NEG_INF;
    if (row >= rows) break;                // behind the last sequence
    if (!p.shared && n == 0) continue;     // the main kernel wrote the row
    float m = mine;
    for (int i = 32 + lane; i < n; i += 32) m = fmaxf(m, lse_of(i));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float4 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
    const float ref = m <= kNoWeight ? 0.f : m;
    for (int j = w0; j < n; j += WARPS) {
      if (j != w0) load(j);
      const float z = j < 32 ? __shfl_sync(0xffffffffu, mine, j) : lse_of(j);
      if (z == NEG_INF) continue;
      const float w = exp2f(z - ref);
      sum += w;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        acc[c].x += w * v[c].x;
        acc[c].y += w * v[c].y;
        acc[c].z += w * v[c].z;
        acc[c].w += w * v[c].w;
      }
    }
    if constexpr (WARPS > 1) {
#pragma unroll
      for (int c = 0; c < 4; ++c) part[w0][32 * c + lane] = acc[c];
      if (lane == 0) part_sum[w0] = sum;
      __syncthreads();
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += part_sum[w];
      // four warps store 128 dims each
      if (w0 < 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float4 u = part[w][32 * w0 + lane];
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
          v.w += u.w;
        }
        acc[0] = v;
      }
      __syncthreads();
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int c = 0; c < (WARPS > 1 ? 1 : 4); ++c) {
      uint2 w;
      w.x = pack_bf16(acc[c].x * inv, acc[c].y * inv);
      w.y = pack_bf16(acc[c].z * inv, acc[c].w * inv);
      if (w0 < 4) *reinterpret_cast<uint2*>(p.out + row * 512 + (WARPS > 1 ? w0 : c) * 128 + lane * 4) = w;
    }
    if (w0 == 0 && lane == 0 && p.lse != nullptr) p.lse[row] = sum == 0.f ? NEG_INF : (ref + log2f(sum)) * kLn2;
  }
}

template <int N>
cudaError_t launch(const DenseMlaParams& p, const DenseMaps& maps, int ctas, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(dense_mla_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<N>::SMEM);
  if (e != cudaSuccess) return e;
  dense_mla_kernel<N><<<ctas, kThreads, Cfg<N>::SMEM, stream>>>(p, maps);
  return cudaGetLastError();
}

}  // namespace

DensePlan dense_plan(const dsa_batch_t* b, int n_heads, bool shared) {
  DensePlan d;
  // Rows an item can hold: the rows of one sequence, or with a shared prefix
  // of the whole batch.  More than 32 go to CTA pairs: 64 sequences x 40 heads at 8K 147
  // us against 221 in items of 32, 64 x 4 tokens x 16 heads 152 against 255 (items of 32
  // are up to 2 us faster only where one to eight short sequences do not fill the GPU: 8 x
  // 64 heads at 1000 keys 18.8 against 20.8).
  const int64_t rows = static_cast<int64_t>(shared ? b->total_q : b->max_q_per_seq) * n_heads;
  d.n = rows <= 16 ? 16 : (rows <= 32 ? 32 : 128);
  // Units that share a key range: the row tiles of an average sequence (of total_q rows, padding
  // among them), in equal gangs of at most 16.  Right for equal numbers of tokens; 63 decode tokens at 16K-32K and
  // a prompt of 2048 at 128 heads take 4.4 ms in one call, 0.41 and 0.70 in two (at 16 heads 1.67, 0.33 and 0.11).
  const int64_t tiles = (static_cast<int64_t>(b->total_q) * n_heads + static_cast<int64_t>(b->num_seqs) * d.n - 1) /
                        (static_cast<int64_t>(b->num_seqs) * d.n);
  const int64_t t = tiles < 1 ? 1 : tiles, parts = (t + 15) / 16;
  d.gang = static_cast<int>((t + parts - 1) / parts);
  return d;
}

cudaError_t launch_dense_mla(const DenseMlaParams& p, const DensePlan& d, const DenseMaps& maps, cudaStream_t stream) {
  cudaError_t e;
  if (d.n == 128) {
    e = launch_dense_pair(p, maps, stream);
  } else {
    int ctas = sm_count();
    if (ctas < 1 || ctas > kDenseMaxCtas) ctas = kDenseMaxCtas;
    ctas = ctas / p.gang * p.gang;
    e = d.n == 16 ? launch<16>(p, maps, ctas, stream) : launch<32>(p, maps, ctas, stream);
  }
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.n_heads;
  // A block per row or a warp: 1024 rows 43-46 us either way (64 x 16 and 16 x 64), 2048 rows (64 x 32) 51 with
  // blocks, 47 with warps.
  const bool few = rows <= 8 * 148;
  const int64_t blocks = few ? rows : (rows + 7) / 8;
  const int grid = static_cast<int>(blocks < 148 * 8 ? blocks : 148 * 8);
  if (few) {
    dense_merge_kernel<8><<<grid, 256, 0, stream>>>(p, d.n, dense_slots(d.n));
  } else {
    dense_merge_kernel<1><<<grid, 256, 0, stream>>>(p, d.n, dense_slots(d.n));
  }
  return cudaGetLastError();
}

}  // namespace dsa
