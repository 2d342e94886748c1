// Latent attention in the expanded form on sm_100a: per head h
//     o[i, h] = sum_{s <= t_i} softmax_s(sm_scale * (qn.kn[s, h] + qr.kr[s])) * v[s, h]
// with 128-d keys kn and values v of each head (made from the latent rows by
// the caller's up-projection) and the 64 RoPE dims kr that all heads share:
// 640 multiply-adds per head and pair against the absorbed form's 1088.
//
// A CTA owns two tiles of 128 query rows of one head (lane = row; or, of a
// sequence's few rows, one tile of two heads, whose key tiles then alternate) and walks
// the keys up to its last row's position in tiles of 128.  Tensor memory: the two
// tiles' scores (128 columns each) and outputs (128 each), all 512 columns; a tile's
// probabilities overwrite its scores as bf16 and are the A operand of the
// second product from there.  The MMA thread alternates: while the softmax
// warps of one tile work on its scores, the tensor cores run the other tile's
// second product and next scores.
//
// Per key tile the tensor cores need 2 x 128 x 128 x (192 + 128) multiply-adds
// (2560 cycles at full rate) and the 2 x 128 x 128 exponentials take 2048 at
// 16 per cycle, so both units have to be kept busy at once.  Measured: ~3360 cycles
// a key tile (the products take 1580 a row tile: S reads 128 B/clk of shared
// memory beside the arriving tiles; handing the probabilities over in two halves
// changed nothing).  8K at 16 heads 269 us (1.28 PFLOP/s of useful work, 78 % of the burst
// GEMM rate), 4K at 128 heads 611 us (1.13 PFLOP/s), 700-730 under the power limit.
//
// Roles: warp 0 TMA, warp 1 MMAs of both tiles, warps 2-3 clean the value
// tiles on the border (below), warps 4-7 and 8-11 softmax and epilogue of the tiles.
//
// Few rows over long contexts: the key tiles are split over several CTAs, whose
// normalised fp32 results and log-sum-exps expanded_merge_kernel joins.
//
// A position that some row of the CTA must not see has probability 0 there,
// and 0 x a non-finite value would reach that row all the same.  So in tiles on
// the border the cleaning warps zero the value rows that no row of the CTA
// sees, and for a non-finite value at a position that only later rows see they
// zero it and note the first such position per dim: rows that do see it get NaN,
// as from every other tile (the epilogue turns infinite sums into NaN).
#include "dense_mla.cuh"

namespace dsa {
namespace {

constexpr int kRows = 128;                 // query rows per tile (TMEM lanes)
constexpr int kKeys = 128;                 // keys per tile
constexpr int kBlk = 128 * 128;            // one [128 rows x 64 dims] block, 128-byte swizzle
constexpr int kSlots = 8;                  // ring of key / value blocks, 3 + 2 per tile
__device__ __forceinline__ int ring(int block) { return block & (kSlots - 1); }
// Of the 126 MB of L2, what a group of heads may take (32, 64, 96 MB, all heads in one group: 4K at 128 heads
// 669, 665, 662, 687 us; 8K at 16 heads, one head after the other, 1.2 x as long).
constexpr int64_t kL2Bytes = 64 << 20;
// Key tiles a part of a split has at least (2, 3, 4, 6: 20 tokens over 3000 keys at 2 heads 13.3, 14.3, 16.2,
// 18.8 us, 1 over 5000 at 16 heads 19.9, 19.9, 19.9, 22.3).
constexpr int kSplitTiles = 3;
constexpr int kThreads = 12 * 32;
constexpr uint32_t kRegLow = 120, kRegHigh = 192;    // 128 * (120 + 2 * 192) = 384 * 168
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 0, TM_O = 256;   // + 128 * tile

constexpr int OFF_Q = 0;                               // 2 tiles x 3 blocks
constexpr int OFF_KV = 6 * kBlk;
constexpr int OFF_AUX = OFF_KV + kSlots * kBlk;
constexpr int kSmem = OFF_AUX + 1536 + 1024;
static_assert(kSmem <= 232448, "shared memory of one CTA");

struct Aux {
  uint64_t q_full[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];      // by tile parity
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drain;
  uint64_t go;              // the values before the border have landed
  // A border tile's values are clean, by turns: the two cleaning warps may be a tile
  // apart, and both arrivals of a phase have to be for the same tile.
  uint64_t clean[2];
  uint32_t tmem;
  int32_t any_bad;
  int32_t bad_pos[2][128];  // first position whose value of this dim is not finite, per head of the CTA and dim
};
static_assert(sizeof(Aux) <= 1536, "");

using dense::exp2_approx;
using dense::finite_or_zero;
using dense::kGrow;
using dense::kLn2;
using dense::kNoWeight;
using dense::pack_bf16;
using dense::store_32;

// f32x2 register pairs (low element first)
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 2^x of two values on the FMA pipe: x = n + f with n an integer and |f| <= 1/2
// (adding 1.5 * 2^23 rounds to n and leaves it in the low bits), 2^f by a degree-4
// polynomial fitted for the smallest relative error on that range (2.7e-6 in fp32, far
// below the rounding to bf16), n added to the exponent.  -125 <= x: what is smaller
// gives 2^-125, so masked scores do not come here.
__device__ __forceinline__ float2 exp2_poly(uint64_t x2) {
  const float2 xv = split(x2);
  const uint64_t x = pair(max_nan(xv.x, -125.f), max_nan(xv.y, -125.f));
  const uint64_t big = pair(12582912.f, 12582912.f), minus = pair(-12582912.f, -12582912.f);
  const uint64_t y = add2(x, big);
  const uint64_t n = add2(y, minus);
  const uint64_t f = fma2(n, pair(-1.f, -1.f), x);
  uint64_t q = fma2(f, pair(0.009570101276040077f, 0.009570101276040077f), pair(0.05591786280274391f, 0.05591786280274391f));
  q = fma2(q, f, pair(0.240247443318367f, 0.240247443318367f));
  q = fma2(q, f, pair(0.6931217908859253f, 0.6931217908859253f));
  q = fma2(q, f, pair(0.9999992847442627f, 0.9999992847442627f));
  const float2 qv = split(q), yv = split(y);
  return make_float2(__int_as_float(__float_as_int(qv.x) + (__float_as_int(yv.x) << 23)),
                     __int_as_float(__float_as_int(qv.y) + (__float_as_int(yv.y) << 23)));
}

// What a CTA works on.
struct Tile {
  int row0, rows;          // rows of q
  int base;                // position of row 0, counted from the CTA's first key
  int n[2];                // key tiles of the two row tiles (0: nothing to do)
  int first_row_key;       // cache row of the first key
  bool bad;
  bool duo;                // the row tiles are the same rows of heads h and h + 1
};

// Row tile `j` of the batch's, the highest of their sequences first (equal ones in the
// sequences' order): its sequence and its number there, or false behind the last.
// Called by every thread of the block.
struct TileScratch {
  int32_t sum[kThreads / 32];
  int32_t b;
};
__device__ __forceinline__ bool find_tile(const ExpandedMlaParams& p, TileScratch& sc, int j, int& b, int& qt) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // row tiles of sequence v (0 where cu_q does not rise; more tokens than max_q: as many as max_q has)
  auto tiles = [&](int v) -> int {
    const int q0 = __ldg(&p.cu_q[v]), q1 = __ldg(&p.cu_q[v + 1]);
    if (q0 < 0 || q1 < q0 || q1 > p.total_q || (v == 0 && q0 != 0)) return 0;
    return min((q1 - q0 + 2 * kRows - 1) / (2 * kRows), p.row_tiles);
  };
  const int first = tid < p.num_seqs ? tiles(tid) : 0;
  // the sum of `c` over the block, and over the threads before this one
  auto scan = [&](int c, int& all) -> int {
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    __syncthreads();
    if (lane == 31) sc.sum[warp] = inc;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sc.sum[w];
      all += sc.sum[w];
    }
    return before + inc - c;
  };
  // tiles of number `least` and up
  auto from = [&](int least) {
    int c = max(first - least, 0), all;
    for (int v = tid + kThreads; v < p.num_seqs; v += kThreads) c += max(tiles(v) - least, 0);
    scan(c, all);
    return all;
  };
  if (j >= from(0)) return false;
  int lo = 0, hi = p.row_tiles, above = 0;      // from(lo) > j >= from(hi) = above
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, n = from(mid);
    if (n > j) {
      lo = mid;
    } else {
      hi = mid;
      above = n;
    }
  }
  qt = lo;
  // the sequence: number j - above of those that have the tile
  int rank = j - above;
  for (int v0 = 0; v0 < p.num_seqs; v0 += kThreads) {
    const int v = v0 + tid;
    const bool has = v < p.num_seqs && (v0 == 0 ? first : tiles(v)) > qt;
    int all;
    const int at = scan(has ? 1 : 0, all);
    if (has && at == rank) sc.b = v;
    if (rank < all) break;                       // uniform
    rank -= all;
  }
  __syncthreads();
  b = sc.b;
  return true;
}

template <bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_mla_kernel(const ExpandedMlaParams p, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_r) {
  // Block order: groups of heads whose keys and values fit L2 together, in a group the
  // longest rows of every head and sequence first (a head's longest row tiles, started
  // last, would run alone at the end: 8K at 16 heads, one head after the other, took 1.2 x).
  const int per_group = p.blocks * p.splits * p.head_group, units = (p.n_heads + p.head_step - 1) / p.head_step;
  const int group = static_cast<int>(blockIdx.x) / per_group;
  const int heads = min(p.head_group, units - group * p.head_group);
  const int in_group = static_cast<int>(blockIdx.x) - group * per_group;
  const int in_heads = in_group / heads;
  const int h = (group * p.head_group + in_group - in_heads * heads) * p.head_step;
  const int j = SPLIT ? in_heads / p.splits : in_heads, part = SPLIT ? in_heads - j * p.splits : 0;
  int b, qt;
  if (p.listed) {
    __shared__ TileScratch scratch;
    if (blockIdx.x == 0)
      for (int v = threadIdx.x; v < p.num_seqs; v += kThreads) {
        const int q0 = __ldg(&p.cu_q[v]), q1 = __ldg(&p.cu_q[v + 1]);
        if (q0 < 0 || q1 < q0 || q1 > p.total_q || (v == 0 && q0 != 0)) report_error(p.err, kDevErrBounds, 601, v);
      }
    if (!find_tile(p, scratch, j, b, qt)) return;
  } else {
    const int tile_up = j / p.num_seqs;
    b = j - tile_up * p.num_seqs;
    qt = p.row_tiles - 1 - tile_up;
  }
  const int q0 = __ldg(&p.cu_q[b]), q1 = __ldg(&p.cu_q[b + 1]);
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || (b == 0 && q0 != 0)) {
    if (qt == 0 && h == 0 && threadIdx.x == 0) report_error(p.err, kDevErrBounds, 601, b);
    return;
  }
  const int q_len = q1 - q0;
  if (qt * 2 * kRows >= q_len) return;
  const int kv = __ldg(&p.kv_len[b]);
  const int64_t ks = __ldg(&p.kv_start[b]);
  Tile w;
  w.bad = q_len > kv || q_len > p.max_q || kv > p.max_kv_len || ks < 0 || ks > p.total_keys - kv;
  w.row0 = q0 + qt * 2 * kRows;
  w.rows = q_len - qt * 2 * kRows;       // rows behind the last tile's are the last tile's where max_q is too small
  if (w.rows > 2 * kRows && !(w.bad && qt == p.row_tiles - 1)) w.rows = 2 * kRows;
  w.base = kv - q_len + qt * 2 * kRows;
  w.n[0] = (w.base + min(w.rows, kRows) - 1) / kKeys + 1;
  w.n[1] = w.rows > kRows ? (w.base + w.rows - 1) / kKeys + 1 : 0;
  w.first_row_key = static_cast<int>(ks);
  const int H = p.n_heads, tid = threadIdx.x;
  const int64_t part_rows = static_cast<int64_t>(part) * p.total_q;      // this part's rows in the partial results
  if (SPLIT && !w.bad) {
    // this CTA's share of the key tiles
    const int all = max(w.n[0], w.n[1]), per = (all + p.splits - 1) / p.splits, t0 = min(part * per, all);
    w.n[0] = max(0, min(w.n[0], t0 + per) - t0);
    w.n[1] = max(0, min(w.n[1], t0 + per) - t0);
    w.base -= t0 * kKeys;
    w.first_row_key += t0 * kKeys;
  }
  w.duo = !SPLIT && p.duo && !w.bad && w.rows <= kRows && (h | 1) < p.n_heads;
  if (w.duo) {
    if (h & 1) return;                       // with the head before
    w.n[1] = w.n[0];
  }
  if (w.bad || max(w.n[0], w.n[1]) == 0) {
    if (w.bad && qt == 0 && h == 0 && part == 0 && tid == 0) report_error(p.err, kDevErrBounds, 602, b);
    if (!SPLIT) {
      for (int g = h; g < min(h + p.head_step, H); ++g)
        for (int u = tid; u < w.rows * 16; u += kThreads)
          *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(w.row0 + (u >> 4)) * H + g) * 128 + (u & 15) * 8) =
              make_uint4(0, 0, 0, 0);
    }
    float* lse = SPLIT ? p.part_lse + part_rows * H : p.lse;
    if (lse != nullptr)
      for (int g = h; g < min(h + p.head_step, H); ++g)
        for (int r = tid; r < w.rows; r += kThreads)
          lse[static_cast<int64_t>(w.row0 + r) * H + g] = __int_as_float(0xff800000);
    return;
  }
  // Key tiles pass the ring one after the other; of two heads in turn (tile g of the
  // ring is key tile g / 2 of head h + (g & 1)).
  const int duo = w.duo ? 1 : 0;
  const int n_tiles = max(w.n[0], w.n[1]) << duo;
  const bool two = w.n[1] > 0;
  // first tile with a position that row 0 must not see
  const int border0 = w.base < 0 ? 0 : ((w.base + 1) / kKeys) << duo;

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Aux* ax = reinterpret_cast<Aux*>(sm + OFF_AUX);
  const uint32_t warp = warp_id(), lane = lane_id();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ax->q_full[i], 1);
      mbar_init(&ax->s_full[i], 1);
      mbar_init(&ax->p_full[i], 4);
      mbar_init(&ax->o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ax->k_full[i], 1);
      mbar_init(&ax->v_full[i], 1);
      mbar_init(&ax->k_empty[i], 1);
      mbar_init(&ax->v_empty[i], 1);
    }
    mbar_init(&ax->drain, 1);
    mbar_init(&ax->go, 1);
    mbar_init(&ax->clean[0], 2);
    mbar_init(&ax->clean[1], 2);
    fence_mbar_init();
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_kv);
    prefetch_tmap(&map_r);
  }
  if (tid < 256) ax->bad_pos[tid >> 7][tid & 127] = 0x7fffffff;
  if (tid == 0) ax->any_bad = 0;
  if (warp == 1) {
    tmem_alloc(&ax->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ax->tmem;

  if (warp < 4) {
    setmaxnreg_dec<kRegLow>();
    if (warp == 0) {
      // ----------------------------------------------------------------- TMA --
      if (elect_one()) {
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (ok && !mbar_wait(bar, parity, p.budget)) {
            report_error(p.err, kDevErrTimeout, 611, blockIdx.x);
            ok = false;
          }
          return ok;
        };
        int n_k = 0, n_v = 0;
        auto keys = [&](int i) {
          // blocks 5 i .. 5 i + 2 of the ring take the place of the last of K(i - 2) and of V(i - 2)
          if (i >= 2 && !wait(&ax->v_empty[i & 1], ((i >> 1) + 1) & 1)) return;
          uint64_t* bar = &ax->k_full[i & 1];
          const int y = w.first_row_key + (i >> duo) * kKeys, hh = h + (i & duo);
          mbar_arrive_expect_tx(bar, 3 * kBlk);
          tma_load_3d(sm + OFF_KV + ring(5 * i) * kBlk, &map_kv, bar, 0, y, hh * 4);
          tma_load_3d(sm + OFF_KV + ring(5 * i + 1) * kBlk, &map_kv, bar, 0, y, hh * 4 + 1);
          tma_load_3d(sm + OFF_KV + ring(5 * i + 2) * kBlk, &map_r, bar, 0, y, 0);
          ++n_k;
        };
        auto values = [&](int i) {
          // blocks 5 i + 3 and 5 i + 4 that of the first two of K(i - 1)
          if (i >= 1 && !wait(&ax->k_empty[(i - 1) & 1], ((i - 1) >> 1) & 1)) return;
          uint64_t* bar = &ax->v_full[i & 1];
          const int y = w.first_row_key + (i >> duo) * kKeys, hh = h + (i & duo);
          mbar_arrive_expect_tx(bar, 2 * kBlk);
          tma_load_3d(sm + OFF_KV + ring(5 * i + 3) * kBlk, &map_kv, bar, 0, y, hh * 4 + 2);
          tma_load_3d(sm + OFF_KV + ring(5 * i + 4) * kBlk, &map_kv, bar, 0, y, hh * 4 + 3);
          ++n_v;
        };
        for (int a = 0; a < (two ? 2 : 1); ++a) {
          mbar_arrive_expect_tx(&ax->q_full[a], 3 * kBlk);
          tma_load_3d(sm + OFF_Q + 3 * a * kBlk, &map_q, &ax->q_full[a], 0, w.row0 + (w.duo ? 0 : a * kRows),
                      (w.duo ? h + a : h) * 3);
          if (a == 0) keys(0);
        }
        values(0);
        if (n_tiles > 1) keys(1);
        for (int i = 1; ok && i < n_tiles; ++i) {
          values(i);
          if (ok && i + 1 < n_tiles) keys(i + 1);
        }
        // all copies land before the block ends, also those that nothing waits for any more
        // because a wait has run out, here or in another role
        bool landed = true;
        for (int a = 0; a < (two ? 2 : 1); ++a) landed = landed && mbar_wait(&ax->q_full[a], 0, kDrainCycles);
        for (int i = max(0, n_k - 2); landed && i < n_k; ++i)
          landed = mbar_wait(&ax->k_full[i & 1], (i >> 1) & 1, kDrainCycles);
        for (int i = max(0, n_v - 2); landed && i < n_v; ++i)
          landed = mbar_wait(&ax->v_full[i & 1], (i >> 1) & 1, kDrainCycles);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMAs --
      // One thread for both row tiles, in a fixed order that keeps them half a
      // period apart: with a thread each they fall into step, both softmaxes
      // and then both products (8K at 16 heads 420 -> 502 us).
      if (elect_one()) {
        constexpr uint32_t idesc_s = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 128, 0, 0);
        constexpr uint32_t idesc_o = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 128, 0, 1);     // V MN-major
        constexpr uint32_t idesc_half = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 64, 0, 1);
        // descriptors: offsets are added to the address field (16-byte units)
        const uint64_t q_desc = smem_desc(smem_u32(sm + OFF_Q), 16, 1024, kSwizzle128B);
        const uint64_t k_desc = smem_desc(smem_u32(sm + OFF_KV), 16, 1024, kSwizzle128B);
        const uint64_t v_desc = smem_desc(smem_u32(sm + OFF_KV), kBlk, 1024, kSwizzle128B);
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
          if (ok && !mbar_wait(bar, parity, p.budget)) {
            report_error(p.err, kDevErrTimeout, site, blockIdx.x);
            ok = false;
          }
          return ok;
        };
        // `last`: of the row tiles that read key tile i
        auto scores = [&](int a, int i, bool last) {
          const uint32_t d_s = tmem + TM_S + 128 * a;
          const uint64_t qd = q_desc + a * ((3 * kBlk) >> 4);
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const uint64_t kd = k_desc + ring(5 * i + c) * (kBlk >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ss(d_s, qd + ((c * kBlk + kk * 32) >> 4), kd + ((kk * 32) >> 4), idesc_s, (c | kk) ? 1u : 0u);
          }
          umma_commit(&ax->s_full[a]);
          if (last) umma_commit(&ax->k_empty[i & 1]);
        };
        auto values = [&](int a, int i, bool last) {
          const uint32_t d_s = tmem + TM_S + 128 * a, d_o = tmem + TM_O + 128 * a;
          // one instruction spans both 64-dim blocks where the ring keeps them side by side, else two
          const int n0 = ring(5 * i + 3), n1 = ring(5 * i + 4);
          const uint64_t vd = v_desc + n0 * (kBlk >> 4);
          if (n1 > n0) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_f16_ts(d_o, d_s + kk * 8, vd + ((kk * 2048) >> 4), idesc_o, ((i >> duo) | kk) ? 1u : 0u);
          } else {
            const uint64_t vd1 = v_desc + n1 * (kBlk >> 4);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              umma_f16_ts(d_o, d_s + kk * 8, vd + ((kk * 2048) >> 4), idesc_half, ((i >> duo) | kk) ? 1u : 0u);
              umma_f16_ts(d_o + 64, d_s + kk * 8, vd1 + ((kk * 2048) >> 4), idesc_half, ((i >> duo) | kk) ? 1u : 0u);
            }
          }
          umma_commit(&ax->o_done[a]);
          if (last) umma_commit(&ax->v_empty[i & 1]);
        };
        if (border0 == 0) mbar_arrive(&ax->go);
        wait(&ax->q_full[0], 0, 620);
        wait(&ax->k_full[0], 0, 621);
        if (two) wait(&ax->q_full[1], 0, 620);
        tc_fence_after();
        if (ok && w.n[0] > 0) scores(0, 0, w.duo || !two);
        if (ok && two && (!w.duo || wait(&ax->k_full[1], 0, 625))) {
          tc_fence_after();
          scores(1, duo, true);
        }
        for (int i = 0; ok && i < n_tiles; ++i) {
          wait(&ax->v_full[i & 1], (i >> 1) & 1, 624);
          if (i + 1 == border0 && p.skip_arrival < 0) mbar_arrive(&ax->go);
          if (i >= border0) wait(&ax->clean[(i - border0) & 1], ((i - border0) >> 1) & 1, 623);
          if (w.duo) {
            // One head's product each; the next keys land over tiles that are done, so the next
            // scores of both heads follow the second's product.
            if (!wait(&ax->p_full[i & 1], (i >> 1) & 1, 622)) break;
            tc_fence_after();
            values(i & 1, i, true);
            for (int g = i + 1; ok && (i & 1) != 0 && g < min(i + 3, n_tiles); ++g)
              if (wait(&ax->k_full[g & 1], (g >> 1) & 1, 625)) {
                tc_fence_after();
                scores(g & 1, g, true);
              }
            continue;
          }
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const bool last = a == 1 || !two;
            if (i >= w.n[a]) continue;
            if (!wait(&ax->p_full[a], i & 1, 622)) break;
            tc_fence_after();
            values(a, i, last);
            if (i + 1 < w.n[a] && wait(&ax->k_full[(i + 1) & 1], ((i + 1) >> 1) & 1, 625)) {
              tc_fence_after();
              scores(a, i + 1, last);
            }
          }
        }
        // the MMAs in flight end before their memory goes, whichever role has given up
        umma_commit(&ax->drain);
        mbar_wait(&ax->drain, 0, kDrainCycles);
      }
    } else {
      // -------------------------------------------- value tiles on the border --
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok && !mbar_wait(bar, parity, p.budget)) {
          report_error(p.err, kDevErrTimeout, 631, blockIdx.x);
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
      };
      // These warps skip the tiles before the border, and a parity alone would not
      // tell them where the ring is: the MMA thread, which follows every phase, does once.
      if (border0 < n_tiles) wait(&ax->go, 0);
      for (int i = border0; ok && i < n_tiles; ++i) {
        wait(&ax->v_full[i & 1], (i >> 1) & 1);
        if (!ok) break;
        const int key0 = (i >> duo) * kKeys;
        const int first = max(0, w.base + 1 - key0);               // the rows before are seen by every row
        const int dead = min(kKeys, w.base + w.rows - key0);       // rows from here on by none
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint4* blk = reinterpret_cast<uint4*>(sm + OFF_KV + ring(5 * i + 3 + c) * kBlk);
          for (int u = 8 * max(first, dead) + tid - 64; u < kBlk / 16; u += 64) blk[u] = make_uint4(0, 0, 0, 0);
          // row r of the block is position key0 + r; unit u of it holds dims 8 (u ^ (r & 7)) ..
#pragma unroll 1
          for (int u0 = 8 * first + tid - 64; u0 < 8 * dead; u0 += 4 * 64) {
            uint4 v[4];
            bool any = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = u0 + 64 * q < 8 * dead ? blk[u0 + 64 * q] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) any |= dense::any_not_finite(v[q]);
            if (!any) continue;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              const int u = u0 + 64 * q, r = u >> 3;
              if (u >= 8 * dead) break;
              const uint4 a = blk[u];
              const uint32_t x[4] = {a.x, a.y, a.z, a.w};
              blk[u] = finite_or_zero(a);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t mask = 0x7F80u << (16 * (e & 1));
                if ((x[e >> 1] & mask) == mask) {
                  atomicMin(&ax->bad_pos[i & duo][c * 64 + 8 * ((u & 7) ^ (r & 7)) + e], key0 + r);
                  ax->any_bad = 1;
                }
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ax->clean[(i - border0) & 1]);
      }
    }
  } else {
    setmaxnreg_inc<kRegHigh>();
    // ----------------------------------------------------- softmax, epilogue --
    const int a = static_cast<int>(warp >> 2) - 1;
    const uint32_t quarter = warp & 3u;
    const int r0 = w.duo ? 0 : a * kRows, r = r0 + static_cast<int>(quarter * 32 + lane);     // row of the CTA
    const uint32_t t_lane = tmem + ((quarter * 32u) << 16);
    const uint32_t tS = t_lane + TM_S + 128 * a, tO = t_lane + TM_O + 128 * a;
    const float scale = p.scale_log2, NEG_INF = __int_as_float(0xff800000);
    // rows behind the last one follow it (their results are not stored)
    const int lim = w.base + min(r, w.rows - 1);
    const int warp_lim = w.base + min(r0 + static_cast<int>(quarter * 32), w.rows - 1);
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
      if (ok && !mbar_wait(bar, parity, p.budget)) {
        report_error(p.err, kDevErrTimeout, site, blockIdx.x);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    float m = NEG_INF, l = 0.f;
    const int nt = w.n[a];
    for (int i = 0; ok && i < nt; ++i) {
      if (!wait(&ax->s_full[a], i & 1, 641)) break;
      tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s[c]);
      tmem_ld_wait();
      const int left = lim - i * kKeys;          // columns 0 .. left are seen
      if (warp_lim - i * kKeys < kKeys - 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (32 * c + j > left) s[c][j] = __float_as_uint(NEG_INF);
      }
      // The row's maximum, NaN if any score is: such a row is NaN from here on.
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int j = 1; j < 32; ++j) mx[c] = max_nan(mx[c], __uint_as_float(s[c][j]));
      }
      const float top = max_nan(max_nan(mx[0], mx[1]), max_nan(mx[2], mx[3])) * scale;
      const bool grow = !(top <= m + kGrow);     // true on the first tile that shows the row a key
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? exp2_approx(m - top) : 1.f;
        if (grow) m = top < __int_as_float(0x7f800000) ? top : __int_as_float(0x7fffffff);      // an infinite score: NaN too
        l *= f;
        if (i > 0) {
          if (!wait(&ax->o_done[a], (i - 1) & 1, 642)) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            asm volatile(
                "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                "%14, %15}, [%16];"
                : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
                  "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
                : "r"(tO + 16 * c));
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st16(tO + 16 * c, o);
          }
        }
      }
      const float ref = m == NEG_INF ? 0.f : -m;
      const uint64_t scale2 = pair(scale, scale), ref2 = pair(ref, ref);
      uint64_t sum2 = pair(0.f, 0.f);
      const bool masked = warp_lim - i * kKeys < kKeys - 1;
      // Some of the exponentials go to the FMA pipe: the two row tiles' 32K at 16 a
      // cycle would alone take 2048 cycles of a period.
      auto probabilities = [&](int c, bool poly) {
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint64_t x = fma2(pair(__uint_as_float(s[c][2 * j]), __uint_as_float(s[c][2 * j + 1])), scale2, ref2);
          float2 e;
          if (poly && (j & 3) == 3) {
            e = exp2_poly(x);
          } else {
            const float2 v = split(x);
            e = make_float2(exp2_approx(v.x), exp2_approx(v.y));
          }
          sum2 = add2(sum2, pair(e.x, e.y));
          pk[j] = pack_bf16(e.x, e.y);
        }
        tmem_st16(tS + 16 * c, pk);
      };
      if (masked) {
#pragma unroll
        for (int c = 0; c < 4; ++c) probabilities(c, false);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) probabilities(c, true);
      }
      const float2 sums = split(sum2);
      l += sums.x + sums.y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ax->p_full[a]);
    }
    if (ok && nt > 0 && wait(&ax->o_done[a], (nt - 1) & 1, 643)) {
      tc_fence_after();
      // 0: no key has a weight, those of a part that the row does not see or scores of -inf throughout
      const float inv = l == 0.f || m == NEG_INF ? 0.f : 1.f / l;
      const uint64_t inv2 = pair(inv, inv), zero2 = pair(0.f, 0.f);
      // o / l; what is not finite in the sum (an infinite value, whatever its weight) becomes NaN
      auto normal = [&](const uint32_t* x) {
        const uint64_t v = pair(__uint_as_float(x[0]), __uint_as_float(x[1]));
        return split(fma2(v, zero2, mul2(v, inv2)));
      };
      const int64_t at = static_cast<int64_t>(w.row0 + r) * H + h + (w.duo ? a : 0);
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        uint32_t o[2][32];
        tmem_ld32(tO + 32 * c, o[0]);
        tmem_ld32(tO + 32 * c + 32, o[1]);
        tmem_ld_wait();
        if (ax->any_bad != 0) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (ax->bad_pos[w.duo ? a : 0][32 * c + j] <= lim) o[j >> 5][j & 31] = 0x7FFFFFFFu;
        }
        if (SPLIT && r < w.rows) {
          float* to = p.part_o + (part_rows * H + at) * 128 + 32 * c;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 y = normal(&o[u >> 2][8 * (u & 3) + e]);
              v[e] = __float_as_uint(y.x);
              v[e + 1] = __float_as_uint(y.y);
            }
            store_32(to + 8 * u, v);
          }
        } else if (r < w.rows) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t* x = &o[u >> 1][16 * (u & 1)];
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 y = normal(x + 2 * e);
              v[e] = pack_bf16(y.x, y.y);
            }
            store_32(p.out + at * 128 + 32 * c + 16 * u, v);
          }
        }
        __syncwarp();
      }
      if (r < w.rows) {
        const float lse2 = l == 0.f ? NEG_INF : m + log2f(l);
        if (SPLIT) {
          p.part_lse[part_rows * H + at] = lse2 == NEG_INF ? kNoWeight : lse2;
        } else if (p.lse != nullptr) {
          p.lse[at] = lse2 * kLn2;
        }
      }
    } else if (SPLIT && nt == 0 && r < w.rows) {
      p.part_lse[part_rows * H + static_cast<int64_t>(w.row0 + r) * H + h] = NEG_INF;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the parts of each (row, head), a warp each, 4 dims a lane: weights 2^(lse_i - max).
__global__ void __launch_bounds__(256) expanded_merge_kernel(const ExpandedMlaParams p) {
  const float NEG_INF = __int_as_float(0xff800000);
  const int64_t all = static_cast<int64_t>(p.total_q) * p.n_heads;
  const int64_t rows = static_cast<int64_t>(min(max(__ldg(&p.cu_q[p.num_seqs]), 0), p.total_q)) * p.n_heads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = static_cast<int>(threadIdx.x & 31u);
  if (row >= rows) return;
  float m = NEG_INF;
  for (int i = lane; i < p.splits; i += 32) m = fmaxf(m, p.part_lse[i * all + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float ref = m <= kNoWeight ? 0.f : m;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < p.splits; ++i) {
    const float z = p.part_lse[i * all + row];
    if (z == NEG_INF) continue;            // an empty part: its output was not written
    const float w = exp2f(z - ref);
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (i * all + row) * 128 + lane * 4);
    sum += w;
    acc.x += w * v.x;
    acc.y += w * v.y;
    acc.z += w * v.z;
    acc.w += w * v.w;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint2 out;
  out.x = pack_bf16(acc.x * inv, acc.y * inv);
  out.y = pack_bf16(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.out + row * 128 + lane * 4) = out;
  if (lane == 0 && p.lse != nullptr) p.lse[row] = sum == 0.f ? NEG_INF : (ref + log2f(sum)) * kLn2;
}

}  // namespace

int expanded_most_splits(int max_kv_len, int n_heads) {
  const int tiles = (max_kv_len + kKeys - 1) / kKeys, s = kDenseMaxCtas / n_heads;
  return s < tiles / kSplitTiles ? s : (tiles / kSplitTiles > 1 ? tiles / kSplitTiles : 1);
}

int expanded_splits(const dsa_batch_t* b, int n_heads) {
  const int64_t units = static_cast<int64_t>((b->max_q_per_seq + 2 * kRows - 1) / (2 * kRows)) * b->num_seqs;
  const int64_t ctas = units * n_heads, rows = static_cast<int64_t>(b->total_q) * n_heads;
  if (ctas < 1 || ctas > kDenseMaxCtas / 2 || rows < 1) return 1;
  const int64_t s = kDenseMaxCtas / ctas, fit = kExpandedPartRows / rows, most = expanded_most_splits(b->max_kv_len, n_heads);
  const int64_t least = s < fit ? (s < most ? s : most) : (fit < most ? fit : most);
  return static_cast<int>(least > 1 ? least : 1);
}

cudaError_t launch_expanded_mla(const ExpandedMlaParams& p, const CUtensorMap& map_q, const CUtensorMap& map_kv,
                                const CUtensorMap& map_r, cudaStream_t stream) {
  const auto kernel = p.splits > 1 ? expanded_mla_kernel<true> : expanded_mla_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  ExpandedMlaParams q = p;
  q.row_tiles = (p.max_q + 2 * kRows - 1) / (2 * kRows);
  // Blocks per head: a row tile of every sequence each, or, where the batch's tokens fill
  // less than half of them, as many as they can fill, which look up their tile.  A block that
  // finds nothing to do costs ~0.8 us of its SM, the search ~0.6 us of each block: 2048 and
  // 63 x 8 tokens at 16 heads 117 -> 81 us, 32 sequences of 1-500 (63 of 64) 72 -> 76.
  const int64_t every = static_cast<int64_t>(q.row_tiles) * p.num_seqs;
  const int64_t most = p.total_q / (2 * kRows) + p.num_seqs;
  q.listed = 2 * most < every ? 1 : 0;
  q.blocks = static_cast<int>(q.listed ? most : every);
  const int64_t seen = static_cast<int64_t>(p.num_seqs) * p.max_kv_len;
  const int64_t fit = kL2Bytes / ((p.total_keys < seen ? p.total_keys : seen) * 512);      // heads' keys and values in L2
  // Two heads per block where a row tile holds at most 128 rows: a block of few rows is a chain of
  // latencies (~7 us for one key tile), and two chains take little longer (16 x 100 tokens at
  // 128 heads 126 -> 92 us, 500 x 40 at 16 391 -> 237, 2 x 5 tokens at 128 heads, 256 blocks, 38 -> 31).
  // Not where the GPU has an SM for every block or nearly so (6 ragged prompts at 16 heads, 128 blocks
  // of 192 in use: 25.6 -> 27.8).
  q.duo = p.splits == 1 && p.n_heads > 1 && 2 * (q.listed ? most : every) * p.n_heads > 3 * sm_count() ? 1 : 0;
  q.head_step = q.duo && p.max_q <= kRows ? 2 : 1;
  const int units = (p.n_heads + q.head_step - 1) / q.head_step;
  const int64_t group = fit / q.head_step;
  q.head_group = static_cast<int>(group < 1 ? 1 : (group < units ? group : units));
  const int64_t blocks = (q.listed ? most : every) * units * p.splits;
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  kernel<<<static_cast<unsigned>(blocks), kThreads, kSmem, stream>>>(q, map_q, map_kv, map_r);
  const cudaError_t f = cudaGetLastError();
  if (f != cudaSuccess || p.splits == 1) return f;
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.n_heads;
  expanded_merge_kernel<<<static_cast<unsigned>((rows + 7) / 8), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
