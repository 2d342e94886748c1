// Latent attention in the expanded form for long prompts: a CTA pair per 512 query
// rows of a head, tcgen05 cta_group::2.
//
// The same work as expanded_mla_sm100.cu (its mathematics, its two row tiles in
// turn, its border), with row tiles of 256 rows: each CTA holds 128 of a tile's
// rows in its tensor memory and half of every key tile, 64 of the 128 keys for S
// and 64 of the 128 value dims for O, which the tensor cores of both read.
// Per key tile a CTA then takes in 40 KB instead of 80 and S reads 96 B/clk of shared
// memory instead of 128, which is what slows the products of the one-CTA kernel down.
//
// Roles per CTA: warp 0 TMA, warp 1 MMAs (rank 0), warps 2-3 clean this CTA's value
// dims on the border, warps 4-7 and 8-11 softmax and epilogue of the two row tiles.
// Key and value blocks have a ring of three stages each.
#include "expanded_mla.cuh"

namespace dsa {
namespace {

using namespace expanded;

constexpr int kRows = 128;                 // rows per row tile and CTA
constexpr int kItemRows = 512;             // 2 tiles x 2 CTAs x 128
constexpr int kKeys = 128;
constexpr int kQBlk = 128 * 128;           // [128 rows x 64 dims]
constexpr int kKBlk = 64 * 128;            // [64 keys x 64 dims]
constexpr int kK = 3 * kKBlk;              // this CTA's keys of a tile
constexpr int kV = 128 * 128;              // [128 keys x 64 dims]: its value dims
constexpr int kStages = 3;
constexpr int kThreads = 12 * 32;
constexpr uint32_t kRegLow = 120, kRegHigh = 192;    // 128 * (120 + 2 * 192) = 384 * 168
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 0, TM_O = 256;   // + 128 * tile
constexpr int64_t kL2Bytes = 64 << 20;     // of L2 that a group of heads may take

constexpr int OFF_Q = 0;                               // 2 tiles x 3 blocks
constexpr int OFF_K = 6 * kQBlk;
constexpr int OFF_V = OFF_K + kStages * kK;
constexpr int OFF_AUX = OFF_V + kStages * kV;
constexpr int kSmem = OFF_AUX + 1024 + 1024;
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(OFF_V % 1024 == 0 && kK % 1024 == 0, "swizzle atoms");

struct Aux {
  // rank 0's: loads of both CTAs
  uint64_t q_full[2];
  uint64_t k_full[kStages], v_full[kStages];
  uint64_t p_full[2];
  uint64_t clean[kStages];  // border tiles by turns: cleaned in both CTAs (warps may be tiles apart, within the ring)
  // each CTA's
  uint64_t k_empty[kStages], v_empty[kStages];
  uint64_t border_full[kStages];      // a border tile's values landed here
  uint64_t s_full[2], o_done[2];
  uint32_t tmem;
  int32_t any_bad;
  int32_t bad_pos[128];     // first position whose value of this dim is not finite, per dim
};
static_assert(sizeof(Aux) <= 1024, "");

// A operand from tensor memory (each CTA's rows in its own).
__device__ __forceinline__ void umma_f16_ts_pair(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expanded_pair_kernel(const ExpandedMlaParams p, const __grid_constant__ ExpandedMaps maps) {
  // item order: see expanded_mla_sm100.cu
  const uint32_t rank = cluster_ctarank();
  const int item = static_cast<int>(blockIdx.x >> 1);
  const int per_group = p.row_tiles * p.num_seqs * p.head_group;
  const int group = item / per_group;
  const int heads = min(p.head_group, p.n_heads - group * p.head_group);
  const int in_group = item - group * per_group;
  const int in_heads = in_group / heads;
  const int h = group * p.head_group + in_group - in_heads * heads;
  const int tile_up = in_heads / p.num_seqs, b = in_heads - tile_up * p.num_seqs;
  const int qt = p.row_tiles - 1 - tile_up;
  const int H = p.n_heads, tid = threadIdx.x;
  const int q0 = __ldg(&p.cu_q[b]), q1 = __ldg(&p.cu_q[b + 1]);
  const int kv = __ldg(&p.kv_len[b]);
  const int64_t ks = __ldg(&p.kv_start[b]);
  // (both CTAs of a pair take the same way out)
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || (b == 0 && q0 != 0)) {
    if (qt == 0 && h == 0 && rank == 0 && tid == 0) report_error(p.err, kDevErrBounds, 601, b);
    return;
  }
  const int q_len = q1 - q0;
  if (qt * kItemRows >= q_len) return;
  const int row0 = q0 + qt * kItemRows, rows = min(kItemRows, q_len - qt * kItemRows);
  if (q_len > kv || q_len > p.max_q || kv > p.max_kv_len || ks < 0 || ks + kv > p.total_keys) {
    if (qt == 0 && h == 0 && rank == 0 && tid == 0) report_error(p.err, kDevErrBounds, 602, b);
    for (int u = 2 * tid + static_cast<int>(rank); u < rows * 16; u += 2 * kThreads)
      *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(row0 + (u >> 4)) * H + h) * 128 + (u & 15) * 8) =
          make_uint4(0, 0, 0, 0);
    if (p.lse != nullptr && rank == 0)
      for (int r = tid; r < rows; r += kThreads)
        p.lse[static_cast<int64_t>(row0 + r) * H + h] = __int_as_float(0xff800000);
    return;
  }
  const int base = kv - q_len + qt * kItemRows;          // position of the item's first row
  const int key0 = static_cast<int>(ks);
  // key tiles of the two row tiles
  const int n0 = (base + min(rows, 2 * kRows) - 1) / kKeys + 1;
  const int n1 = rows > 2 * kRows ? (base + rows - 1) / kKeys + 1 : 0;
  const int n_tiles = max(n0, n1);
  const bool two = n1 > 0;
  const int border0 = (base + 1) / kKeys;                // first tile with a position that row 0 must not see

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Aux* ax = reinterpret_cast<Aux*>(sm + OFF_AUX);
  const uint32_t warp = warp_id(), lane = lane_id();
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ax->q_full[i], 1);
      mbar_init(&ax->p_full[i], 8);           // the tile's softmax warps of both CTAs
      mbar_init(&ax->s_full[i], 1);
      mbar_init(&ax->o_done[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&ax->k_full[i], 1);
      mbar_init(&ax->v_full[i], 1);
      mbar_init(&ax->k_empty[i], 1);
      mbar_init(&ax->v_empty[i], 1);
      mbar_init(&ax->border_full[i], 1);
      mbar_init(&ax->clean[i], 4);            // the cleaning warps of both CTAs
    }
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.k);
    prefetch_tmap(&maps.r);
    prefetch_tmap(&maps.v);
  }
  if (tid < 128) ax->bad_pos[tid] = 0x7fffffff;
  if (tid == 0) ax->any_bad = 0;
  if (warp == 1) tmem_alloc_pair(&ax->tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();                              // the other CTA's barriers exist
  const uint32_t tmem = ax->tmem;

  if (warp < 4) {
    setmaxnreg_dec<kRegLow>();
    if (warp == 0) {
      // ----------------------------------------------------------------- TMA --
      if (elect_one()) {
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          if (ok && !mbar_wait(bar, parity, p.budget)) {
            report_error(p.err, kDevErrTimeout, 651, blockIdx.x);
            ok = false;
          }
          return ok;
        };
        auto rows_of = [&](int a) {
          if (rank == 0) mbar_arrive_expect_tx(&ax->q_full[a], 2 * 3 * kQBlk);
          tma_load_3d_pair(sm + OFF_Q + 3 * a * kQBlk, &maps.q, mapa_shared(smem_u32(&ax->q_full[a]), 0), 0,
                           row0 + a * 2 * kRows + static_cast<int>(rank) * kRows, h * 3);
        };
        auto keys = [&](int i) {
          const int s = i % kStages;
          if (i >= kStages && !wait(&ax->k_empty[s], ((i / kStages) + 1) & 1)) return;
          if (rank == 0) mbar_arrive_expect_tx(&ax->k_full[s], 2 * kK);
          const uint32_t bar = mapa_shared(smem_u32(&ax->k_full[s]), 0);
          const int y = key0 + i * kKeys + 64 * static_cast<int>(rank);
          tma_load_3d_pair(sm + OFF_K + s * kK, &maps.k, bar, 0, y, h * 4);
          tma_load_3d_pair(sm + OFF_K + s * kK + 2 * kKBlk, &maps.r, bar, 0, y, 0);
        };
        auto values = [&](int i) {
          const int s = i % kStages, y = key0 + i * kKeys, z = h * 4 + 2 + static_cast<int>(rank);
          if (i >= kStages && !wait(&ax->v_empty[s], ((i / kStages) + 1) & 1)) return;
          if (i >= border0) {                  // this CTA's cleaning warps take it from here
            mbar_arrive_expect_tx(&ax->border_full[s], kV);
            tma_load_3d(sm + OFF_V + s * kV, &maps.v, &ax->border_full[s], 0, y, z);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&ax->v_full[s], 2 * kV);
            tma_load_3d_pair(sm + OFF_V + s * kV, &maps.v, mapa_shared(smem_u32(&ax->v_full[s]), 0), 0, y, z);
          }
        };
        rows_of(0);
        keys(0);
        if (two) rows_of(1);
        values(0);
        for (int i = 1; ok && i < n_tiles; ++i) {
          keys(i);
          if (ok) values(i);
        }
        if (!ok) drain_pause();
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMAs --
      if (rank == 0 && elect_one()) {
        constexpr uint32_t idesc_s = idesc_f32acc(kFmtBF16, kFmtBF16, 256, 128, 0, 0);
        constexpr uint32_t idesc_o = idesc_f32acc(kFmtBF16, kFmtBF16, 256, 128, 0, 1);     // V MN-major
        const uint64_t q_desc = smem_desc(smem_u32(sm + OFF_Q), 16, 1024, kSwizzle128B);
        const uint64_t k_desc = smem_desc(smem_u32(sm + OFF_K), 16, 1024, kSwizzle128B);
        const uint64_t v_desc = smem_desc(smem_u32(sm + OFF_V), kV, 1024, kSwizzle128B);
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
          const int s = i % kStages;
          const uint32_t d_s = tmem + TM_S + 128 * a;
          const uint64_t qd = q_desc + a * ((3 * kQBlk) >> 4), kd = k_desc + s * (kK >> 4);
#pragma unroll
          for (int c = 0; c < 3; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ss_pair(d_s, qd + ((c * kQBlk + kk * 32) >> 4), kd + ((c * kKBlk + kk * 32) >> 4), idesc_s,
                               (c | kk) ? 1u : 0u);
          umma_commit_pair(&ax->s_full[a]);
          if (last) umma_commit_pair(&ax->k_empty[s]);
        };
        auto values = [&](int a, int i, bool last) {
          const int s = i % kStages;
          const uint32_t d_s = tmem + TM_S + 128 * a, d_o = tmem + TM_O + 128 * a;
          const uint64_t vd = v_desc + s * (kV >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_f16_ts_pair(d_o, d_s + kk * 8, vd + ((kk * 2048) >> 4), idesc_o, (i | kk) ? 1u : 0u);
          umma_commit_pair(&ax->o_done[a]);
          if (last) umma_commit_pair(&ax->v_empty[s]);
        };
        wait(&ax->q_full[0], 0, 660);
        wait(&ax->k_full[0], 0, 661);
        tc_fence_after();
        if (ok) scores(0, 0, !two);
        if (ok && two && wait(&ax->q_full[1], 0, 660)) {
          tc_fence_after();
          scores(1, 0, true);
        }
        for (int i = 0; ok && i < n_tiles; ++i) {
          if (i < border0) {
            wait(&ax->v_full[i % kStages], (i / kStages) & 1, 664);
          } else {
            wait(&ax->clean[(i - border0) % kStages], ((i - border0) / kStages) & 1, 663);
          }
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            const bool last = a == 1 || !two;
            const int n = a == 0 ? n0 : n1;
            if (i >= n) continue;
            if (!wait(&ax->p_full[a], i & 1, 662)) break;
            tc_fence_after();
            values(a, i, last);
            if (i + 1 < n && wait(&ax->k_full[(i + 1) % kStages], ((i + 1) / kStages) & 1, 665)) {
              tc_fence_after();
              scores(a, i + 1, last);
            }
          }
        }
        if (!ok) drain_pause();      // the MMAs in flight, before their memory goes
      }
    } else {
      // -------------------------------------------- value tiles on the border --
      bool ok = true;
      const uint32_t clean0 = mapa_shared(smem_u32(&ax->clean[0]), 0);
      const uint32_t other_pos = mapa_shared(smem_u32(&ax->bad_pos[0]), rank ^ 1u);
      const uint32_t other_any = mapa_shared(smem_u32(&ax->any_bad), rank ^ 1u);
      const int dim0 = 64 * static_cast<int>(rank);        // this CTA's value dims
      for (int i = border0; i < n_tiles; ++i) {
        const int s = i % kStages;
        // the stage's uses by border tiles before this one: i - 3, i - 6, .. from border0 on
        if (ok && !mbar_wait(&ax->border_full[s], ((i - border0) / kStages) & 1, p.budget)) {
          report_error(p.err, kDevErrTimeout, 671, blockIdx.x);
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int first = max(0, base + 1 - i * kKeys);               // the keys before are seen by every row
        const int dead = min(kKeys, base + rows - i * kKeys);         // keys from here on by none
        uint4* blk = reinterpret_cast<uint4*>(sm + OFF_V + s * kV);
        for (int u = 8 * max(first, dead) + tid - 64; u < kV / 16; u += 64) blk[u] = make_uint4(0, 0, 0, 0);
        bool found = false;
        // row r of the block is position i * 128 + r; unit u of it holds dims 8 (u ^ (r & 7)) ..
#pragma unroll 1
        for (int u0 = 8 * first + tid - 64; u0 < 8 * dead; u0 += 4 * 64) {
          uint4 v[4];
          uint32_t t = 0;
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = u0 + 64 * q < 8 * dead ? blk[u0 + 64 * q] : make_uint4(0, 0, 0, 0);
          // an exponent of all ones carries into its half's top bit
#pragma unroll
          for (int q = 0; q < 4; ++q)
            t |= ((v[q].x & 0x7F807F80u) + 0x00800080u) | ((v[q].y & 0x7F807F80u) + 0x00800080u) |
                 ((v[q].z & 0x7F807F80u) + 0x00800080u) | ((v[q].w & 0x7F807F80u) + 0x00800080u);
          if ((t & 0x80008000u) == 0) continue;
          found = true;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int u = u0 + 64 * q, r = u >> 3;
            if (u >= 8 * dead) break;
            const uint4 x4 = blk[u];
            const uint32_t x[4] = {x4.x, x4.y, x4.z, x4.w};
            blk[u] = make_uint4(finite_or_zero(x4.x), finite_or_zero(x4.y), finite_or_zero(x4.z), finite_or_zero(x4.w));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t mask = 0x7F80u << (16 * (e & 1));
              if ((x[e >> 1] & mask) == mask) {
                // noted in both CTAs: their rows read all value dims
                const int dim = dim0 + 8 * ((u & 7) ^ (r & 7)) + e;
                atomicMin(&ax->bad_pos[dim], i * kKeys + r);
                asm volatile("red.relaxed.cluster.shared::cluster.min.s32 [%0], %1;" ::"r"(other_pos + 4 * dim),
                             "r"(i * kKeys + r)
                             : "memory");
                ax->any_bad = 1;
                asm volatile("st.relaxed.cluster.shared::cluster.s32 [%0], %1;" ::"r"(other_any), "r"(1) : "memory");
              }
            }
          }
        }
        if (__any_sync(0xffffffffu, found)) asm volatile("fence.acq_rel.cluster;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(clean0 + 8 * ((i - border0) % kStages));
      }
      if (!ok) drain_pause();
    }
  } else {
    setmaxnreg_inc<kRegHigh>();
    // ----------------------------------------------------- softmax, epilogue --
    const int a = static_cast<int>(warp >> 2) - 1;
    const uint32_t quarter = warp & 3u;
    const int r0 = a * 2 * kRows + static_cast<int>(rank) * kRows + static_cast<int>(quarter * 32);   // warp's first row
    const int r = r0 + static_cast<int>(lane);                                                        // row of the item
    const uint32_t t_lane = tmem + ((quarter * 32u) << 16);
    const uint32_t tS = t_lane + TM_S + 128 * a, tO = t_lane + TM_O + 128 * a;
    const float scale = p.scale_log2, NEG_INF = __int_as_float(0xff800000);
    const uint32_t p_full = mapa_shared(smem_u32(&ax->p_full[a]), 0);
    // rows behind the last one follow it (their results are not stored)
    const int lim = base + min(r, rows - 1), warp_lim = base + min(r0, rows - 1);
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
    const int nt = a == 0 ? n0 : n1;
    for (int i = 0; ok && i < nt; ++i) {
      if (!wait(&ax->s_full[a], i & 1, 681)) break;
      tc_fence_after();
      if (!softmax_tile(tS, tO, scale, lim - i * kKeys, warp_lim - i * kKeys < kKeys - 1, i == 0, m, l,
                        [&] { return wait(&ax->o_done[a], (i - 1) & 1, 682); }))
        break;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(p_full);
    }
    if (ok && nt > 0 && wait(&ax->o_done[a], (nt - 1) & 1, 683)) {
      tc_fence_after();
      asm volatile("fence.acq_rel.cluster;" ::: "memory");       // the other CTA's notes of bad values
      const bool any_bad = *reinterpret_cast<volatile int32_t*>(&ax->any_bad) != 0;
      const float inv = 1.f / l;
      const int64_t at = static_cast<int64_t>(row0 + r) * H + h;
#pragma unroll 1
      for (int c = 0; c < 4; c += 2) {
        uint32_t o[2][32];
        tmem_ld32(tO + 32 * c, o[0]);
        tmem_ld32(tO + 32 * c + 32, o[1]);
        tmem_ld_wait();
        if (any_bad) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (*reinterpret_cast<volatile int32_t*>(&ax->bad_pos[32 * c + j]) <= lim) o[j >> 5][j & 31] = 0x7FFFFFFFu;
        }
        if (r < rows) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t* x = &o[u >> 1][16 * (u & 1)];
            uint32_t v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              v[e] = pack_bf16(__uint_as_float(x[2 * e]) * inv, __uint_as_float(x[2 * e + 1]) * inv);
            store_32(p.out + at * 128 + 32 * c + 16 * u, v);
          }
        }
        __syncwarp();
      }
      if (r < rows && p.lse != nullptr) p.lse[at] = (m + log2f(l)) * kLn2;
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

}  // namespace

cudaError_t launch_expanded_pair(const ExpandedMlaParams& p, const ExpandedMaps& maps, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(expanded_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  ExpandedMlaParams q = p;
  q.row_tiles = (p.max_q + kItemRows - 1) / kItemRows;
  const int64_t fit = kL2Bytes / (p.total_keys * 512);      // heads' keys and values in L2
  q.head_group = static_cast<int>(fit < 1 ? 1 : (fit < p.n_heads ? fit : p.n_heads));
  const int64_t blocks = static_cast<int64_t>(q.row_tiles) * p.n_heads * p.num_seqs * 2;
  if (blocks >= (int64_t(1) << 31)) return cudaErrorInvalidConfiguration;
  expanded_pair_kernel<<<static_cast<unsigned>(blocks), kThreads, kSmem, stream>>>(q, maps);
  return cudaGetLastError();
}

}  // namespace dsa
