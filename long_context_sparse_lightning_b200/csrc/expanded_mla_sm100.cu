// Latent attention in the expanded form on sm_100a: per head h
//     o[i, h] = sum_{s <= t_i} softmax_s(sm_scale * (qn.kn[s, h] + qr.kr[s])) * v[s, h]
// with 128-d keys kn and values v of each head (made from the latent rows by
// the caller's up-projection) and the 64 RoPE dims kr that all heads share:
// 640 multiply-adds per head and pair against the absorbed form's 1088.
//
// A CTA owns two tiles of 128 query rows of one head (lane = row) and walks
// the keys up to its last row's position in tiles of 128.  Tensor memory: the two
// tiles' scores (128 columns each) and outputs (128 each), all 512 columns; a tile's
// probabilities overwrite its scores as bf16 and are the A operand of the
// second product from there.  The MMA thread alternates: while the softmax
// warps of one tile work on its scores, the tensor cores run the other tile's
// second product and next scores.
//
// Per key tile the tensor cores need 2 x 128 x 128 x (192 + 128) multiply-adds
// (2560 cycles at full rate) and the 2 x 128 x 128 exponentials take 2048 at
// 16 per cycle, so both units have to be kept busy at once.
//
// Roles: warp 0 TMA, warp 1 MMAs, warps 2-3 clean the value tiles on the border
// (below), warps 4-7 and 8-11 softmax and epilogue of the two tiles.
//
// A position that some row of the CTA must not see has probability 0 there,
// and 0 x a non-finite value would reach that row all the same.  So in tiles on
// the border the cleaning warps zero the value rows that no row of the CTA
// sees, and for a non-finite value at a position that only later rows see they
// zero it and note the first such position per dim: rows that do see it get NaN.
#include <cuda_bf16.h>

#include "kernels.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kRows = 128;                 // query rows per tile (TMEM lanes)
constexpr int kKeys = 128;                 // keys per tile
constexpr int kBlk = 128 * 128;            // one [128 rows x 64 dims] block, 128-byte swizzle
constexpr int kSlots = 8;                  // key / value blocks in flight: 3 + 2 per tile
constexpr int kThreads = 12 * 32;
constexpr uint32_t kRegLow = 88, kRegHigh = 208;     // 128 * (88 + 2 * 208) = 384 * 168
constexpr float kGrow = 24.f;              // log2 units a score may exceed its row's reference by
constexpr float kLn2 = 0.69314718055994531f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_S = 0, TM_O = 256;   // + 128 * tile

constexpr int OFF_Q = 0;                               // 2 tiles x 3 blocks
constexpr int OFF_KV = 6 * kBlk;
constexpr int OFF_AUX = OFF_KV + kSlots * kBlk;
constexpr int kSmem = OFF_AUX + 1024 + 1024;
static_assert(kSmem <= 232448, "shared memory of one CTA");

struct Aux {
  uint64_t q_full[2];
  uint64_t full[kSlots], empty[kSlots];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t go, clean;       // border tiles: the values have landed / are clean
  uint32_t tmem;
  int32_t bad_pos[128];     // first position whose value of this dim is not finite, per dim
};
static_assert(sizeof(Aux) <= 1024, "");

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// What a CTA works on.
struct Tile {
  int row0, rows;          // rows of q
  int base;                // position of row 0
  int n[2];                // key tiles of the two row tiles (0: no rows)
  int first_row_key;       // cache row of position 0
  bool bad;
};

__global__ void __launch_bounds__(kThreads, 1)
    expanded_mla_kernel(const ExpandedMlaParams p, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_kv, const __grid_constant__ CUtensorMap map_r) {
  const int b = blockIdx.z, h = blockIdx.y;
  const int qt = static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x);     // the longest rows first
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
  w.bad = q_len > kv || kv > p.max_kv_len || ks < 0 || ks + kv > p.total_keys;
  w.row0 = q0 + qt * 2 * kRows;
  w.rows = min(2 * kRows, q_len - qt * 2 * kRows);
  w.base = kv - q_len + qt * 2 * kRows;
  w.n[0] = (w.base + min(w.rows, kRows) - 1) / kKeys + 1;
  w.n[1] = w.rows > kRows ? (w.base + w.rows - 1) / kKeys + 1 : 0;
  w.first_row_key = static_cast<int>(ks);
  const int H = p.n_heads, tid = threadIdx.x;
  if (w.bad) {
    if (qt == 0 && h == 0 && tid == 0) report_error(p.err, kDevErrBounds, 602, b);
    for (int u = tid; u < w.rows * 16; u += kThreads)
      *reinterpret_cast<uint4*>(p.out + (static_cast<int64_t>(w.row0 + (u >> 4)) * H + h) * 128 + (u & 15) * 8) =
          make_uint4(0, 0, 0, 0);
    if (p.lse != nullptr)
      for (int r = tid; r < w.rows; r += kThreads)
        p.lse[static_cast<int64_t>(w.row0 + r) * H + h] = __int_as_float(0xff800000);
    return;
  }
  const int n_tiles = max(w.n[0], w.n[1]);
  const bool two = w.n[1] > 0;
  const int border0 = (w.base + 1) / kKeys;      // first tile with a position that row 0 must not see

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
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&ax->full[i], 1);
      mbar_init(&ax->empty[i], 1);
    }
    mbar_init(&ax->go, 1);
    mbar_init(&ax->clean, 2);
    fence_mbar_init();
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_kv);
    prefetch_tmap(&map_r);
  }
  if (tid < 128) ax->bad_pos[tid] = 0x7fffffff;
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
        int n = 0;
        auto load = [&](const CUtensorMap* m, int block, int y) {
          const int s = n % kSlots;
          if (ok && n >= kSlots && !mbar_wait(&ax->empty[s], ((n / kSlots) + 1) & 1, p.budget)) {
            report_error(p.err, kDevErrTimeout, 611, blockIdx.x);
            ok = false;
          }
          if (!ok) return;
          mbar_arrive_expect_tx(&ax->full[s], kBlk);
          tma_load_3d(sm + OFF_KV + s * kBlk, m, &ax->full[s], 0, y, block);
          ++n;
        };
        for (int a = 0; a < (two ? 2 : 1); ++a) {
          mbar_arrive_expect_tx(&ax->q_full[a], 3 * kBlk);
          tma_load_3d(sm + OFF_Q + 3 * a * kBlk, &map_q, &ax->q_full[a], 0, w.row0 + a * kRows, h * 3);
          if (a == 0) {
            load(&map_kv, h * 4, w.first_row_key);
            load(&map_kv, h * 4 + 1, w.first_row_key);
            load(&map_r, 0, w.first_row_key);
          }
        }
        for (int i = 0; ok && i < n_tiles; ++i) {
          const int y = w.first_row_key + i * kKeys;
          if (i > 0) {
            load(&map_kv, h * 4, y);
            load(&map_kv, h * 4 + 1, y);
            load(&map_r, 0, y);
          }
          load(&map_kv, h * 4 + 2, y);
          load(&map_kv, h * 4 + 3, y);
        }
        if (!ok) {      // let the copies in flight land before the block ends
          bool landed = true;
          for (int a = 0; a < (two ? 2 : 1); ++a) landed = landed && mbar_wait(&ax->q_full[a], 0, p.budget);
          for (int i = max(0, n - kSlots); landed && i < n; ++i)
            landed = mbar_wait(&ax->full[i % kSlots], (i / kSlots) & 1, p.budget);
        }
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMAs --
      if (elect_one()) {
        constexpr uint32_t idesc_s = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 128, 0, 0);
        constexpr uint32_t idesc_o = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 128, 0, 1);     // V MN-major
        const uint32_t q_addr = smem_u32(sm + OFF_Q), kv_addr = smem_u32(sm + OFF_KV);
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
          if (ok && !mbar_wait(bar, parity, p.budget)) {
            report_error(p.err, kDevErrTimeout, site, blockIdx.x);
            ok = false;
          }
          return ok;
        };
        auto scores = [&](int a, int i) {
          const bool last = a == 1 || !two;        // of the row tiles that read key tile i
          for (int c = 0; c < 3; ++c) {
            const int n = 5 * i + c, s = n % kSlots;
            if (!wait(&ax->full[s], (n / kSlots) & 1, 621)) return;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_f16_ss(tmem + TM_S + 128 * a, smem_desc(q_addr + (3 * a + c) * kBlk + kk * 32, 16, 1024, kSwizzle128B),
                          smem_desc(kv_addr + s * kBlk + kk * 32, 16, 1024, kSwizzle128B), idesc_s, (c | kk) ? 1u : 0u);
            if (last) umma_commit(&ax->empty[s]);
          }
          umma_commit(&ax->s_full[a]);
          if (last && i >= border0) {
            for (int c = 0; c < 2; ++c) {
              const int n = 5 * i + 3 + c;
              if (!wait(&ax->full[n % kSlots], (n / kSlots) & 1, 625)) return;
            }
            mbar_arrive(&ax->go);
          }
        };
        auto values = [&](int a, int i) {
          const bool last = a == 1 || !two;
          if (!wait(&ax->p_full[a], i & 1, 622)) return;
          if (i >= border0 && !wait(&ax->clean, (i - border0) & 1, 623)) return;
          for (int c = 0; c < 2; ++c) {
            const int n = 5 * i + 3 + c;
            if (!wait(&ax->full[n % kSlots], (n / kSlots) & 1, 624)) return;
          }
          tc_fence_after();
          // one instruction spans both 64-dim blocks where the ring keeps them side by side, else two
          const int n0 = (5 * i + 3) % kSlots, n1 = (5 * i + 4) % kSlots;
          const uint32_t step = static_cast<uint32_t>((n1 - n0) * kBlk);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t acc = (i | kk) ? 1u : 0u;
            if (n1 > n0) {
              umma_f16_ts(tmem + TM_O + 128 * a, tmem + TM_S + 128 * a + kk * 8,
                          smem_desc(kv_addr + n0 * kBlk + kk * 2048, step, 1024, kSwizzle128B), idesc_o, acc);
            } else {
              constexpr uint32_t idesc_half = idesc_f32acc(kFmtBF16, kFmtBF16, 128, 64, 0, 1);
              umma_f16_ts(tmem + TM_O + 128 * a, tmem + TM_S + 128 * a + kk * 8,
                          smem_desc(kv_addr + n0 * kBlk + kk * 2048, kBlk, 1024, kSwizzle128B), idesc_half, acc);
              umma_f16_ts(tmem + TM_O + 128 * a + 64, tmem + TM_S + 128 * a + kk * 8,
                          smem_desc(kv_addr + n1 * kBlk + kk * 2048, kBlk, 1024, kSwizzle128B), idesc_half, acc);
            }
          }
          if (last) {
            umma_commit(&ax->empty[n0]);
            umma_commit(&ax->empty[n1]);
          }
          umma_commit(&ax->o_done[a]);
        };
        wait(&ax->q_full[0], 0, 620);
        if (ok) scores(0, 0);
        if (ok && two && wait(&ax->q_full[1], 0, 620)) scores(1, 0);
        for (int i = 0; ok && i < n_tiles; ++i) {
          if (i < w.n[0]) values(0, i);
          if (ok && i + 1 < w.n[0]) scores(0, i + 1);
          if (ok && i < w.n[1]) values(1, i);
          if (ok && i + 1 < w.n[1]) scores(1, i + 1);
        }
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
      for (int i = border0; ok && i < n_tiles; ++i) {
        // The MMA thread, which follows every phase of the ring, tells when: these
        // warps skip the tiles before, and a parity alone would not tell them.
        wait(&ax->go, (i - border0) & 1);
        for (int c = 0; ok && c < 2; ++c) {
          const int n = 5 * i + 3 + c, s = n % kSlots;
          wait(&ax->full[s], (n / kSlots) & 1);
          if (!ok) break;
          // row r of the block is position i * 128 + r; unit u of it holds dims 8 (u ^ (r & 7)) ..
          for (int u = tid - 64; u < kBlk / 16; u += 64) {
            const int r = u >> 3, pos = i * kKeys + r;
            if (pos <= w.base) continue;                       // every row sees it
            uint4* at = reinterpret_cast<uint4*>(sm + OFF_KV + s * kBlk) + u;
            if (pos > w.base + w.rows - 1) {                   // no row sees it
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            const uint4 v = *at;
            uint32_t x[4] = {v.x, v.y, v.z, v.w};
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t mask = 0x7F80u << (16 * (e & 1));
              if ((x[e >> 1] & mask) == mask) {
                x[e >> 1] &= 0xFFFFu << (16 * ((e & 1) ^ 1));
                atomicMin(&ax->bad_pos[c * 64 + 8 * ((u & 7) ^ (r & 7)) + e], pos);
                hit = true;
              }
            }
            if (hit) *at = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ax->clean);
      }
    }
  } else {
    setmaxnreg_inc<kRegHigh>();
    // ----------------------------------------------------- softmax, epilogue --
    const int a = static_cast<int>(warp >> 2) - 1;
    const uint32_t quarter = warp & 3u;
    const int r = a * kRows + static_cast<int>(quarter * 32 + lane);     // row of the CTA
    const uint32_t t_lane = tmem + ((quarter * 32u) << 16);
    const uint32_t tS = t_lane + TM_S + 128 * a, tO = t_lane + TM_O + 128 * a;
    const float scale = p.scale_log2, NEG_INF = __int_as_float(0xff800000);
    // rows behind the last one follow it (their results are not stored)
    const int lim = w.base + min(r, w.rows - 1);
    const int warp_lim = w.base + min(a * kRows + static_cast<int>(quarter * 32), w.rows - 1);
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
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
        for (int j = 1; j < 32; ++j) mx[c] = fmaxf(mx[c], __uint_as_float(s[c][j]));
      }
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
      const bool grow = top > m + kGrow;         // true on the first tile that shows the row a key
      if (__any_sync(0xffffffffu, grow)) {
        const float f = grow ? exp2_approx(m - top) : 1.f;
        if (grow) m = top;
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
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const float x = exp2_approx(fmaf(__uint_as_float(s[c][2 * j]), scale, ref));
          const float y = exp2_approx(fmaf(__uint_as_float(s[c][2 * j + 1]), scale, ref));
          sum += x + y;
          pk[j] = pack_bf16(x, y);
        }
        l += sum;
        tmem_st16(tS + 16 * c, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ax->p_full[a]);
    }
    if (ok && nt > 0 && wait(&ax->o_done[a], (nt - 1) & 1, 643)) {
      tc_fence_after();
      const float inv = 1.f / l;
      const int64_t at = static_cast<int64_t>(w.row0 + r) * H + h;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * c, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (ax->bad_pos[32 * c + j] <= lim) o[j] = 0x7FFFFFFFu;
        if (r < w.rows) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint4 v;
            v.x = pack_bf16(__uint_as_float(o[8 * u]) * inv, __uint_as_float(o[8 * u + 1]) * inv);
            v.y = pack_bf16(__uint_as_float(o[8 * u + 2]) * inv, __uint_as_float(o[8 * u + 3]) * inv);
            v.z = pack_bf16(__uint_as_float(o[8 * u + 4]) * inv, __uint_as_float(o[8 * u + 5]) * inv);
            v.w = pack_bf16(__uint_as_float(o[8 * u + 6]) * inv, __uint_as_float(o[8 * u + 7]) * inv);
            *reinterpret_cast<uint4*>(p.out + at * 128 + 32 * c + 8 * u) = v;
          }
        }
      }
      if (r < w.rows && p.lse != nullptr) p.lse[at] = (m + log2f(l)) * kLn2;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_expanded_mla(const ExpandedMlaParams& p, int max_q_per_seq, const CUtensorMap& map_q,
                                const CUtensorMap& map_kv, const CUtensorMap& map_r, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(expanded_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((max_q_per_seq + 2 * kRows - 1) / (2 * kRows), p.n_heads, p.num_seqs);
  expanded_mla_kernel<<<grid, kThreads, kSmem, stream>>>(p, map_q, map_kv, map_r);
  return cudaGetLastError();
}

}  // namespace dsa
