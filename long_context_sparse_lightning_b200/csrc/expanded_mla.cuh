// What the two kernels of the expanded form share: the softmax of a key tile.
#pragma once

#include "dense_mla.cuh"

namespace dsa {
namespace expanded {

using dense::exp2_approx;
using dense::finite_or_zero;
using dense::kGrow;
using dense::kLn2;
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

// One key tile of a softmax warp: its 32 rows' scores (128 columns at tS, lane =
// row) become bf16 probabilities in the first 64 of those columns, relative to the
// row's reference m; l gathers their sum.  Columns behind `left` are not seen
// (masked: whether any row of the warp has such).  The reference is the first tile's
// maximum and replaced when a score exceeds it by 2^24; the outputs at tO are then
// rescaled, once o_idle() says that no product is writing them.
template <class OIdle>
__device__ __forceinline__ bool softmax_tile(uint32_t tS, uint32_t tO, float scale, int left, bool masked, bool first,
                                             float& m, float& l, OIdle o_idle) {
  const float NEG_INF = __int_as_float(0xff800000);
  uint32_t s[4][32];
#pragma unroll
  for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, s[c]);
  tmem_ld_wait();
  if (masked) {
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
    if (!first) {
      if (!o_idle()) return false;
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
  return true;
}

}  // namespace expanded
}  // namespace dsa
