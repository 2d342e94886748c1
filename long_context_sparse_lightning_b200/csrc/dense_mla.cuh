// What the two dense latent attention kernels share: the work list (sequences, or a
// shared prefix and then the sequences' own parts, cut into items of N query
// rows and laid end to end by their tile counts), the walk of one unit's equal
// share of it, and small helpers.  A unit is a CTA or a CTA pair; W units form a
// gang that walks the same keys with neighbouring row tiles.
#pragma once

#include <cuda_bf16.h>

#include "kernels.cuh"
#include "ptx.cuh"

namespace dsa {
namespace dense {

constexpr int kTile = 64;                 // keys per tile
constexpr float kGrow = 24.f;             // log2 units a score may exceed its row's reference by
// An item's prologue and epilogue in tiles: ~3 us of 1.7 us in the one-CTA
// kernel, ~5 us of 0.8 us in the pair kernel.
template <int N>
constexpr int kItemCost = N == 128 ? 6 : 2;
constexpr int kMinShare = 3;              // tiles (and item costs) a gang takes at least (1, 2, 3, 4: one request of 1000
                                          // keys at 16 heads 15.2, 15.2, 14.6, 15.9 us)
constexpr float kLn2 = 0.69314718055994531f;
// Log-sum-exp (log2 units) of a piece with keys none of which has a weight for the row: of
// weight 0 like an empty piece's -inf, but written, and a NaN in it counts.
constexpr float kNoWeight = -3e38f;

struct Item {
  int32_t n_tiles;      // -1: no more items
  int32_t tile0;        // first tile (position / 64)
  int32_t row0;         // first row of the item in [total_q * H]
  int32_t rows;         // rows of the item (<= N)
  int32_t seq_row0;     // first row of the item's sequence
  int32_t base;         // position of the sequence's first query
  int32_t lo;           // first position of the item (suffix of a shared prefix)
  int32_t last;         // last position any row of the item sees
  int32_t slot;         // partial slot, -1: the item is whole
  int32_t pieces;       // pieces of the item (set where begins), 0: a sequence that is out of range
  int32_t begins;
  int32_t prefix;       // an item of the shared prefix
  int32_t b;            // sequence (block-table row), and of a flat cache its first row
  int32_t kstart;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 32 bytes to a 16-byte aligned address.
__device__ __forceinline__ void store_32(void* dst, const uint32_t* v) {
  if ((reinterpret_cast<uintptr_t>(dst) & 31u) == 0) {
    st_global_32(dst, v);
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Barrier `id` of `threads` threads; the first returns the OR of `v` over them.
__device__ __forceinline__ bool bar_any(bool v, uint32_t id, uint32_t threads) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(v ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void bar_sync(uint32_t id, uint32_t threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Non-finite bf16 values become 0 (both halves of a word).
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
  if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
  return w;
}

// True where one of the eight bf16 values is not finite (an exponent of all ones
// carries into its half's top bit).
__device__ __forceinline__ bool any_not_finite(const uint4& v) {
  const uint32_t t = ((v.x & 0x7F807F80u) + 0x00800080u) | ((v.y & 0x7F807F80u) + 0x00800080u) |
                     ((v.z & 0x7F807F80u) + 0x00800080u) | ((v.w & 0x7F807F80u) + 0x00800080u);
  return (t & 0x80008000u) != 0;
}
__device__ __forceinline__ uint4 finite_or_zero(const uint4& v) {
  return make_uint4(finite_or_zero(v.x), finite_or_zero(v.y), finite_or_zero(v.z), finite_or_zero(v.w));
}

// Entry v of the launch's work list.  With a shared prefix entry 0 is the prefix
// (every row of the batch, positions 0 .. prefix-1) and entry v > 0 the rest
// of sequence v - 1; without one entry v is sequence v.
struct Entry {
  int row0, rows;      // rows in [total_q * H]
  int q_len, kv;
  int b;               // sequence (block-table row; the prefix's positions go through sequence 0's)
  int lo;              // first position
  int gangs;           // groups of W row tiles
  int status;          // 0, or the error site
  bool prefix;
  int64_t kstart;      // flat caches: row of position 0
};

// What an entry is made of, read at once.
struct RawEntry {
  int q0, q1, kv;
  int64_t kstart;
};

__device__ __forceinline__ RawEntry read_entry(const DenseMlaParams& p, int v) {
  RawEntry w{0, 0, 0, 0};
  if (v >= p.num_seqs + p.shared) return w;
  if (p.shared && v == 0) {
    w.q1 = __ldg(&p.cu_q[p.num_seqs]);
    return w;
  }
  const int b = v - p.shared;
  w.q0 = __ldg(&p.cu_q[b]);
  w.q1 = __ldg(&p.cu_q[b + 1]);
  w.kv = __ldg(&p.kv_len[b]);
  w.kstart = seq_start(p.pt, p.kv_start, b);
  return w;
}

template <int N>
__device__ __forceinline__ Entry make_entry(const DenseMlaParams& p, int v, const RawEntry& w) {
  Entry e;
  e.status = 0;
  e.prefix = p.shared && v == 0;
  e.kstart = w.kstart;
  if (e.prefix) {
    e.b = 0;
    e.row0 = 0;
    e.q_len = min(max(w.q1, 0), p.total_q);
    e.rows = p.prefix_len > 0 ? e.q_len * p.n_heads : 0;
    e.kv = p.prefix_len;
    e.lo = 0;
  } else {
    e.b = v - p.shared;
    e.kv = w.kv;
    e.lo = p.shared ? p.prefix_len : 0;
    if (w.q0 < 0 || w.q1 < w.q0 || w.q1 > p.total_q || (e.b == 0 && w.q0 != 0)) {
      e.row0 = e.rows = e.q_len = 0;                // no rows of q: nothing is read or written
      e.status = 501;
    } else {
      e.row0 = w.q0 * p.n_heads;
      e.q_len = w.q1 - w.q0;
      e.rows = e.q_len * p.n_heads;
      if (e.q_len > e.kv || e.kv > p.max_kv_len || !seq_rows_ok(p.pt, w.kstart, e.kv, p.total_keys))
        e.status = 502;
      else if (e.q_len > 0 && e.kv - e.q_len < e.lo)
        e.status = 503;                             // the sequence does not hold the whole prefix
    }
  }
  e.gangs = e.rows <= N * p.gang ? (e.rows > 0 ? 1 : 0) : (e.rows + N * p.gang - 1) / (N * p.gang);
  return e;
}

template <int N>
__device__ __forceinline__ Entry entry_at(const DenseMlaParams& p, int v) {
  return make_entry<N>(p, v, read_entry(p, v));
}

// Last position the rows [.., row_end) of the entry see.
__device__ __forceinline__ int last_seen(const DenseMlaParams& p, const Entry& e, int row_end) {
  if (e.prefix || row_end == e.rows) return e.kv - 1;      // (divisions are left out where they can be)
  return e.kv - e.q_len + (row_end - 1) / p.n_heads;
}

// Tiles of gang g of the entry (0 for an entry that is out of range).
template <int N>
__device__ __forceinline__ int gang_tiles(const DenseMlaParams& p, const Entry& e, int g) {
  if (e.status != 0) return 0;
  const int end = min(e.rows, (g + 1) * N * p.gang);
  return last_seen(p, e, end) / kTile + 1 - e.lo / kTile;
}

template <int N>
__device__ __forceinline__ long long entry_cost(const DenseMlaParams& p, const Entry& e) {
  if (e.prefix || e.gangs <= 1 || e.status != 0)
    return e.gangs > 0 ? static_cast<long long>(e.gangs) * (gang_tiles<N>(p, e, 0) + kItemCost<N>) : 0;
  long long c = 0;
  for (int g = 0; g < e.gangs; ++g) c += gang_tiles<N>(p, e, g) + kItemCost<N>;
  return c;
}

// One gang's share [lo, hi) of the line, and where it begins.  The first `rem` of
// the gangs take per + 1 units of cost, the others per.
struct Share {
  long long per, lo, hi, start;        // start: of entry `entry` on the line
  int rem, entry, gang, gangs, member;
  Entry e;                             // entry `entry`
};

// a / b for a >= 0, b > 0 (a 64-bit division costs several hundred cycles)
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 31) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The gang whose share holds position x of the line.
__device__ __forceinline__ int gang_of(const Share& s, long long x) {
  const long long wide = s.rem * (s.per + 1);
  return static_cast<int>(x < wide ? divide(x, s.per + 1) : s.rem + divide(x - wide, s.per));
}

// Shared memory of find_share.
struct ShareScratch {
  long long scan[16];
  long long start;
  int32_t entry;
  Entry e;
};

// Called by every thread of the block (THREADS <= 512); unit of n_units.  The
// lengths are read once where the block has a thread per entry.  Entries that are
// out of range go to the error word, once per launch.
// `first` is read_entry of entry threadIdx.x, read before the block's other preparations.
template <int N, int THREADS>
__device__ __forceinline__ Share find_share(const DenseMlaParams& p, ShareScratch& sc, const RawEntry& first, int unit,
                                            int n_units) {
  constexpr int WARPS = THREADS / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n_entries = p.num_seqs + p.shared;
  // the block's running sum of `c`: this thread's start, and the sum over all
  auto scan = [&](long long c, long long& all) -> long long {
    long long inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += t;
    }
    if (lane == 31) sc.scan[warp] = inc;
    __syncthreads();
    long long before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const long long t = sc.scan[w];
      if (w < warp) before += t;
      all += t;
    }
    return before + inc - c;
  };
  auto cost_of = [&](const Entry& e) {
    if (blockIdx.x == 0 && e.status != 0) report_error(p.err, kDevErrBounds, e.status, e.b);
    return entry_cost<N>(p, e);
  };
  Entry e{};
  long long c = 0, total = 0;
  if (tid < n_entries) {
    e = make_entry<N>(p, tid, first);
    c = cost_of(e);
  }
  if (tid == 0) sc.entry = -1;
  long long start = scan(c, total);
  // more entries than threads: the others' sum (each is read again below)
  if (n_entries > THREADS) {
    long long more = 0, sum;
    for (int v = tid + THREADS; v < n_entries; v += THREADS) more += cost_of(entry_at<N>(p, v));
    __syncthreads();
    scan(more, sum);
    total += sum;
  }
  Share s;
  s.gang = p.gang == 1 ? unit : unit / p.gang;
  s.member = unit - s.gang * p.gang;
  s.gangs = static_cast<int>(min(static_cast<long long>(p.gang == 1 ? n_units : n_units / p.gang),
                                 max(1LL, (total + kMinShare - 1) / kMinShare)));
  s.per = divide(total, s.gangs);
  s.rem = static_cast<int>(total - s.per * s.gangs);
  s.lo = s.gang < s.gangs ? s.gang * s.per + min(s.gang, s.rem) : total;
  s.hi = s.gang < s.gangs ? s.lo + s.per + (s.gang < s.rem ? 1 : 0) : total;
  if (s.lo < s.hi) {
    // the entry that holds lo
    long long base = 0, all = 0;
    for (int v0 = 0;;) {
      if (c > 0 && start <= s.lo && s.lo < start + c) {
        sc.entry = v0 + tid;
        sc.start = start;
        sc.e = e;
      }
      v0 += THREADS;
      if (v0 >= n_entries) break;
      if (v0 == THREADS) {           // the first chunk's sum, from its scan
        __syncthreads();
        scan(c, all);
      }
      base += all;
      if (base > s.lo) break;        // uniform
      __syncthreads();
      c = 0;
      if (v0 + tid < n_entries) {
        e = entry_at<N>(p, v0 + tid);
        c = entry_cost<N>(p, e);
      }
      start = base + scan(c, all);
    }
  }
  __syncthreads();
  s.entry = s.lo < s.hi ? sc.entry : -1;
  s.start = s.entry >= 0 ? sc.start : 0;
  s.e = sc.e;
  return s;
}

// The pieces of a share, in order (one warp, every lane the same).
template <int N>
struct Walk {
  const DenseMlaParams& p;
  const Share sh;
  int unit, v, g = 0;
  long long at, start;                 // position on the line, start of gang g of entry v
  Entry e;

  __device__ __forceinline__ Walk(const DenseMlaParams& p_, const Share& s, int unit_)
      : p(p_), sh(s), unit(unit_), v(s.entry), at(s.lo), start(s.start), e(s.e) {}

  // The next piece; false at the end of the share.
  __device__ __forceinline__ bool next(Item& it) {
    const int n_entries = p.num_seqs + (p.shared ? 1 : 0);
    while (v >= 0 && v < n_entries && at < sh.hi) {
      const int nt = gang_tiles<N>(p, e, g);
      const long long end = start + nt + kItemCost<N>;
      if (at >= end) {                                       // gang g lies before the share's position
        start = end;
        if (++g >= e.gangs) {
          g = 0;
          do ++v;
          while (v < n_entries && (e = entry_at<N>(p, v)).gangs == 0);
        }
        continue;
      }
      const int t0 = static_cast<int>(min(at - start, static_cast<long long>(nt)));
      const int t1 = static_cast<int>(min(sh.hi - start, static_cast<long long>(nt)));
      const bool begins = at == start;
      at = min(sh.hi, end);
      if (!begins && t0 == t1) continue;                     // only the item's constant cost is left
      const int first = (g * p.gang + sh.member) * N;        // row tile of this member
      if (first >= e.rows) continue;
      it.rows = min(N, e.rows - first);
      it.row0 = e.row0 + first;
      it.seq_row0 = e.row0;
      it.base = e.kv - e.q_len;
      it.lo = e.lo;
      it.prefix = e.prefix ? 1 : 0;
      it.b = e.b;
      it.kstart = static_cast<int>(e.kstart);
      it.begins = begins ? 1 : 0;
      it.pieces = 0;
      it.last = -1;
      it.tile0 = e.lo / kTile + t0;
      it.n_tiles = 0;
      it.slot = -1;
      if (e.status == 0) {
        it.last = last_seen(p, e, first + it.rows);
        const int own = it.last / kTile + 1 - e.lo / kTile;  // this row tile may end before the gang's last
        it.n_tiles = max(0, min(t1, own) - t0);
        const long long x = start + nt;                      // one past the item's last tile
        it.pieces = begins ? gang_of(sh, x - 1) - sh.gang + 1 : 0;
        if (!begins || t1 < nt) it.slot = unit * 2 + (begins ? 1 : 0);
      }
      return true;
    }
    return false;
  }
};

// An infinite cache value whose product with q is -inf gives its key the weight 0, and 0 x
// infinity is NaN in the value's dim for every row that sees the key.  The second product shows
// that by itself but for the positions that the border's cleaning has zeroed although some
// rows of the item see them: behind the first row's last, up to the last row's.  Where the
// cleaning met such a value, the item's epilogue looks it up and overwrites the rows' outputs
// in its dim.
struct Hidden {
  int first, last;      // those positions in the item's tiles
};
__device__ __forceinline__ Hidden hidden(const Item& it, int min_lim) {
  return {max(min_lim + 1, it.tile0 * kTile), min(it.last, (it.tile0 + it.n_tiles) * kTile - 1)};
}

// NaN into the outputs (fp32 if there are any, else bf16; row n at + n * 512) of the rows that see such a
// value: row n sees positions up to base + (row + n) / heads.  Not inlined: nearly never called.
static __device__ __noinline__ void write_nan(PageTable pt, const uint16_t* kv, int b, int kstart, Hidden h, int rows,
                                              int base, int row, int heads, float* dst32, uint16_t* dst16, int t,
                                              int threads) {
  for (int d = t; d < 512; d += threads)
    for (int s = h.first; s <= h.last; ++s) {
      const int64_t at = cache_row(pt, b, kstart, s);
      if (at < 0 || (kv[at * 576 + d] & 0x7F80u) != 0x7F80u) continue;
      for (int n = max((s - base) * heads - row, 0); n < rows; ++n) {      // the rows that see position s
        if (dst32 != nullptr) {
          dst32[static_cast<int64_t>(n) * 512 + d] = __int_as_float(0x7FFFFFFF);
        } else {
          dst16[static_cast<int64_t>(n) * 512 + d] = 0x7FFFu;
        }
      }
      break;      // later positions are seen by fewer rows
    }
}

// Where row n of an item's log-sum-exp (log2 units) goes, and the item's record.
__device__ __forceinline__ void store_lse(const DenseMlaParams& p, const Item& it, int N, int n, float lse2) {
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.n_heads, r = it.row0 + n;
  const float piece = lse2 == __int_as_float(0xff800000) && it.n_tiles > 0 ? kNoWeight : lse2;
  if (it.slot >= 0) {
    p.part_lse[static_cast<int64_t>(it.slot) * N + n] = piece;
  } else if (p.shared) {
    p.row_lse[(it.prefix ? 0 : rows) + r] = piece;
  } else if (p.lse != nullptr) {
    p.lse[r] = lse2 * kLn2;
  }
  if (it.begins) p.rec[(p.shared && !it.prefix ? rows : 0) + r] = make_int4(it.slot, it.pieces, n, p.gang);
}

// fp32 destination of the item's rows (row n at + n * 512), null: the bf16 output.
__device__ __forceinline__ float* fp32_rows(const DenseMlaParams& p, const Item& it, int N) {
  if (it.slot >= 0) return p.part_o + static_cast<int64_t>(it.slot) * N * 512;
  if (p.shared) return p.row_o + (static_cast<int64_t>(it.prefix ? 0 : 1) * p.total_q * p.n_heads + it.row0) * 512;
  return nullptr;
}

}  // namespace dense
}  // namespace dsa
