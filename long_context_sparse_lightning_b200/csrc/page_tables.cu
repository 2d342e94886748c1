// Block tables, offsets, positions and cache slots of a step's new tokens from
// the requests' lengths (one launch).
//
// Two running sums over the sequences (tokens, pages taken) give every output.
// A block takes 256 sequences: it sums the lengths of the sequences before them
// (a strided read, in cache for all blocks but the first), scans its own in
// shared memory, and then walks its tokens and its new pages flat, finding
// each one's sequence by a binary search over the 257 offsets, so that one long
// prompt among decode tokens keeps all threads busy.  blockIdx.y splits the walk.
// A call moves a few hundred KB at most: it is bound by the launch and two
// dependent reads.
#include "kernels.cuh"
#include "ptx.cuh"

namespace dsa {
namespace {

constexpr int kSeqs = 256;       // sequences (and threads) per block
constexpr int kTokens = 512;     // tokens a block walks before the walk is split further (4096: 10.3 against 5 us for 33K tokens)

// x / page: a shift where the page size is a power of two
__device__ __forceinline__ int page_of(const PageTablesParams& p, int x) {
  return p.page_shift >= 0 ? x >> p.page_shift : x / p.page;
}

struct SeqPages {
  int q, before, have, need, bad;
};

__device__ __forceinline__ SeqPages seq_pages(const PageTablesParams& p, int b) {
  SeqPages s;
  s.q = __ldg(&p.q_len[b]);
  s.before = __ldg(&p.kv_before[b]);
  const long long cap = static_cast<long long>(p.blocks) * p.page;
  s.bad = s.q < 0 || s.before < 0 || static_cast<long long>(s.before) + s.q > cap;
  if (s.bad) s.q = 0;
  s.before = max(s.before, 0);
  s.have = static_cast<int>((static_cast<long long>(s.before) + p.page - 1) / p.page);
  s.need = s.bad ? 0 : static_cast<int>((static_cast<long long>(s.before) + s.q + p.page - 1) / p.page) - s.have;
  return s;
}

// Largest i in [0, n) with off[i] <= x.
__device__ __forceinline__ int find(const long long* off, int n, long long x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= x) {
      lo = mid;
    } else {
      hi = mid - 1;
    }
  }
  return lo;
}

__global__ void __launch_bounds__(kSeqs) page_tables_kernel(const PageTablesParams p) {
  __shared__ long long tok[kSeqs + 1], pg[kSeqs + 1];   // offsets of this block's sequences
  __shared__ int before_s[kSeqs], have_s[kSeqs];
  __shared__ long long red[2][kSeqs / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b0 = blockIdx.x * kSeqs, n = min(kSeqs, p.num_seqs - b0);
  // sums over the sequences before this block's
  long long t0 = 0, g0 = 0;
  for (int b = tid; b < b0; b += kSeqs) {
    const SeqPages s = seq_pages(p, b);
    t0 += s.q;
    g0 += s.need;
  }
  SeqPages s{};
  if (tid < n) s = seq_pages(p, b0 + tid);
  long long t = s.q, g = s.need;       // inclusive scans
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, t, o), c = __shfl_up_sync(0xffffffffu, g, o);
    if (lane >= o) {
      t += a;
      g += c;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    t0 += __shfl_xor_sync(0xffffffffu, t0, o);
    g0 += __shfl_xor_sync(0xffffffffu, g0, o);
  }
  __shared__ long long pre[2][kSeqs / 32];
  if (lane == 31) {
    red[0][warp] = t;
    red[1][warp] = g;
    pre[0][warp] = t0;
    pre[1][warp] = g0;
  }
  before_s[tid] = s.before;
  have_s[tid] = s.have;
  __syncthreads();
  long long tb = 0, gb = 0, tw = 0, gw = 0;
#pragma unroll
  for (int w = 0; w < kSeqs / 32; ++w) {
    tb += pre[0][w];
    gb += pre[1][w];
    if (w < warp) {
      tw += red[0][w];
      gw += red[1][w];
    }
  }
  if (tid == 0) {
    tok[0] = tb;
    pg[0] = gb;
  }
  tok[tid + 1] = tb + tw + t;
  pg[tid + 1] = gb + gw + g;
  __syncthreads();

  const long long tok_end = tok[kSeqs], pg_end = pg[kSeqs];
  const bool last = b0 + n == p.num_seqs;
  if (blockIdx.y == 0) {
    if (tid < n) {
      const int b = b0 + tid;
      p.kv_len[b] = s.before + s.q;
      p.cu_q[b + 1] = static_cast<int>(min(tok[tid + 1], static_cast<long long>(p.max_tokens)));
      if (s.bad) report_error(p.err, kDevErrBounds, 701, b);
    }
    if (b0 == 0 && tid == 0) p.cu_q[0] = 0;
    if (last && tid == 0) {
      *p.used = static_cast<int>(min(pg_end, static_cast<long long>(p.n_free)));
      if (pg_end > p.n_free) report_error(p.err, kDevErrBounds, 702, p.num_seqs);
      if (tok_end > p.max_tokens) report_error(p.err, kDevErrBounds, 703, p.num_seqs);
    }
  }
  // page taken as number x of the launch, -1 if there is none
  auto page_at = [&](long long x) -> int {
    const int id = x < p.n_free ? __ldg(&p.free_pages[x]) : -1;
    return id < 0 ? -1 : id;
  };
  // the walks: this block's part of its new pages and tokens
  const int step = kSeqs * gridDim.y, at = blockIdx.y * kSeqs + tid;
  for (long long x = pg[0] + at; x < pg_end; x += step) {
    const int i = find(pg, n, x);
    const int id = page_at(x);
    if (id < 0) report_error(p.err, kDevErrBounds, 702, b0 + i);
    p.block_table[static_cast<int64_t>(b0 + i) * p.blocks + have_s[i] + (x - pg[i])] = id;
  }
  const long long end = min(tok_end, static_cast<long long>(p.max_tokens));
  for (long long r = tok[0] + at; r < end; r += step) {
    const int i = find(tok, n, r);
    const int pos = before_s[i] + static_cast<int>(r - tok[i]);
    const int blk = page_of(p, pos);
    // an entry held before the call, or one that this call takes (no other block's write is read)
    const int id = blk < have_s[i] ? p.block_table[static_cast<int64_t>(b0 + i) * p.blocks + blk]
                                   : page_at(pg[i] + blk - have_s[i]);
    if (id < 0) report_error(p.err, kDevErrBounds, 704, b0 + i);
    p.pos[r] = pos;
    p.slots[r] = id < 0 ? -1 : static_cast<int64_t>(id) * p.page + (pos - blk * p.page);
  }
  if (last) {
    for (long long r = end + at; r < p.max_tokens; r += step) {
      p.pos[r] = 0;
      p.slots[r] = -1;
    }
  }
}

}  // namespace

cudaError_t launch_page_tables(const PageTablesParams& p, cudaStream_t stream) {
  const int nx = (p.num_seqs + kSeqs - 1) / kSeqs;
  // the walk over max_tokens, split while there are at most two blocks per SM
  int ny = (p.max_tokens + kTokens - 1) / kTokens;
  const int most = nx < 2 * sm_count() ? 2 * sm_count() / nx : 1;
  ny = ny < 1 ? 1 : (ny > most ? most : ny);
  page_tables_kernel<<<dim3(nx, ny), kSeqs, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
