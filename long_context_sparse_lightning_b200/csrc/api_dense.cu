// C ABI of the dense latent attentions and of the page tables: argument checks,
// workspace carving, TMA descriptors and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/dsa.h"
#include "kernels.cuh"

namespace {

constexpr size_t kHeader = 256;      // device error word + reserved

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Workspace behind the header: item records, partial slots, with a shared
// prefix the rows' whole results.
struct DenseLayout {
  size_t rec, part_lse, part_o, row_lse, row_o, bytes;
};

DenseLayout dense_layout(const dsa_batch_t* b, int n_heads, bool shared) {
  const dsa::DensePlan d = dsa::dense_plan(b, n_heads, shared);
  const size_t rows = static_cast<size_t>(b->total_q) * n_heads, halves = shared ? 2 : 1;
  const size_t slots = static_cast<size_t>(dsa::dense_slots(d.n)) * d.n;
  DenseLayout l;
  l.rec = kHeader;
  l.part_lse = l.rec + round_up(halves * rows * sizeof(int4), 256);
  l.part_o = l.part_lse + round_up(slots * sizeof(float), 256);
  l.row_lse = l.part_o + slots * 512 * sizeof(float);
  l.row_o = l.row_lse + (shared ? round_up(2 * rows * sizeof(float), 256) : 0);
  l.bytes = l.row_o + (shared ? 2 * rows * 512 * sizeof(float) : 0);
  return l;
}

// The same of the expanded form: partial results where the keys are split.
struct ExpandedLayout {
  int splits;
  size_t part_lse, part_o, bytes;
};

ExpandedLayout expanded_layout(int splits, int64_t total_q, int n_heads) {
  ExpandedLayout l;
  l.splits = splits;
  const size_t rows = splits > 1 ? static_cast<size_t>(splits) * static_cast<size_t>(total_q) * n_heads : 0;
  l.part_lse = kHeader;
  l.part_o = l.part_lse + round_up(rows * sizeof(float), 256);
  l.bytes = l.part_o + rows * 128 * sizeof(float);
  return l;
}

dsa_status_t run_dense(const dsa_batch_t* b, int prefix_len, const void* q, int n_heads, const void* kv, float sm_scale,
                       void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const bool shared = prefix_len >= 0;
  const dsa_status_t s = dsa::validate_batch(b);
  if (s != DSA_OK) return s;
  // a step without tokens may come with empty tensors
  if (b->total_q > 0 && (q == nullptr || kv == nullptr || out == nullptr)) return DSA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(kv, 16) || misaligned(out, 16) || misaligned(lse, 4)) return DSA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
  if (n_heads < 1 || n_heads > 128) return DSA_ERR_UNSUPPORTED;
  if (shared && b->block_table == nullptr) return DSA_ERR_UNSUPPORTED;
  if (shared && prefix_len > b->max_kv_len) return DSA_ERR_INVALID_ARG;
  if (ws == nullptr || misaligned(ws, 16)) return DSA_ERR_INVALID_ARG;
  const DenseLayout l = dense_layout(b, n_heads, shared);
  if (ws_bytes < l.bytes) return DSA_ERR_WORKSPACE;
  if (b->total_q == 0) return DSA_OK;
  const dsa::DensePlan d = dsa::dense_plan(b, n_heads, shared);
  uint8_t* base = static_cast<uint8_t*>(ws);
  dsa::DenseMlaParams p;
  p.cu_q = b->cu_q;
  p.kv_len = b->kv_len;
  p.kv_start = b->kv_start;
  p.pt = dsa::batch_pages(b);
  p.total_keys = b->total_keys;
  p.total_q = b->total_q;
  p.num_seqs = b->num_seqs;
  p.max_kv_len = b->max_kv_len;
  p.n_heads = n_heads;
  p.gang = d.gang;
  p.shared = shared ? 1 : 0;
  p.prefix_len = shared ? prefix_len : 0;
  p.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  p.kv = static_cast<const uint16_t*>(kv);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.rec = reinterpret_cast<int4*>(base + l.rec);
  p.part_lse = reinterpret_cast<float*>(base + l.part_lse);
  p.part_o = reinterpret_cast<float*>(base + l.part_o);
  p.row_lse = reinterpret_cast<float*>(base + l.row_lse);
  p.row_o = reinterpret_cast<float*>(base + l.row_o);
  p.err = reinterpret_cast<uint32_t*>(base);
  p.budget = dsa::wait_budget();
  p.skip_arrival = dsa::test_skip_arrival();
  const bool pair = d.n == 128;
  const uint64_t rows = static_cast<uint64_t>(b->total_q) * n_heads, keys = static_cast<uint64_t>(b->total_keys);
  dsa::DenseMaps maps;
  if (!dsa::make_tmap_blocks(&maps.q, q, rows, 9, 576, pair ? 64 : d.n, 9) ||
      !dsa::make_tmap_blocks(&maps.c, kv, keys, 9, 576, pair ? 32 : 64, pair ? 9 : 2) ||
      !dsa::make_tmap_blocks(&maps.v, kv, keys, 9, 576, pair ? 32 : 64, pair ? 4 : 1))
    return DSA_ERR_CUDA;
  return dsa::launch_dense_mla(p, d, maps, stream) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

namespace dsa {
size_t dense_ws_bytes(const dsa_batch_t* b, int n_heads, bool shared) {
  if (n_heads < 1 || n_heads > 128) return 0;
  if (shared && b->block_table == nullptr) return 0;
  return dense_layout(b, n_heads, shared).bytes;
}

size_t expanded_ws_bytes(const dsa_batch_t* b, int n_heads) {
  if (n_heads < 1 || n_heads > 128 || b->block_table != nullptr) return 0;
  // enough for every batch within this one's bounds: those of fewer rows are split into more parts
  size_t most = kHeader;
  for (int s = 2; s <= dsa::expanded_most_splits(b->max_kv_len, n_heads); ++s) {
    const int64_t fit = dsa::kExpandedPartRows / (s * n_heads);
    const size_t bytes = expanded_layout(s, b->total_q < fit ? b->total_q : fit, n_heads).bytes;
    if (bytes > most) most = bytes;
  }
  return most;
}
}  // namespace dsa

extern "C" {

dsa_status_t dsa_dense_mla(const dsa_batch_t* batch, const void* q, int32_t n_heads, const void* kv, float sm_scale,
                           void* out, float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  return run_dense(batch, -1, q, n_heads, kv, sm_scale, out, lse, ws, ws_bytes, reinterpret_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_prefix_mla(const dsa_batch_t* batch, int32_t prefix_len, const void* q, int32_t n_heads, const void* kv,
                            float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  if (prefix_len < 0) return DSA_ERR_INVALID_ARG;
  return run_dense(batch, prefix_len, q, n_heads, kv, sm_scale, out, lse, ws, ws_bytes,
                   reinterpret_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_expanded_mla(const dsa_batch_t* b, const void* q, int32_t n_heads, const void* kv_up, const void* rope,
                              int64_t rope_stride, float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                              dsa_stream_t stream) {
  const dsa_status_t s = dsa::validate_batch(b);
  if (s != DSA_OK) return s;
  if (b->total_q > 0 && (q == nullptr || kv_up == nullptr || rope == nullptr || out == nullptr)) return DSA_ERR_INVALID_ARG;
  if (misaligned(q, 16) || misaligned(kv_up, 16) || misaligned(rope, 16) || misaligned(out, 16) || misaligned(lse, 4))
    return DSA_ERR_INVALID_ARG;
  if (rope_stride < 64 || rope_stride % 8 != 0 || rope_stride >= (int64_t(1) << 31)) return DSA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !std::isfinite(sm_scale)) return DSA_ERR_INVALID_ARG;
  if (n_heads < 1 || n_heads > 128 || b->block_table != nullptr) return DSA_ERR_UNSUPPORTED;
  if (ws == nullptr || misaligned(ws, 16)) return DSA_ERR_INVALID_ARG;
  const ExpandedLayout l = expanded_layout(dsa::expanded_splits(b, n_heads), b->total_q, n_heads);
  if (ws_bytes < l.bytes) return DSA_ERR_WORKSPACE;
  if (b->total_q == 0) return DSA_OK;
  dsa::ExpandedMlaParams p;
  p.max_q = b->max_q_per_seq;
  p.splits = l.splits;
  p.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.part_lse);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + l.part_o);
  p.cu_q = b->cu_q;
  p.kv_len = b->kv_len;
  p.kv_start = b->kv_start;
  p.total_keys = b->total_keys;
  p.total_q = b->total_q;
  p.num_seqs = b->num_seqs;
  p.max_kv_len = b->max_kv_len;
  p.n_heads = n_heads;
  p.scale_log2 = static_cast<float>(static_cast<double>(sm_scale) * 1.4426950408889634);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.err = static_cast<uint32_t*>(ws);
  p.budget = dsa::wait_budget();
  p.skip_arrival = dsa::test_skip_arrival();
  const uint64_t h = static_cast<uint64_t>(n_heads);
  CUtensorMap map_q, map_kv, map_r;
  if (!dsa::make_tmap_blocks(&map_q, q, static_cast<uint64_t>(b->total_q), h * 3, h * 192, 128, 3) ||
      !dsa::make_tmap_blocks(&map_kv, kv_up, static_cast<uint64_t>(b->total_keys), h * 4, h * 256, 128, 1) ||
      !dsa::make_tmap_blocks(&map_r, rope, static_cast<uint64_t>(b->total_keys), 1, static_cast<uint64_t>(rope_stride),
                             128, 1))
    return DSA_ERR_CUDA;
  return dsa::launch_expanded_mla(p, map_q, map_kv, map_r, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? DSA_OK
             : DSA_ERR_CUDA;
}

dsa_status_t dsa_page_tables(int32_t num_seqs, const int32_t* q_len, const int32_t* kv_before,
                             const int32_t* free_pages, int32_t n_free, int32_t page_size, int32_t* block_table,
                             int32_t blocks_per_seq, int32_t max_tokens, int32_t* cu_q, int32_t* kv_len, int32_t* pos,
                             int64_t* slots, int32_t* pages_used, void* ws, size_t ws_bytes, dsa_stream_t stream) {
  if (num_seqs < 1 || num_seqs > 65535 || n_free < 0 || max_tokens < 0) return DSA_ERR_INVALID_ARG;
  if (page_size < 64 || page_size % 64 != 0 || blocks_per_seq < 1) return DSA_ERR_INVALID_ARG;
  if (q_len == nullptr || kv_before == nullptr || block_table == nullptr || cu_q == nullptr || kv_len == nullptr ||
      pages_used == nullptr || (free_pages == nullptr && n_free > 0) ||
      ((pos == nullptr || slots == nullptr) && max_tokens > 0))
    return DSA_ERR_INVALID_ARG;
  // positions and pool rows are int32 in a batch
  if (static_cast<int64_t>(blocks_per_seq) * page_size >= (int64_t(1) << 31)) return DSA_ERR_UNSUPPORTED;
  struct Range {
    const void* at;
    size_t bytes;
    uintptr_t align;
  };
  const size_t n = static_cast<size_t>(num_seqs), tokens = static_cast<size_t>(max_tokens);
  const Range in[] = {{q_len, n * 4, 4}, {kv_before, n * 4, 4}, {free_pages, static_cast<size_t>(n_free) * 4, 4}};
  const Range out[] = {{block_table, n * static_cast<size_t>(blocks_per_seq) * 4, 4},
                       {cu_q, (n + 1) * 4, 4},
                       {kv_len, n * 4, 4},
                       {pos, tokens * 4, 4},
                       {slots, tokens * 8, 8},
                       {pages_used, 4, 4}};
  auto overlap = [](const Range& a, const Range& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
  };
  for (const Range& a : in)
    if (misaligned(a.at, a.align)) return DSA_ERR_INVALID_ARG;
  for (const Range& a : out) {
    if (misaligned(a.at, a.align)) return DSA_ERR_INVALID_ARG;
    for (const Range& b : in)
      if (overlap(a, b)) return DSA_ERR_INVALID_ARG;
    for (const Range& b : out)
      if (&a != &b && overlap(a, b)) return DSA_ERR_INVALID_ARG;
  }
  if (ws == nullptr || misaligned(ws, 16)) return DSA_ERR_INVALID_ARG;
  if (ws_bytes < kHeader) return DSA_ERR_WORKSPACE;
  dsa::PageTablesParams p;
  p.q_len = q_len;
  p.kv_before = kv_before;
  p.free_pages = free_pages;
  p.block_table = block_table;
  p.cu_q = cu_q;
  p.kv_len = kv_len;
  p.pos = pos;
  p.slots = slots;
  p.used = pages_used;
  p.num_seqs = num_seqs;
  p.page = page_size;
  if ((page_size & (page_size - 1)) == 0)
    for (p.page_shift = 0; (1 << p.page_shift) < page_size;) ++p.page_shift;
  p.blocks = blocks_per_seq;
  p.n_free = n_free;
  p.max_tokens = max_tokens;
  p.err = static_cast<uint32_t*>(ws);
  return dsa::launch_page_tables(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // extern "C"
