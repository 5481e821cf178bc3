// api_step.cu -- the C ABI of a step's rotary positions and of the cache's pages
// (include/mla_decode.h): argument checks, the rotary plan, launches.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "internal.h"
#include "mla_decode.h"

namespace {

constexpr int32_t kRopeCols = 64;
constexpr int32_t kRank = 512;
constexpr int32_t kHeadDim = 576;
constexpr double kTwoPi = 6.283185307179586476925;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

mla_status_t cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return MLA_OK;
  mla::record_cuda_error(e);
  return MLA_ERR_CUDA;
}

mla_status_t check_rope(const mla_rope_problem_t& p) {
  if (p.dim < 2 || p.dim > kRopeCols || p.dim % 2 != 0) return MLA_ERR_INVALID_ARG;
  if (p.layout != MLA_ROPE_INTERLEAVED && p.layout != MLA_ROPE_HALF) return MLA_ERR_INVALID_ARG;
  if (p.scaling < MLA_ROPE_SCALING_NONE || p.scaling > MLA_ROPE_SCALING_YARN) return MLA_ERR_INVALID_ARG;
  if (!std::isfinite(p.base) || !(p.base > 1.0)) return MLA_ERR_INVALID_ARG;
  if (p.scaling == MLA_ROPE_SCALING_NONE) return MLA_OK;
  if (!std::isfinite(p.factor) || !(p.factor > 0.0)) return MLA_ERR_INVALID_ARG;
  if (p.scaling == MLA_ROPE_SCALING_LINEAR) return MLA_OK;
  if (p.original_max_position <= 0 || !std::isfinite(p.beta_fast) || !std::isfinite(p.beta_slow) ||
      !(p.beta_fast > 0.0) || !(p.beta_slow > 0.0) || !(p.beta_fast >= p.beta_slow) || !std::isfinite(p.mscale) ||
      !std::isfinite(p.mscale_all_dim) || p.mscale < 0.0 || p.mscale_all_dim < 0.0)
    return MLA_ERR_INVALID_ARG;
  return MLA_OK;
}

// Growth of the attention's temperature with the stretch of the context.
double stretch_scale(double factor, double m) { return factor <= 1.0 ? 1.0 : 0.1 * m * std::log(factor) + 1.0; }

// The cache's blocks as the copies see them.
mla_status_t check_pages(void* kv_cache, float* kv_scales, int32_t num_blocks, int32_t block_size, int32_t kv_dtype,
                         int32_t scale_group, mla::PageCopy* c) {
  if (num_blocks <= 0 || block_size <= 0 || scale_group < 0) return MLA_ERR_INVALID_ARG;
  if (kv_dtype != MLA_DTYPE_BF16 && kv_dtype != MLA_DTYPE_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(num_blocks) * block_size > INT32_MAX) return MLA_ERR_UNSUPPORTED;
  if (kv_cache == nullptr || !aligned(kv_cache, 16)) return MLA_ERR_INVALID_ARG;
  if ((scale_group > 0) != (kv_scales != nullptr)) return MLA_ERR_INVALID_ARG;
  if (scale_group > 0 && (kv_dtype != MLA_DTYPE_FP8_E4M3 || block_size % scale_group != 0 || !aligned(kv_scales, 4)))
    return MLA_ERR_INVALID_ARG;
  const int64_t units = static_cast<int64_t>(block_size) * kHeadDim * (kv_dtype == MLA_DTYPE_BF16 ? 2 : 1) / 16;
  if (units > INT32_MAX / 4) return MLA_ERR_UNSUPPORTED;
  c->cache = kv_cache;
  c->num_blocks = num_blocks;
  c->block_units = static_cast<int32_t>(units);
  c->scales = kv_scales;
  c->block_scales = scale_group > 0 ? block_size / scale_group : 0;
  return MLA_OK;
}

// Workspace of the page lists: a ticket and two counts, the bitmap of freed blocks, the
// lists of a compaction.
struct PageLayout {
  size_t bitmap, holes, from, back, end;
};
PageLayout page_layout(int32_t num_blocks) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t n = static_cast<size_t>(num_blocks);
  PageLayout l;
  l.bitmap = 256;
  l.holes = l.bitmap + up((n + 31) / 32 * 4);
  l.from = l.holes + up((n / 2 + 1) * 4);
  l.back = l.from + up((n / 2 + 1) * 4);
  l.end = l.back + up(n * 4);
  return l;
}

}  // namespace

extern "C" {

mla_status_t mla_rope_plan(const mla_rope_problem_t* prob, mla_rope_t* rope) {
  if (prob == nullptr || rope == nullptr) return MLA_ERR_INVALID_ARG;
  const mla_rope_problem_t p = *prob;
  const mla_status_t s = check_rope(p);
  if (s != MLA_OK) return s;
  std::memset(rope, 0, sizeof(*rope));
  rope->prob = p;
  rope->mscale = 1.f;
  const double d = p.dim;
  double low = 0.0, high = 0.0;
  if (p.scaling == MLA_ROPE_SCALING_YARN) {
    // the pair that makes `beta` turns over the original context
    auto pair_of = [&](double beta) {
      return d * std::log(p.original_max_position / (beta * kTwoPi)) / (2.0 * std::log(p.base));
    };
    low = std::fmax(std::floor(pair_of(p.beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_of(p.beta_slow)), d - 1.0);
    rope->mscale = static_cast<float>(stretch_scale(p.factor, p.mscale) / stretch_scale(p.factor, p.mscale_all_dim));
  }
  for (int i = 0; i < p.dim / 2; ++i) {
    double f = std::pow(p.base, -2.0 * i / d);
    if (p.scaling == MLA_ROPE_SCALING_LINEAR) {
      f /= p.factor;
    } else if (p.scaling == MLA_ROPE_SCALING_YARN) {
      const double span = high == low ? 0.001 : high - low;
      const double ramp = std::fmin(std::fmax((i - low) / span, 0.0), 1.0);
      f = f / p.factor * ramp + f * (1.0 - ramp);
    }
    rope->turns[i] = f / kTwoPi;
  }
  return MLA_OK;
}

mla_status_t mla_rope_qk(const mla_rope_t* rope, const int32_t* positions, int32_t num_tokens, int32_t num_heads,
                         const void* ql_nope, int64_t nope_stride_t, int64_t nope_stride_h, const void* q_pe,
                         int64_t pe_stride_t, int64_t pe_stride_h, int32_t out_dtype, float q_scale, void* q_out,
                         const void* k_pe, int64_t k_pe_stride, void* k_out, int64_t k_out_stride,
                         cudaStream_t stream) {
  if (rope == nullptr || num_tokens < 0 || num_heads < 0) return MLA_ERR_INVALID_ARG;
  const mla_status_t s = check_rope(rope->prob);
  if (s != MLA_OK) return s;
  if (!std::isfinite(rope->mscale)) return MLA_ERR_INVALID_ARG;
  const bool q = num_heads > 0;
  if (out_dtype != MLA_DTYPE_BF16 && out_dtype != MLA_DTYPE_FP8_E4M3) return MLA_ERR_INVALID_ARG;
  const bool fp8 = out_dtype == MLA_DTYPE_FP8_E4M3;
  // (1 / q_scale must be finite too)
  if (q && fp8 && !(std::isfinite(q_scale) && q_scale > 0.f && std::isfinite(1.f / q_scale))) return MLA_ERR_INVALID_ARG;
  if (num_tokens == 0) return MLA_OK;
  if (!q && k_pe == nullptr) return MLA_ERR_INVALID_ARG;
  if (positions == nullptr || !aligned(positions, 4)) return MLA_ERR_INVALID_ARG;
  mla::RopeParams p{};
  if (q) {
    if (ql_nope == nullptr || q_pe == nullptr || q_out == nullptr) return MLA_ERR_INVALID_ARG;
    if (nope_stride_t < 0 || nope_stride_h < 0 || pe_stride_t < 0 || pe_stride_h < 0) return MLA_ERR_INVALID_ARG;
    // 16-byte accesses of the latent part and the output, pairs of the rope part
    if (!aligned(ql_nope, 16) || !aligned(q_out, 16) || !aligned(q_pe, 4) || nope_stride_t % 8 || nope_stride_h % 8 ||
        pe_stride_t % 2 || pe_stride_h % 2)
      return MLA_ERR_INVALID_ARG;
    p.num_heads = num_heads;
    p.nope = ql_nope;
    p.nope_st = nope_stride_t;
    p.nope_sh = nope_stride_h;
    p.pe = q_pe;
    p.pe_st = pe_stride_t;
    p.pe_sh = pe_stride_h;
    p.fp8 = fp8 ? 1 : 0;
    p.q_inv = fp8 ? 1.f / q_scale : 1.f;
    p.out = q_out;
  }
  if (k_pe != nullptr) {
    if (k_out == nullptr || !aligned(k_pe, 4) || !aligned(k_out, 4) || k_pe_stride % 2 || k_out_stride % 2)
      return MLA_ERR_INVALID_ARG;
    if (num_tokens > 1 && (k_pe_stride < 0 || k_out_stride < kRopeCols)) return MLA_ERR_INVALID_ARG;
    if (num_tokens > 1 && k_pe == k_out && k_pe_stride != k_out_stride) return MLA_ERR_INVALID_ARG;
    p.k_pe = k_pe;
    p.k_st = k_pe_stride;
    p.k_out = k_out;
    p.k_out_st = k_out_stride;
  }
  p.positions = positions;
  p.num_tokens = num_tokens;
  p.dim = rope->prob.dim;
  p.half = rope->prob.layout == MLA_ROPE_HALF ? 1 : 0;
  p.mscale = rope->mscale;
  static_assert(sizeof(p.turns) == sizeof(rope->turns), "the plan's pairs");
  std::memcpy(p.turns, rope->turns, sizeof(p.turns));
  return cuda_status(mla::launch_rope(p, stream));
}

size_t mla_cache_workspace(int32_t num_blocks) { return num_blocks > 0 ? page_layout(num_blocks).end : 0; }

mla_status_t mla_cache_copy_blocks(const int32_t* src, const int32_t* dst, int32_t num_pairs, int32_t num_blocks,
                                   int32_t block_size, int32_t kv_dtype, int32_t scale_group, void* kv_cache,
                                   float* kv_scales, cudaStream_t stream) {
  mla::PageCopy c{};
  if (num_pairs < 0) return MLA_ERR_INVALID_ARG;
  const mla_status_t s = check_pages(kv_cache, kv_scales, num_blocks, block_size, kv_dtype, scale_group, &c);
  if (s != MLA_OK) return s;
  if (num_pairs == 0) return MLA_OK;
  if (src == nullptr || dst == nullptr || !aligned(src, 4) || !aligned(dst, 4)) return MLA_ERR_INVALID_ARG;
  return cuda_status(mla::launch_copy_blocks(c, src, dst, num_pairs, stream));
}

mla_status_t mla_cache_fork(const int32_t* parent, const int32_t* child, const int32_t* lens, int32_t num_forks,
                            const int32_t* free_blocks, int32_t num_free, int32_t* block_table,
                            int64_t block_table_stride, int32_t num_rows, int32_t max_blocks_per_req,
                            int32_t* ref_counts, int32_t num_blocks, int32_t block_size, int32_t kv_dtype,
                            int32_t scale_group, void* kv_cache, float* kv_scales, int32_t* taken,
                            cudaStream_t stream) {
  mla::ForkParams p{};
  if (num_forks < 0 || num_free < 0 || num_rows < 0 || max_blocks_per_req <= 0) return MLA_ERR_INVALID_ARG;
  const mla_status_t s = check_pages(kv_cache, kv_scales, num_blocks, block_size, kv_dtype, scale_group, &p.copy);
  if (s != MLA_OK) return s;
  if (taken == nullptr || !aligned(taken, 4)) return MLA_ERR_INVALID_ARG;
  if (num_forks > 0) {
    if (block_table_stride < max_blocks_per_req || num_rows == 0) return MLA_ERR_INVALID_ARG;
    if (parent == nullptr || child == nullptr || lens == nullptr || block_table == nullptr || ref_counts == nullptr)
      return MLA_ERR_INVALID_ARG;
    if (!aligned(parent, 4) || !aligned(child, 4) || !aligned(lens, 4) || !aligned(block_table, 4) ||
        !aligned(ref_counts, 4))
      return MLA_ERR_INVALID_ARG;
    if (num_free > 0 && (free_blocks == nullptr || !aligned(free_blocks, 4))) return MLA_ERR_INVALID_ARG;
  }
  p.parent = parent;
  p.child = child;
  p.lens = lens;
  p.num_forks = num_forks;
  p.block_size = block_size;
  p.free_blocks = free_blocks;
  p.num_free = num_free;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.num_rows = num_rows;
  p.cols = max_blocks_per_req;
  p.ref_counts = ref_counts;
  p.taken = taken;
  return cuda_status(mla::launch_fork(p, stream));
}

mla_status_t mla_cache_free(const int32_t* rows, const int32_t* lens, int32_t num_listed, int32_t* block_table,
                            int64_t block_table_stride, int32_t num_rows, int32_t max_blocks_per_req,
                            int32_t* ref_counts, int32_t num_blocks, int32_t block_size, int32_t* freed,
                            int32_t capacity, int32_t* num_freed, void* workspace, size_t workspace_bytes,
                            cudaStream_t stream) {
  if (num_listed < 0 || num_rows < 0 || max_blocks_per_req <= 0 || num_blocks <= 0 || block_size <= 0 || capacity < 0)
    return MLA_ERR_INVALID_ARG;
  if (num_freed == nullptr || !aligned(num_freed, 4)) return MLA_ERR_INVALID_ARG;
  if (capacity > 0 && (freed == nullptr || !aligned(freed, 4))) return MLA_ERR_INVALID_ARG;
  if (num_listed > 0) {
    if (block_table_stride < max_blocks_per_req || num_rows == 0) return MLA_ERR_INVALID_ARG;
    if (rows == nullptr || block_table == nullptr || ref_counts == nullptr || !aligned(rows, 4) ||
        !aligned(block_table, 4) || !aligned(ref_counts, 4) || (lens != nullptr && !aligned(lens, 4)))
      return MLA_ERR_INVALID_ARG;
  }
  const PageLayout l = page_layout(num_blocks);
  if (workspace == nullptr || workspace_bytes < l.end) return MLA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  mla::FreeParams p{};
  p.rows = rows;
  p.lens = lens;
  p.num_listed = num_listed;
  p.block_size = block_size;
  p.block_table = block_table;
  p.bt_stride = block_table_stride;
  p.num_rows = num_rows;
  p.cols = max_blocks_per_req;
  p.ref_counts = ref_counts;
  p.num_blocks = num_blocks;
  p.freed = freed;
  p.capacity = capacity;
  p.num_freed = num_freed;
  p.ticket = reinterpret_cast<int32_t*>(ws);
  p.bitmap = reinterpret_cast<uint32_t*>(ws + l.bitmap);
  return cuda_status(mla::launch_free(p, stream));
}

mla_status_t mla_cache_compact(const int32_t* ref_counts, int32_t* ref_counts_out, const int32_t* block_table,
                               int64_t block_table_stride, int32_t* block_table_out, int64_t block_table_out_stride,
                               int32_t num_rows, int32_t max_blocks_per_req, int32_t num_blocks, int32_t block_size,
                               int32_t kv_dtype, int32_t scale_group, void* kv_cache, float* kv_scales,
                               int32_t* num_live, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  mla::CompactParams p{};
  if (num_rows < 0 || max_blocks_per_req <= 0) return MLA_ERR_INVALID_ARG;
  const mla_status_t s = check_pages(kv_cache, kv_scales, num_blocks, block_size, kv_dtype, scale_group, &p.copy);
  if (s != MLA_OK) return s;
  if (ref_counts == nullptr || ref_counts_out == nullptr || num_live == nullptr || !aligned(ref_counts, 4) ||
      !aligned(ref_counts_out, 4) || !aligned(num_live, 4))
    return MLA_ERR_INVALID_ARG;
  if (num_rows > 0) {
    if (block_table == nullptr || block_table_out == nullptr || !aligned(block_table, 4) || !aligned(block_table_out, 4))
      return MLA_ERR_INVALID_ARG;
    if (block_table_stride < max_blocks_per_req || block_table_out_stride < max_blocks_per_req) return MLA_ERR_INVALID_ARG;
    if (block_table == block_table_out && block_table_stride != block_table_out_stride) return MLA_ERR_INVALID_ARG;
  }
  const PageLayout l = page_layout(num_blocks);
  if (workspace == nullptr || workspace_bytes < l.end) return MLA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.refs = ref_counts;
  p.refs_out = ref_counts_out;
  p.table = block_table;
  p.table_stride = block_table_stride;
  p.table_out = block_table_out;
  p.table_out_stride = block_table_out_stride;
  p.num_rows = num_rows;
  p.cols = max_blocks_per_req;
  p.num_live = num_live;
  p.head = reinterpret_cast<int32_t*>(ws) + 8;
  p.holes = reinterpret_cast<int32_t*>(ws + l.holes);
  p.from = reinterpret_cast<int32_t*>(ws + l.from);
  p.back = reinterpret_cast<int32_t*>(ws + l.back);
  return cuda_status(mla::launch_compact(p, stream));
}

}  // extern "C"
