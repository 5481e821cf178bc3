// block_tables.cu -- the block table's new columns, the slot map, and each
// token's request and position, from the request lengths of one step. With
// q_r new tokens of the len_r of request r, c_r = len_r - q_r of them already
// in the cache and bs tokens per block, the request owns the first
// old_r = ceil(c_r / bs) columns of its table row and takes
//   new_r = min(ceil(len_r / bs), columns) - old_r
// blocks of the free list, in request order from base_r = sum_{i < r} new_i;
// token t sits at position c_r + t - query_start_loc[r].
//
// One launch and no workspace: a CTA owns kTok consecutive tokens. It adds up
// new_r of the requests that end before its tokens (a strided read of the two
// length arrays by all threads), scans those of the requests that meet its
// tokens, and leaves a record at the first token of each; a maximum scan over
// the tokens then gives every token its record. A token at the start of a
// block is that column's first (c_r <= its position), so it also writes the
// column: no pass over the table is needed. Each CTA re-reads the lengths of
// all earlier requests (8 bytes each, from L2): with R requests in all that is
// R / kTok strips, against a second launch that a precomputed prefix would
// cost.
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kTok = 512;  // tokens, and threads, per CTA
constexpr int kNWarps = kTok / 32;

struct Lens {
  int q0, q1;    // the request's first token and the one past its last
  int ctx, old;  // tokens and blocks it has already
  int fresh;     // blocks it takes
};

__device__ __forceinline__ Lens request_lens(const BlockTableParams& p, int r) {
  Lens l;
  l.q0 = p.qsl[r];
  l.q1 = p.qsl[r + 1];
  const int len = p.seq_lens[r];
  l.ctx = max(len - (l.q1 - l.q0), 0);
  l.old = l.ctx / p.block_size + (l.ctx % p.block_size != 0);
  const int need = min(len / p.block_size + (len % p.block_size != 0), p.cols);
  l.fresh = max(need - l.old, 0);
  return l;
}

__global__ void __launch_bounds__(kTok) block_tables_kernel(const BlockTableParams p) {
  __shared__ int s_sum[2][kNWarps];
  __shared__ int s_head[kTok];             // 1 + index of the record that starts at a token, or 0
  __shared__ int4 s_rec[kTok];             // {request, base - old, old, ctx - q0}
  __shared__ int s_end[kTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t0 = blockIdx.x * kTok;
  const int t1 = min(t0 + kTok, p.num_tokens);
  s_head[tid] = 0;

  // requests whose tokens all lie before t0 (they come first: query_start_loc
  // does not decrease): how many, and the blocks they take
  int count = 0, taken = 0;
  if (t0 > 0) {
    for (int r = tid; r < p.num_reqs; r += kTok) {
      const Lens l = request_lens(p, r);
      if (l.q1 > t0) break;
      ++count;
      taken += l.fresh;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    count += __shfl_xor_sync(0xffffffffu, count, o);
    taken += __shfl_xor_sync(0xffffffffu, taken, o);
  }
  if (lane == 0) {
    s_sum[0][warp] = count;
    s_sum[1][warp] = taken;
  }
  __syncthreads();
  int first = 0, carry = 0;
#pragma unroll
  for (int w = 0; w < kNWarps; ++w) {
    first += s_sum[0][w];
    carry += s_sum[1][w];
  }

  // the requests that meet [t0, t1), in strips: records and running base
  for (int r0 = first; r0 < p.num_reqs; r0 += kTok) {
    const int r = r0 + tid;
    Lens l{};
    bool meets = false;
    if (r < p.num_reqs) {
      l = request_lens(p, r);
      meets = l.q0 < t1 && l.q1 > l.q0 && l.q1 > t0;
      if (l.q0 >= p.num_tokens) l.fresh = 0;  // no token of it is in this step
    }
    int inc = l.fresh;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();  // every thread has read s_sum
    if (lane == 31) s_sum[0][warp] = inc;
    const int more = __syncthreads_or(r + 1 < p.num_reqs && tid == kTok - 1 && l.q1 < t1);
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kNWarps; ++w) {
      const int s = s_sum[0][w];
      if (w < warp) before += s;
      total += s;
    }
    if (meets) {
      const int at = max(l.q0 - t0, 0);
      s_rec[at] = make_int4(r, carry + before + inc - l.fresh - l.old, l.old, l.ctx - l.q0);
      s_end[at] = l.q1;
      s_head[at] = at + 1;
    }
    carry += total;
    if (!more) break;
  }
  if (blockIdx.x == gridDim.x - 1 && tid == 0) *p.taken = carry;
  __syncthreads();

  // each token's record: the last one that starts at or before it
  int head = s_head[tid];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, head, o);
    if (lane >= o) head = max(head, v);
  }
  if (lane == 31) s_sum[1][warp] = head;
  __syncthreads();
  for (int w = 0; w < warp; ++w) head = max(head, s_sum[1][w]);
  const int t = t0 + tid;
  if (t >= t1) return;
  int slot = -1, req = -1, pos = -1;
  if (head > 0 && t < s_end[head - 1]) {
    const int4 rec = s_rec[head - 1];
    req = rec.x;
    pos = t + rec.w;
    const int col = pos / p.block_size, off = pos - col * p.block_size;
    if (col < p.cols) {
      int32_t* cell = p.block_table + static_cast<int64_t>(req) * p.bt_stride + col;
      int block;
      if (col < rec.z) {
        block = *cell;
      } else {
        const int i = rec.y + col;
        block = i < p.num_free ? p.free_blocks[i] : -1;
        if (off == 0) *cell = block;
      }
      if (block >= 0) slot = block * p.block_size + off;
    }
  }
  p.slots[t] = slot;
  if (p.req_id != nullptr) p.req_id[t] = req;
  if (p.positions != nullptr) p.positions[t] = pos;
}

}  // namespace

cudaError_t launch_block_tables(const BlockTableParams& p, cudaStream_t stream) {
  const int ctas = p.num_tokens > 0 ? (p.num_tokens - 1) / kTok + 1 : 1;
  block_tables_kernel<<<static_cast<unsigned>(ctas), kTok, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
