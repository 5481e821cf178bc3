// cache_pages.cu -- the pages of a cache whose requests share them: forking
// table rows, copying, freeing and compacting blocks. A block is block_size rows
// (576 bf16 or e4m3 columns) and, of a cache with group scales, its scales;
// ref_counts[b] is the number of table cells that hold block b.
//
// All of it is bound by the bytes moved: 16-byte loads, kUnroll of them in flight
// a thread, spread over all SMs by the total, not by the block. The bookkeeping
// around it is done by the same launches.
//
// Measured: 4000 bf16 blocks of 64 copied in 95.5 us, 6.2 TB/s (0.91 of the copy rate);
// 16384 e4m3 blocks, 60 % in use, compacted in 57.5 (scan 7, then the moves at 0.92 of the
// rate); 64 prompts forked into 8 samples each in 6.2 us and 4 forks of one in 3.4 in a
// captured graph, latency: earlier forks counted, table cells, rows.
#include "common.cuh"
#include "internal.h"
#include "tc_ops.cuh"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 8;

__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

// Units of 16 bytes [u0, u1) of the whole-block copies `pair(k) = {src, dst}`, laid
// end to end; pairs with a negative member are passed over. Called by all threads.
template <typename Pair>
__device__ void copy_units(const PageCopy& c, int64_t u0, int64_t u1, Pair pair) {
  const int upb = c.block_units;
  int64_t k = u0 / upb;
  int off = static_cast<int>(u0 - k * upb) + static_cast<int>(threadIdx.x);
  uint4* base = static_cast<uint4*>(c.cache);
  for (int64_t u = u0 + threadIdx.x; u < u1; u += kUnroll * kThreads) {
    uint4 v[kUnroll];
    uint4* to[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      to[i] = nullptr;
      if (u + i * kThreads < u1) {
        while (off >= upb) {
          off -= upb;
          ++k;
        }
        const int2 m = pair(k);
        if (m.x >= 0 && m.y >= 0 && m.x < c.num_blocks && m.y < c.num_blocks) {
          v[i] = load_stream(base + static_cast<int64_t>(m.x) * upb + off);
          to[i] = base + static_cast<int64_t>(m.y) * upb + off;
          if (off < c.block_scales)  // (at most block_size scales a block, fewer than its units)
            c.scales[static_cast<int64_t>(m.y) * c.block_scales + off] =
                c.scales[static_cast<int64_t>(m.x) * c.block_scales + off];
        }
      }
      off += kThreads;
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (to[i] != nullptr) *to[i] = v[i];
  }
}

// The share of `total` units that CTA `i` of `n` takes, in whole steps of its threads.
__device__ __forceinline__ int64_t share_begin(int64_t total, int i, int n) {
  constexpr int64_t kStep = kThreads;
  const int64_t steps = (total + kStep - 1) / kStep;
  const int64_t b = steps * i / n * kStep;
  return b < total ? b : total;
}

__global__ void __launch_bounds__(kThreads) copy_kernel(const PageCopy c, const int32_t* src, const int32_t* dst, int n) {
  const int64_t total = static_cast<int64_t>(n) * c.block_units;
  copy_units(c, share_begin(total, blockIdx.x, gridDim.x), share_begin(total, blockIdx.x + 1, gridDim.x),
             [&](int64_t k) { return make_int2(src[k], dst[k]); });
}

// ------------------------------------------------------------------ fork
struct ForkLens {
  int whole, rest;  // shared blocks; rows of the block that is copied
};
// Shape of fork i; nothing where a row does not exist.
__device__ __forceinline__ ForkLens fork_lens(const ForkParams& p, int i) {
  ForkLens l{0, 0};
  const int parent = p.parent[i], child = p.child[i];
  if (parent < 0 || parent >= p.num_rows || child < 0 || child >= p.num_rows) return l;
  const int len = max(p.lens[i], 0);
  l.whole = min(len / p.block_size, p.cols);
  l.rest = l.whole < p.cols ? len % p.block_size : 0;
  // (a partly filled column without a block takes none)
  if (l.rest > 0 && p.block_table[parent * p.bt_stride + l.whole] < 0) l.rest = -1;
  return l;
}

// CTA (i, part): fork i's table row and counts (part 0), and its part of the rows
// copied. Its place in the free list is the number of forks before it that
// copy a block, counted by each CTA anew: n^2 / 2 reads from L2 in all, no second launch.
__global__ void __launch_bounds__(kThreads) fork_kernel(const ForkParams p) {
  __shared__ int s_before[kThreads / 32];
  const int i = blockIdx.x, part = blockIdx.y;
  int before = 0;
  for (int j = threadIdx.x; j < i; j += kThreads) before += fork_lens(p, j).rest > 0 ? 1 : 0;
  before = __reduce_add_sync(0xffffffffu, before);
  if ((threadIdx.x & 31) == 0) s_before[threadIdx.x >> 5] = before;
  const ForkLens l = fork_lens(p, i);
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) before += s_before[w];
  if (part == 0 && i + 1 == p.num_forks && threadIdx.x == 0) *p.taken = before + (l.rest > 0 ? 1 : 0);
  const int fresh = l.rest > 0 && before < p.num_free ? p.free_blocks[before] : -1;
  if (l.whole == 0 && l.rest == 0) return;
  const int32_t* from = p.block_table + p.parent[i] * p.bt_stride;
  int32_t* to = p.block_table + p.child[i] * p.bt_stride;
  if (part == 0) {
    for (int c = threadIdx.x; c < l.whole; c += kThreads) {
      const int b = from[c];
      to[c] = b;
      if (b >= 0 && b < p.copy.num_blocks) atomicAdd(p.ref_counts + b, 1);
    }
    if (threadIdx.x == 0 && l.rest != 0) {
      to[l.whole] = fresh;
      if (fresh >= 0 && fresh < p.copy.num_blocks) p.ref_counts[fresh] = 1;
    }
  }
  if (l.rest <= 0 || fresh < 0 || fresh >= p.copy.num_blocks) return;
  const int old = from[l.whole];
  if (old >= p.copy.num_blocks) return;
  const int upb = p.copy.block_units, units = l.rest * (upb / p.block_size);
  const uint4* src = static_cast<const uint4*>(p.copy.cache) + static_cast<int64_t>(old) * upb;
  uint4* dst = static_cast<uint4*>(p.copy.cache) + static_cast<int64_t>(fresh) * upb;
  const int stride = kThreads * gridDim.y;
  int u = part * kThreads + threadIdx.x;
  for (; u + 3 * stride < units; u += 4 * stride) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = load_stream(src + u + k * stride);
#pragma unroll
    for (int k = 0; k < 4; ++k) dst[u + k * stride] = v[k];
  }
  for (; u < units; u += stride) dst[u] = load_stream(src + u);
  if (part == 0 && p.copy.block_scales > 0) {
    const int group = p.block_size / p.copy.block_scales;
    const int n = (l.rest + group - 1) / group;
    for (int k = threadIdx.x; k < n; k += kThreads)
      p.copy.scales[static_cast<int64_t>(fresh) * p.copy.block_scales + k] =
          p.copy.scales[static_cast<int64_t>(old) * p.copy.block_scales + k];
  }
}

// ------------------------------------------------------------------ free
// CTA i gives up row rows[i]: each cell is taken out of the table by an exchange (a
// row that is listed twice is given up once), its block's count falls, and a block
// that reaches zero is marked in the bitmap. The last CTA to finish lists the
// marked blocks in ascending order (so that the list is the same on every run),
// and leaves bitmap and ticket zero for the next call.
__global__ void __launch_bounds__(kThreads) free_kernel(const FreeParams p) {
  __shared__ int s_last, s_warp[kThreads / 32];
  for (int i = blockIdx.x; i < p.num_listed; i += gridDim.x) {
    const int row = p.rows[i];
    if (row < 0 || row >= p.num_rows) continue;
    const int len = p.lens != nullptr ? max(p.lens[i], 0) : 0;
    const int cols = p.lens != nullptr ? min(len / p.block_size + (len % p.block_size != 0), p.cols) : p.cols;
    for (int c = threadIdx.x; c < cols; c += kThreads) {
      const int b = atomicExch(p.block_table + row * p.bt_stride + c, -1);
      if (b < 0 || b >= p.num_blocks) continue;
      if (atomicSub(p.ref_counts + b, 1) == 1) atomicOr(p.bitmap + (b >> 5), 1u << (b & 31));
    }
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    s_last = atomicAdd(p.ticket, 1) == static_cast<int>(gridDim.x) - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  const int words = (p.num_blocks + 31) / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int carry = 0;
  for (int w0 = 0; w0 < words; w0 += kThreads) {
    const int w = w0 + threadIdx.x;
    uint32_t bits = w < words ? __ldcg(p.bitmap + w) : 0u;
    const int mine = __popc(bits);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int at = carry + inc - mine;
    for (int k = 0; k < kThreads / 32; ++k) {
      const int v = s_warp[k];
      if (k < warp) at += v;
      carry += v;
    }
    if (bits != 0u) p.bitmap[w] = 0u;
    while (bits != 0u) {
      const int b = __ffs(bits) - 1;
      bits &= bits - 1;
      if (at < p.capacity) p.freed[at] = 32 * w + b;
      ++at;
    }
  }
  if (threadIdx.x == 0) {
    *p.num_freed = carry;
    *p.ticket = 0;
  }
}

// ------------------------------------------------------------------ compact
// With L blocks in use, the k-th unused block below L takes the contents of the
// k-th used block from L on: the fewest moves, in an order of its own. One
// cluster of kScanCtas CTAs finds both lists: each counts its segment of the
// counts, the numbers are exchanged through shared memory, then each writes its
// segment's entries: holes[k], and, of the used blocks from L on, which are
// numbered from the last one back (so that no CTA needs their number), from[back]
// and back[b - L] (-1 of an unused one). The CTA that owns block L knows their
// number M = L - used below L.
constexpr int kScanCtas = 8;
constexpr int kScanThreads = 1024;

// Exclusive prefix of v over the block.
__device__ __forceinline__ int scan_block(int v, int* s_warp, int* total) {
  static_assert(kScanThreads == 32 * 32, "a lane for each warp's sum");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  const int mine = s_warp[lane];
  int all = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, all, o);
    if (lane >= o) all += x;
  }
  *total = __shfl_sync(0xffffffffu, all, 31);
  return __shfl_sync(0xffffffffu, all - mine, warp) + inc - v;
}

// A thread takes a run of blocks and keeps what it read of up to 32 of them (the counts
// read twice and scanned 1024 at a time: 59.6 us for the call, of 16384 blocks).
__global__ void __cluster_dims__(kScanCtas, 1, 1) __launch_bounds__(kScanThreads) compact_scan_kernel(const CompactParams p) {
  __shared__ int s_warp[kScanThreads / 32];
  __shared__ int s_count;
  const int rank = static_cast<int>(tc::cluster_ctarank());
  const int N = p.copy.num_blocks;
  const int run = (N - 1) / (kScanCtas * kScanThreads) + 1;
  const int64_t begin = static_cast<int64_t>(rank * kScanThreads + threadIdx.x) * run;
  const int b0 = static_cast<int>(begin < N ? begin : N);
  const int n = min(run, N - b0);
  uint32_t kept = 0u;
  int mine = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const bool used = p.refs[b0 + i] > 0;
    mine += used ? 1 : 0;
    if (i < 32) kept |= used ? 1u << i : 0u;
  }
  int total;
  int at = scan_block(mine, s_warp, &total);
  if (threadIdx.x == 0) s_count = total;
  __syncthreads();
  tc::cluster_sync();
  int live = 0, before = 0;  // used blocks of the pool, and below this CTA's
#pragma unroll
  for (int r = 0; r < kScanCtas; ++r) {
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(tc::map_to_rank(smem_u32(&s_count), r)) : "memory");
    live += v;
    if (r < rank) before += v;
  }
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  if (rank == 0 && threadIdx.x == 0) {
    *p.num_live = live;
    p.head[0] = live;
    if (live == N) p.head[1] = 0;
  }
  at += before;  // used blocks before b
  for (int i = 0; i < n; ++i) {
    const int b = b0 + i;
    const bool used = i < 32 ? (kept >> i & 1u) != 0u : p.refs[b] > 0;
    if (b == live) p.head[1] = live - at;
    if (b < live) {
      if (!used) p.holes[b - at] = b;
    } else {
      const int back = live - 1 - at;  // used blocks behind b
      p.back[b - live] = used ? back : -1;
      if (used) p.from[back] = b;
    }
    at += used ? 1 : 0;
  }
  tc::cluster_sync();  // (every CTA has read the others' counts: they may exit)
}

// The counts, the table and the contents by the two lists. refs_out and table_out
// may be the inputs: the count of a moved block and that of its new place are
// written by one thread, and every other entry only by the thread that reads it.
__global__ void __launch_bounds__(kThreads) compact_move_kernel(const CompactParams p) {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int live = __ldcg(p.head), moves = __ldcg(p.head + 1);
  const int N = p.copy.num_blocks;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  auto pair = [&](int64_t k) { return make_int2(p.from[moves - 1 - k], p.holes[k]); };
  const int64_t total = static_cast<int64_t>(moves) * p.copy.block_units;
  copy_units(p.copy, share_begin(total, blockIdx.x, gridDim.x), share_begin(total, blockIdx.x + 1, gridDim.x), pair);
  for (int64_t k = first; k < moves; k += step) {
    const int2 m = pair(k);
    const int n = p.refs[m.x];
    p.refs_out[m.y] = n;
    p.refs_out[m.x] = 0;
  }
  for (int64_t b = first; b < N; b += step) {
    if (b < live) {
      const int n = p.refs[b];
      if (n > 0) p.refs_out[b] = n;  // (else a hole, above)
    } else if (p.back[b - live] < 0) {
      p.refs_out[b] = 0;
    }
  }
  const int64_t cells = static_cast<int64_t>(p.num_rows) * p.cols;
  for (int64_t i = first; i < cells; i += step) {
    const int64_t r = i / p.cols, c = i - r * p.cols;
    int b = p.table[r * p.table_stride + c];
    if (b >= live && b < N) {
      const int back = p.back[b - live];
      if (back >= 0) b = p.holes[moves - 1 - back];
    }
    p.table_out[r * p.table_out_stride + c] = b;
  }
}

}  // namespace

cudaError_t launch_copy_blocks(const PageCopy& c, const int32_t* src, const int32_t* dst, int n, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int64_t total = static_cast<int64_t>(n) * c.block_units;
  const int64_t want = (total + kUnroll * kThreads - 1) / (kUnroll * kThreads);
  const int64_t most = static_cast<int64_t>(sms) * 64;
  copy_kernel<<<static_cast<unsigned>(want < most ? want : most), kThreads, 0, stream>>>(c, src, dst, n);
  return cudaGetLastError();
}

cudaError_t launch_fork(const ForkParams& p, cudaStream_t stream) {
  if (p.num_forks == 0) return cudaMemsetAsync(p.taken, 0, sizeof(int32_t), stream);
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  // a block's rows by one to eight CTAs: up to four an SM in all, no CTA without work
  const int upb = p.copy.block_units;
  int parts = 4 * sms / p.num_forks;
  if (parts > upb / (2 * kThreads)) parts = upb / (2 * kThreads);
  if (parts > 8) parts = 8;
  if (parts < 1) parts = 1;
  fork_kernel<<<dim3(static_cast<unsigned>(p.num_forks), static_cast<unsigned>(parts)), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_free(const FreeParams& p, cudaStream_t stream) {
  if (p.num_listed == 0) return cudaMemsetAsync(p.num_freed, 0, sizeof(int32_t), stream);
  const int ctas = p.num_listed < 4096 ? p.num_listed : 4096;
  free_kernel<<<static_cast<unsigned>(ctas), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_compact(const CompactParams& p, cudaStream_t stream) {
  int sms = 0;
  cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  compact_scan_kernel<<<kScanCtas, kScanThreads, 0, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(sms) * 8u);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, compact_move_kernel, p);
}

}  // namespace mla
