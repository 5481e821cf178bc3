// cache_append.cu -- a step's latent rows (c_kv || k_pe, bf16) into an e4m3
// cache with one fp32 scale for each group of g slots of a block.
//
// A run is a maximal stretch of consecutive tokens at consecutive slots of one
// group; its team (a warp for groups of at most 8 slots, else a CTA) is the
// only one that touches the group. With a the largest finite magnitude of the
// run's rows, the group's scale becomes
//   s = max(2^k, 2^-60, s_old if the run starts behind rows of its group),
// k the least integer with a <= 448 2^k, and the rows are stored as
// e4m3(x / s). Where s grew, the rows before the run are requantised by
// s_old / s. Scales made here are powers of two, so that this changes no code
// but those that fall below e4m3's normal range: a group that grows again and
// again loses no more than one that grew once. (A floating-point format gains
// nothing from a finer scale but part of a binade of range.)
//
// What bounds it: memory, 1152 bytes read and 576 written a token. The rows of
// a run are read once and kept in registers (18 16-byte pieces a thread cover
// 64 rows with 256 threads, 8 rows with a warp) between the maximum and the
// rounding; longer runs are read a second time, from L2.
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kThreads = 256;
constexpr int kPieces = kHeadDim / 8;      // 16-byte bf16 pieces of a row: 64 latent, 8 rope
constexpr int kNopePieces = kRank / 8;
constexpr int kHold = 18;                  // pieces a thread keeps in registers
constexpr int kWarpGroup = 8;              // largest group a warp takes
constexpr int kMaxWindow = 256;            // tokens of a CTA team's window
constexpr int kMinExp = -60;               // the smallest scale is 2^-60

template <int TS>
__device__ __forceinline__ void team_sync() {
  if constexpr (TS == 32) __syncwarp(); else __syncthreads();
}

__device__ __forceinline__ uint4 load_piece(const AppendParams& p, int64_t t, int piece) {
  const __nv_bfloat16* src = piece < kNopePieces
                                 ? static_cast<const __nv_bfloat16*>(p.c_kv) + t * p.c_stride + piece * 8
                                 : static_cast<const __nv_bfloat16*>(p.k_pe) + t * p.pe_stride + (piece - kNopePieces) * 8;
  return __ldg(reinterpret_cast<const uint4*>(src));
}

// Largest finite magnitudes of a piece, as bf16 bits in both halves.
__device__ __forceinline__ uint32_t piece_max(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFF7FFFu;
    m = __vmaxu2(m, a & ~__vcmpgtu2(a, 0x7F7F7F7Fu));
  }
  return m;
}

// The power of two that brings a bf16 magnitude (its bits) to 448 or below:
// 448 = 1.75 * 2^8, and the mantissa of 1.75 is 0x60.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  int e = static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);
  e = max(e, kMinExp);
  return __int_as_float((e + 127) << 23);
}

__device__ __forceinline__ uint2 quantise(uint4 v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(f.x * inv, f.y * inv), __NV_SATFINITE, __NV_E4M3);
    out[i >> 1] |= (c & 0xFFFFu) << ((i & 1) * 16);
  }
  return make_uint2(out[0], out[1]);
}

__device__ __forceinline__ uint32_t requantise(uint32_t codes, float ratio) {
  uint32_t out = 0u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(codes >> (16 * i)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE, __NV_E4M3);
    out |= (c & 0xFFFFu) << (16 * i);
  }
  return out;
}

// Team of TS threads (rank `tr`): the run of n tokens from t at slot s0.
template <int TS>
__device__ void append_run(const AppendParams& p, int t, int s0, int n, int tr, uint32_t* red) {
  const int g = p.group;
  const int before = s0 % g;  // rows of the group that are there already
  const float old = before > 0 ? p.scales[s0 / g] : 0.f;
  const int pieces = n * kPieces;
  const bool held = pieces <= kHold * TS;
  uint4 v[kHold];
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int i = j * TS + tr;
    v[j] = make_uint4(0u, 0u, 0u, 0u);
    if (i < pieces) v[j] = load_piece(p, t + i / kPieces, i % kPieces);
  }
#pragma unroll
  for (int j = 0; j < kHold; ++j) m = piece_max(v[j], m);
  for (int i = kHold * TS + tr; i < pieces; i += TS) m = piece_max(load_piece(p, t + i / kPieces, i % kPieces), m);
  m = max(m & 0xFFFFu, m >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (TS > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < TS / 32; ++w) m = max(m, red[w]);
  }
  const float s = fmaxf(scale_of(m), old);
  const float inv = 1.f / s;
  uint8_t* rows = static_cast<uint8_t*>(p.cache) + static_cast<int64_t>(s0) * kHeadDim;
  if (tr == 0) p.scales[s0 / g] = s;
#pragma unroll
  for (int j = 0; j < kHold; ++j) {
    const int i = j * TS + tr;
    if (i < pieces) *reinterpret_cast<uint2*>(rows + static_cast<int64_t>(i) * 8) = quantise(v[j], inv);
  }
  if (!held)
    for (int i = kHold * TS + tr; i < pieces; i += TS)
      *reinterpret_cast<uint2*>(rows + static_cast<int64_t>(i) * 8) =
          quantise(load_piece(p, t + i / kPieces, i % kPieces), inv);
  if (before > 0 && s > old) {
    const float ratio = old / s;
    uint4* head = reinterpret_cast<uint4*>(rows - static_cast<int64_t>(before) * kHeadDim);
    for (int i = tr; i < before * (kHeadDim / 16); i += TS) {
      uint4 c = head[i];
      c.x = requantise(c.x, ratio);
      c.y = requantise(c.y, ratio);
      c.z = requantise(c.z, ratio);
      c.w = requantise(c.w, ratio);
      head[i] = c;
    }
  }
}

// A token's slot, or -1 where it has none (or one outside the cache).
__device__ __forceinline__ int slot_at(const AppendParams& p, int t) {
  const int s = t >= 0 && t < p.num_tokens ? p.slots[t] : -1;
  return s >= 0 && s < p.num_slots ? s : -1;
}

__device__ __forceinline__ bool starts_run(int prev, int s, int g) {
  return s >= 0 && !(prev + 1 == s && s % g != 0);
}

// Groups of at most kWarpGroup slots: a warp per token; those that start a run work.
__global__ void __launch_bounds__(kThreads) append_warp_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.num_tokens) return;
  const int mine = slot_at(p, t - 1 + lane);  // lane 0: the token before
  const int s0 = __shfl_sync(0xffffffffu, mine, 1);
  const int prev = __shfl_sync(0xffffffffu, mine, 0);
  if (!starts_run(prev, s0, p.group)) return;
  const int room = p.group - s0 % p.group;
  const uint32_t same = __ballot_sync(0xffffffffu, lane >= 1 && lane - 1 < room && mine == s0 + lane - 1);
  const int n = __ffs(~(same >> 1)) - 1;  // consecutive slots from the first
  append_run<32>(p, t, s0, n, lane, nullptr);
}

// Larger groups: a CTA per window of tokens takes the runs that start in it.
__global__ void __launch_bounds__(kThreads) append_cta_kernel(const AppendParams p, int window) {
  __shared__ int s_slot[kMaxWindow + 1];
  __shared__ int s_len;
  __shared__ uint32_t s_red[kThreads / 32];
  const int tid = threadIdx.x;
  const int w0 = blockIdx.x * window;
  for (int i = tid; i <= window; i += kThreads) s_slot[i] = slot_at(p, w0 - 1 + i);
  __syncthreads();
  for (int i = 0; i < window; ++i) {
    const int s0 = s_slot[i + 1];
    if (!starts_run(s_slot[i], s0, p.group)) continue;
    const int t = w0 + i;
    const int room = p.group - s0 % p.group;
    if (tid == 0) s_len = room;
    __syncthreads();
    for (int j = tid; j < room; j += kThreads)
      if (slot_at(p, t + j) != s0 + j) {
        atomicMin(&s_len, j);
        break;
      }
    __syncthreads();
    append_run<kThreads>(p, t, s0, s_len, tid, s_red);
    __syncthreads();  // s_len and s_red are free again
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (p.group <= kWarpGroup) {
    const unsigned ctas = (static_cast<unsigned>(p.num_tokens) + kThreads / 32 - 1) / (kThreads / 32);
    append_warp_kernel<<<ctas, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
  }
  // one token a CTA while that leaves at most about eight CTAs an SM, so that
  // the tokens of a decode step (a run each) spread over the SMs; more tokens
  // are taken in windows, whose CTAs mostly find one run of a prompt
  int window = (p.num_tokens + 1215) / 1216;
  if (window > kMaxWindow) window = kMaxWindow;
  const unsigned ctas = static_cast<unsigned>((p.num_tokens - 1) / window + 1);
  append_cta_kernel<<<ctas, kThreads, 0, stream>>>(p, window);
  return cudaGetLastError();
}

}  // namespace mla
