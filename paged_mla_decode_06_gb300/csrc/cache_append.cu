// cache_append.cu -- a step's latent rows (c_kv || k_pe, bf16) into an e4m3
// cache with one fp32 scale for each group of g slots of a block.
//
// A run is a maximal stretch of consecutive tokens at consecutive slots of one
// group; its team (a warp for groups of at most 8 slots, else a CTA) is the
// only one that touches the group. With a the largest finite magnitude of the
// run's rows, the group's scale becomes
//   s = max(min(2^k, 2^60), 2^-60, s_old if the run starts behind rows of its
//       group),
// k the least integer with a <= 448 2^k, and the rows are stored as
// e4m3(x / s), saturating. (The decode weighs groups against each other in
// fp32, which scales within 2^60 of one on either side allow.) Where s grew,
// the rows before the run are requantised by s_old / s. Scales made here are
// powers of two, so that this changes no code but those that fall below e4m3's
// normal range. Those are rounded once more at each growth, by half of the
// smallest step of the scale of the time: however often a group grows, what is
// stored stays within one smallest step (2^-9 of the scale) of the row, where
// one rounding leaves half a step. (A floating-point format gains nothing from
// a finer scale but part of a binade of range.)
//
// What bounds it: memory, 1152 bytes read and 576 written a token, once a call
// is larger than its latency (slots, then rows, then codes: three trips). The
// rows of a run are read once and stay in registers between the maximum and
// the rounding; the rows of a longer run past those are read again, from L2.
// (16 prompts of 2047 tokens, groups of 64: 14.5 us, 3.9 TB/s of reads and
// writes; without either the same call takes 9.9 us. Asking for a CTA's rows in
// L2 before its slots are known 17.4 us; batches of 32 rows at more CTAs an SM,
// all but the last read twice, 15.4.)
// A CTA has four threads for each 16-byte piece of a row (4 x 72), so that a
// thread walks down one column with a constant stride, 16 pieces in flight for
// 64 rows; a warp, whose runs are short, takes the pieces row after row.
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kPieces = kHeadDim / 8;      // 16-byte bf16 pieces of a row: 64 latent, 8 rope
constexpr int kNopePieces = kRank / 8;
constexpr int kRowTeams = 4;               // CTA kernel: rows in work at a time
constexpr int kThreads = kRowTeams * kPieces;
constexpr int kHoldRows = 16;              // rows a thread of the CTA kernel keeps
constexpr int kWarpThreads = 256;          // warp kernel
constexpr int kWarpGroup = 8;              // largest group a warp takes
constexpr int kMaxWindow = 256;            // tokens of a CTA's window
constexpr int kSlotCache = 512;            // slots a CTA keeps in shared memory
constexpr int kMaxExp = 60;                // scales lie in [2^-60, 2^60]
constexpr int kWindowCtas = 2;             // CTAs an SM of a long call, once over (twice over:
                                           // 16 prompts of 2047 tokens 15.6 us against 14.5)

// Row t's piece (the caller's pointer to it advances by the part's stride).
struct Column {
  const __nv_bfloat16* base;
  int64_t stride;
  __device__ __forceinline__ Column(const AppendParams& p, int piece) {
    const bool nope = piece < kNopePieces;
    base = static_cast<const __nv_bfloat16*>(nope ? p.c_kv : p.k_pe) + (nope ? piece : piece - kNopePieces) * 8;
    stride = nope ? p.c_stride : p.pe_stride;
  }
  __device__ __forceinline__ uint4 at(int64_t t) const {
    return __ldg(reinterpret_cast<const uint4*>(base + t * stride));
  }
};

// Largest magnitudes of a piece, two columns at a time (NaN is passed over).
__device__ __forceinline__ __nv_bfloat162 piece_max(uint4 v, __nv_bfloat162 m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w[i])));
  return m;
}
// The same over the finite values alone.
__device__ __noinline__ uint32_t piece_max_finite(uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
    if (a < 0x7F80u) m = max(m, a);
  }
  return m;
}
// The larger of the two, as bf16 bits (NaN, where there is nothing else, as 0).
__device__ __forceinline__ uint32_t max_bits(__nv_bfloat162 m) {
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&m) & 0x7FFF7FFFu;
  const uint32_t lo = b & 0xFFFFu, hi = b >> 16;
  return max(lo > 0x7F80u ? 0u : lo, hi > 0x7F80u ? 0u : hi);
}

// The power of two that brings a bf16 magnitude (its bits) to 448 or below,
// within the range of scales: 448 = 1.75 * 2^8, and the mantissa of 1.75 is 0x60.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  int e = static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7Fu) > 0x60u ? 1 : 0);
  e = min(max(e, -kMaxExp), kMaxExp);
  return __int_as_float((e + 127) << 23);
}

// Eight bf16 values, times inv, as e4m3 codes.
__device__ __forceinline__ uint2 quantise(uint4 v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint16_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n .reg .b32 a, b;\n .reg .b64 x, y;\n shl.b32 a, %1, 16;\n and.b32 b, %1, 0xffff0000;\n"
        " mov.b64 x, {a, b};\n mov.b64 y, {%2, %2};\n mul.rn.f32x2 x, x, y;\n mov.b64 {a, b}, x;\n"
        " cvt.rn.satfinite.e4m3x2.f32 %0, b, a;\n}\n"
        : "=h"(c[i])
        : "r"(w[i]), "f"(inv));
  return make_uint2(c[0] | (static_cast<uint32_t>(c[1]) << 16), c[2] | (static_cast<uint32_t>(c[3]) << 16));
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

// The rows of the group before the run, from scale `old` to scale `s`, by
// `threads` threads.
__device__ __noinline__ void requantise_head(const AppendParams& p, int s0, int before, float ratio, int tr, int threads) {
  uint4* head = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.cache) +
                                         static_cast<int64_t>(s0 - before) * kHeadDim);
  for (int i = tr; i < before * (kHeadDim / 16); i += threads) {
    uint4 c = head[i];
    c.x = requantise(c.x, ratio);
    c.y = requantise(c.y, ratio);
    c.z = requantise(c.z, ratio);
    c.w = requantise(c.w, ratio);
    head[i] = c;
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

// Groups of at most kWarpGroup slots: a warp per token; those that start a
// run work. HOLD pieces a lane cover the longest run of the group size.
template <int HOLD>
__global__ void __launch_bounds__(kWarpThreads) append_warp_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kWarpThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.num_tokens) return;
  const int g = p.group;
  const int mine = slot_at(p, t - 1 + lane);  // lane 0: the token before
  const int s0 = __shfl_sync(0xffffffffu, mine, 1);
  const int prev = __shfl_sync(0xffffffffu, mine, 0);
  if (!starts_run(prev, s0, g)) return;
  const int before = s0 % g;  // rows of the group that are there already
  const uint32_t same = __ballot_sync(0xffffffffu, lane >= 1 && lane - 1 < g - before && mine == s0 + lane - 1);
  const int n = __ffs(~(same >> 1)) - 1;  // consecutive slots from the first
  const int pieces = n * kPieces;
  const float old = before > 0 ? p.scales[s0 / g] : 0.f;
  uint4 v[HOLD];
  __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < HOLD; ++j) {
    const int i = j * 32 + lane;
    v[j] = make_uint4(0u, 0u, 0u, 0u);
    if (i < pieces) v[j] = Column(p, i % kPieces).at(t + i / kPieces);
  }
#pragma unroll
  for (int j = 0; j < HOLD; ++j) m2 = piece_max(v[j], m2);
  uint32_t m = __reduce_max_sync(0xffffffffu, max_bits(m2));
  if (m == 0x7F80u) {  // an infinity among them: the largest finite value instead
    m = 0u;
#pragma unroll 1
    for (int i = lane; i < pieces; i += 32) m = piece_max_finite(Column(p, i % kPieces).at(t + i / kPieces), m);
    m = __reduce_max_sync(0xffffffffu, m);
  }
  const float s = fmaxf(scale_of(m), old);
  const float inv = 1.f / s;
  uint8_t* rows = static_cast<uint8_t*>(p.cache) + static_cast<int64_t>(s0) * kHeadDim;
  if (lane == 0) p.scales[s0 / g] = s;
#pragma unroll
  for (int j = 0; j < HOLD; ++j) {
    const int i = j * 32 + lane;
    if (i < pieces) *reinterpret_cast<uint2*>(rows + i * 8) = quantise(v[j], inv);
  }
  if (before > 0 && s > old) requantise_head(p, s0, before, old / s, lane, 32);
}

// Larger groups: a CTA per window of tokens takes the runs that start in it.
__global__ void __launch_bounds__(kThreads, 2) append_cta_kernel(const AppendParams p, int window) {
  __shared__ int s_slot[kSlotCache];            // slots of tokens w0 - 1, w0, ...
  __shared__ uint32_t s_red[2][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = p.group;
  const int w0 = blockIdx.x * window;
  const int cached = min(window + g, kSlotCache);
  for (int i = tid; i < cached; i += kThreads) s_slot[i] = slot_at(p, w0 - 1 + i);
  const int piece = tid % kPieces, team = tid / kPieces;
  const Column col(p, piece);
  __syncthreads();
  int turn = 0;
  uint32_t starts = 0u;  // of the 32 tokens from `base` (every warp looks for itself)
  for (int base = 0, next = 0;;) {
    while (starts == 0u && next < window) {
      base = next;
      next += 32;
      const int j = base + lane;
      starts = __ballot_sync(0xffffffffu, j < window && starts_run(s_slot[j], s_slot[j + 1], g));
    }
    if (starts == 0u) break;
    const int i = base + __ffs(starts) - 1;
    starts &= starts - 1u;
    const int s0 = s_slot[i + 1];
    const int t = w0 + i;
    const int before = s0 % g;  // rows of the group that are there already
    const float old = before > 0 ? p.scales[s0 / g] : 0.f;
    // consecutive slots from the first (every warp counts for itself)
    int n = 1;
    for (bool all = true; all && n < g - before;) {
      const int j = n + lane;
      const bool in = j < g - before && (i + 1 + j < cached ? s_slot[i + 1 + j] : slot_at(p, t + j)) == s0 + j;
      const uint32_t b = __ballot_sync(0xffffffffu, in);
      all = b == 0xffffffffu;
      n += all ? 32 : __ffs(~b) - 1;
    }
    uint4 v[kHoldRows];
#pragma unroll
    for (int j = 0; j < kHoldRows; ++j) {
      const int r = j * kRowTeams + team;
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (r < n) v[j] = col.at(t + r);
    }
    __nv_bfloat162 m2 = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kHoldRows; ++j) m2 = piece_max(v[j], m2);
    for (int r = kHoldRows * kRowTeams + team; r < n; r += kRowTeams) m2 = piece_max(col.at(t + r), m2);
    auto all_max = [&](uint32_t mine) {
      mine = __reduce_max_sync(0xffffffffu, mine);
      if (lane == 0) s_red[turn & 1][warp] = mine;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) mine = max(mine, s_red[turn & 1][w]);
      ++turn;
      return mine;
    };
    uint32_t m = all_max(max_bits(m2));
    if (m == 0x7F80u) {  // an infinity among them: the largest finite value instead
      uint32_t f = 0u;
#pragma unroll 1
      for (int r = team; r < n; r += kRowTeams) f = piece_max_finite(col.at(t + r), f);
      m = all_max(f);
    }
    const float s = fmaxf(scale_of(m), old);
    const float inv = 1.f / s;
    uint8_t* dst = static_cast<uint8_t*>(p.cache) + static_cast<int64_t>(s0) * kHeadDim + piece * 8;
    if (tid == 0) p.scales[s0 / g] = s;
#pragma unroll
    for (int j = 0; j < kHoldRows; ++j) {
      const int r = j * kRowTeams + team;
      if (r < n) *reinterpret_cast<uint2*>(dst + r * kHeadDim) = quantise(v[j], inv);
    }
    for (int r = kHoldRows * kRowTeams + team; r < n; r += kRowTeams)
      *reinterpret_cast<uint2*>(dst + static_cast<int64_t>(r) * kHeadDim) = quantise(col.at(t + r), inv);
    if (before > 0 && s > old) requantise_head(p, s0, before, old / s, tid, kThreads);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendParams& p, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (p.group <= kWarpGroup) {
    constexpr int kPer = kWarpThreads / 32;
    const unsigned ctas = (static_cast<unsigned>(p.num_tokens) + kPer - 1) / kPer;
    if (p.group == 1)
      append_warp_kernel<3><<<ctas, kWarpThreads, 0, stream>>>(p);  // 72 pieces
    else if (p.group <= 4)
      append_warp_kernel<9><<<ctas, kWarpThreads, 0, stream>>>(p);  // 4 rows
    else
      append_warp_kernel<18><<<ctas, kWarpThreads, 0, stream>>>(p);  // 8 rows
    return cudaGetLastError();
  }
  // one token a CTA while there are few, so that the tokens of a decode step
  // (a run each) spread over the SMs; more tokens are taken in windows, whose
  // CTAs mostly find one run of a prompt
  int sms = 0;
  const cudaError_t e = device_sms(&sms);
  if (e != cudaSuccess) return e;
  int window = (p.num_tokens - 1) / (kWindowCtas * sms) + 1;
  if (window > kMaxWindow) window = kMaxWindow;
  const unsigned ctas = static_cast<unsigned>((p.num_tokens - 1) / window + 1);
  append_cta_kernel<<<ctas, kThreads, 0, stream>>>(p, window);
  return cudaGetLastError();
}

}  // namespace mla
