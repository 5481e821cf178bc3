// rope.cu -- rotary positions of a step's queries and keys, with the q
// pre-step of the decode (q = ql_nope || rotated q_pe, bf16 or e4m3) in the same
// pass. Pair i of a rope part turns by the angle p f_i of its token's position:
//   y_a = (x_a cos - x_b sin) m,   y_b = (x_b cos + x_a sin) m,
// (a, b) = (2 i, 2 i + 1) or (i, i + dim / 2), m the factor of a stretched
// context; columns from `dim` on pass. The plan holds f_i in turns, and p f_i is
// formed and reduced to [-1/2, 1/2] in 64 bits: at positions of millions an fp32
// angle is off by tenths of a radian. One rounding, to the output type.
//
// Bound by the bytes: 1152 in and 576 or 1152 out a row. A warp takes one token
// and kBatch heads at a time: lane l holds columns 2 l and 2 l + 1 of a
// rope part (a column's partner comes by one shuffle, whatever dim is) and two
// 16-byte pieces of each latent part, so that its cosines and sines are made
// once, in registers, and the loads of kBatch heads are in flight together while
// they are. (Angles of both of a lane's columns are made even where they are one pair's:
// the two do not show beside the loads.)
//
// Measured: 8191 tokens of 16 heads to bf16 47.7 us, 6.4 TB/s (0.94 of the copy rate); 64 of
// 128 heads to e4m3 4.8 us in a captured graph, of which 2.0 are its 13.5 MB and the rest
// the chain of position, angle, rows.
#include "common.cuh"
#include "internal.h"

namespace mla {
namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 4;  // heads a warp loads at once

struct Turn {
  float cos0, sin0, cos1, sin1;  // of the lane's columns; the sine with its column's sign
  int from0, from1;              // the partner columns
};

__device__ __forceinline__ void turn_of(const RopeParams& p, int pos, int col, float* c, float* s, int* from) {
  *c = 1.f;
  *s = 0.f;
  *from = col;
  if (col >= p.dim) return;
  const int half = p.dim >> 1;
  const int i = p.half ? (col < half ? col : col - half) : col >> 1;
  const bool second = p.half ? col >= half : (col & 1) != 0;
  *from = p.half ? (second ? col - half : col + half) : col ^ 1;
  const double t = static_cast<double>(pos) * p.turns[i];
  float sn, cs;
  sincospif(2.f * static_cast<float>(t - rint(t)), &sn, &cs);
  *c = cs * p.mscale;
  *s = (second ? sn : -sn) * p.mscale;
}

// The rotated columns 2 lane and 2 lane + 1 of the row whose words the lanes hold.
__device__ __forceinline__ float2 rotate(uint32_t w, const Turn& t) {
  const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  const uint32_t a = __shfl_sync(0xffffffffu, w, t.from0 >> 1);
  const uint32_t b = __shfl_sync(0xffffffffu, w, t.from1 >> 1);
  // a bf16 value is the upper half of its fp32
  const float y0 = __uint_as_float((t.from0 & 1) != 0 ? a & 0xffff0000u : a << 16);
  const float y1 = __uint_as_float((t.from1 & 1) != 0 ? b & 0xffff0000u : b << 16);
  // a column without a partner (beyond dim) is itself, NaN and infinities too
  float2 r;
  const int col = 2 * static_cast<int>(threadIdx.x & 31);
  r.x = t.from0 == col ? x.x : fmaf(y0, t.sin0, x.x * t.cos0);
  r.y = t.from1 == col + 1 ? x.y : fmaf(y1, t.sin1, x.y * t.cos1);
  return r;
}

__device__ __forceinline__ uint32_t to_bf16x2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ uint32_t to_e4m3x2(float2 v, float inv) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(v.x * inv, v.y * inv), __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint2 quant8(uint4 v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) c[k] = to_e4m3x2(__bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[k])), inv);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

template <bool FP8>
__global__ void __launch_bounds__(kWarps * 32) rope_kernel(const __grid_constant__ RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t t = w / p.shares;
  const int share = static_cast<int>(w - t * p.shares);
  if (t >= p.num_tokens) return;
  const int pos = p.positions[t];
  if (pos < 0) return;  // padding: its rows stay as they were
  const int h0 = share * p.share_heads, h1 = min(h0 + p.share_heads, p.num_heads);
  const __nv_bfloat16* nope = static_cast<const __nv_bfloat16*>(p.nope) + t * p.nope_st;
  const __nv_bfloat16* pe = static_cast<const __nv_bfloat16*>(p.pe) + t * p.pe_st;
  const bool keys = p.k_pe != nullptr && share == 0;
  uint32_t kw = 0u;
  if (keys) kw = *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.k_pe) + t * p.k_st + 2 * lane);
  uint4 v[kBatch][2];
  uint32_t r[kBatch];
  auto load = [&](int h) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (h + b >= h1) {
        r[b] = 0u;
        continue;
      }
      const uint4* row = reinterpret_cast<const uint4*>(nope + (h + b) * p.nope_sh);
      v[b][0] = __ldg(row + lane);
      v[b][1] = __ldg(row + 32 + lane);
      r[b] = __ldg(reinterpret_cast<const uint32_t*>(pe + (h + b) * p.pe_sh) + lane);
    }
  };
  load(h0);
  Turn tn;
  turn_of(p, pos, 2 * lane, &tn.cos0, &tn.sin0, &tn.from0);
  turn_of(p, pos, 2 * lane + 1, &tn.cos1, &tn.sin1, &tn.from1);
  if (keys) {
    const float2 y = rotate(kw, tn);
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.k_out) + t * p.k_out_st + 2 * lane) = to_bf16x2(y);
  }
  for (int h = h0; h < h1; h += kBatch) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const float2 y = rotate(r[b], tn);  // (all lanes: shuffles)
      if (h + b >= h1) continue;
      const int64_t row = t * p.num_heads + h + b;
      if constexpr (FP8) {
        uint8_t* out = static_cast<uint8_t*>(p.out) + row * kHeadDim;
        *reinterpret_cast<uint2*>(out + 8 * lane) = quant8(v[b][0], p.q_inv);
        *reinterpret_cast<uint2*>(out + 256 + 8 * lane) = quant8(v[b][1], p.q_inv);
        *reinterpret_cast<uint16_t*>(out + kRank + 2 * lane) = static_cast<uint16_t>(to_e4m3x2(y, p.q_inv));
      } else {
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row * kHeadDim;
        reinterpret_cast<uint4*>(out)[lane] = v[b][0];
        reinterpret_cast<uint4*>(out)[32 + lane] = v[b][1];
        *reinterpret_cast<uint32_t*>(out + kRank + 2 * lane) = to_bf16x2(y);
      }
    }
    if (h + kBatch < h1) load(h + kBatch);
  }
}

}  // namespace

cudaError_t launch_rope(RopeParams p, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  // kBatch heads a warp while that leaves the GPU unfilled, twice that where rows
  // abound (fewer angles a row)
  const int64_t batches = (p.num_heads + kBatch - 1) / kBatch;
  p.share_heads = batches * p.num_tokens > 32768 ? 2 * kBatch : kBatch;
  p.shares = p.num_heads > 0 ? (p.num_heads + p.share_heads - 1) / p.share_heads : 1;
  const int64_t ctas = (static_cast<int64_t>(p.num_tokens) * p.shares + kWarps - 1) / kWarps;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  if (p.fp8)
    rope_kernel<true><<<static_cast<unsigned>(ctas), kWarps * 32, 0, stream>>>(p);
  else
    rope_kernel<false><<<static_cast<unsigned>(ctas), kWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
