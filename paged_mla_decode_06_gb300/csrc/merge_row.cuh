// merge_row.cuh -- one warp merges the base-2 partials of one (token, head)
// row into its bf16 output and natural-log LSE (rocm_aiter_mla_merge page,
// merge_mla_segments_triton): partial s sits at index base + s * stride of
// the max / expsum arrays and at that index times the row width in the
// outputs.
// Partials with expsum > 0 take part with weight l_s * 2^(m2_s - M), M the
// largest of their maxima and the sink's base-2 logit; the sink adds
// 2^(sink2 - M) to the denominator only. A row with no mass gets zeros and
// -inf. Coherent selects L2 loads (partials written by other CTAs of the
// same grid) instead of the read-only path.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"

namespace mla {

// The end of a row that the merge has nothing to do for. The decode lets its merge
// launch early, and what follows the merge on the stream, or in a captured graph,
// waits for the merge alone: a grid that ended without waiting for the decode would
// let it run while the decode still writes. So the first block, whose first warp
// always has a row, waits before it leaves. (The others need not: rows that leave
// make room for those that wait.)
__device__ __forceinline__ void leave_merge() {
  if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

template <bool Coherent>
__device__ __forceinline__ float4 merge_load(const float4* p) {
  if constexpr (Coherent) return __ldcg(p);
  else return __ldg(p);
}

template <bool Coherent>
__device__ __forceinline__ float merge_load_f(const float* p) {
  if constexpr (Coherent) return __ldcg(p);
  else return __ldg(p);
}

// Rows of WIDTH * 128 values, of which this warp merges the `slice`-th VPL *
// 128: lane i handles float4 i, i + 32, ... . The (max, expsum) pairs of the
// first kMeta partials are loaded together and kept; the outputs of four
// partials at a time are loaded together, so that a row costs about two memory
// round trips. Further pairs are loaded by 32 lanes at a time, and each lane
// forms one's weight; the sums are in the order of the partials either way.
constexpr int kMeta = 8;

template <int VPL, int WIDTH, bool Coherent>
__device__ void merge_row(const float* segm_out, const float* segm_max, const float* segm_expsum,
                          int64_t base, int64_t stride, int live, float sink2, __nv_bfloat16* out,
                          float* lse, int lane, int slice) {
  const int first = slice * VPL * 32 + lane;  // float4
  constexpr int kBatch = VPL == 1 ? 16 : 4;
  float lk[kMeta], mk[kMeta];
#pragma unroll
  for (int u = 0; u < kMeta; ++u) {
    lk[u] = u < live ? merge_load_f<Coherent>(segm_expsum + base + u * stride) : 0.f;
    mk[u] = u < live ? merge_load_f<Coherent>(segm_max + base + u * stride) : -INFINITY;
  }
  // the outputs of the first four partials are loaded with no wait for their
  // weights (one memory round trip instead of two); a partial that carries
  // no mass (possibly never written: stale or NaN) is excluded by select
  float4 x0[4][VPL];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const float4* src = reinterpret_cast<const float4*>(segm_out + (base + u * stride) * (WIDTH * 128));
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      x0[u][v] = u < live ? merge_load<Coherent>(src + v * 32 + first) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  float M = sink2;
#pragma unroll
  for (int u = 0; u < kMeta; ++u)
    if (lk[u] > 0.f) M = fmaxf(M, mk[u]);
  for (int s = kMeta + lane; s - lane < live; s += 32) {
    const int64_t i = base + s * stride;
    const float l = s < live ? merge_load_f<Coherent>(segm_expsum + i) : 0.f;
    const float m = s < live ? merge_load_f<Coherent>(segm_max + i) : -INFINITY;
    if (l > 0.f) M = fmaxf(M, m);
  }
  if (live > kMeta) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  }
  float acc[VPL][4];
#pragma unroll
  for (int v = 0; v < VPL; ++v) acc[v][0] = acc[v][1] = acc[v][2] = acc[v][3] = 0.f;
  float W = 0.f;
  if (M == -INFINITY) {
#pragma unroll
    for (int v = 0; v < VPL; ++v)
      *reinterpret_cast<uint2*>(out + (v * 32 + first) * 4) = make_uint2(0u, 0u);
    if (first == 0) *lse = -INFINITY;
    return;
  }
  auto weight = [&](float l, float m) { return l > 0.f ? l * exp2f(m - M) : 0.f; };
  auto add = [&](float wu, const float4 (&xu)[VPL]) {
    W += wu;
    if (wu != 0.f) {
#pragma unroll
      for (int v = 0; v < VPL; ++v) {
        acc[v][0] += wu * xu[v].x;
        acc[v][1] += wu * xu[v].y;
        acc[v][2] += wu * xu[v].z;
        acc[v][3] += wu * xu[v].w;
      }
    }
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) add(weight(lk[u], mk[u]), x0[u]);
  // the outputs of `count` partials from s0, of weights w
  auto add_batch = [&](int s0, const auto& w, auto count) {
    constexpr int kCount = decltype(count)::value;
    float4 x[kCount][VPL];
#pragma unroll
    for (int u = 0; u < kCount; ++u) {
      const float4* src = reinterpret_cast<const float4*>(segm_out + (base + (s0 + u) * stride) * (WIDTH * 128));
#pragma unroll
      for (int v = 0; v < VPL; ++v)
        x[u][v] = w[u] != 0.f ? merge_load<Coherent>(src + v * 32 + first) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < kCount; ++u) add(w[u], x[u]);
  };
  if (live > 4) {
    float w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = weight(lk[4 + u], mk[4 + u]);
    add_batch(4, w, std::integral_constant<int, 4>{});
  }
  for (int s0 = kMeta; s0 < live; s0 += 32) {
    const int s = s0 + lane;
    const float l = s < live ? merge_load_f<Coherent>(segm_expsum + base + s * stride) : 0.f;
    const float m = s < live ? merge_load_f<Coherent>(segm_max + base + s * stride) : -INFINITY;
    const float mine = weight(l, m);
    for (int k = 0; k < 32 && s0 + k < live; k += kBatch) {
      float w[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) w[u] = __shfl_sync(0xffffffffu, mine, k + u);
      add_batch(s0 + k, w, std::integral_constant<int, kBatch>{});
    }
  }
  if (sink2 != -INFINITY) W += exp2f(sink2 - M);
  const float inv = 1.f / W;
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    __nv_bfloat162 lo = __floats2bfloat162_rn(acc[v][0] * inv, acc[v][1] * inv);
    __nv_bfloat162 hi = __floats2bfloat162_rn(acc[v][2] * inv, acc[v][3] * inv);
    *reinterpret_cast<uint2*>(out + (v * 32 + first) * 4) =
        make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
  }
  if (first == 0) *lse = kLn2 * (M + log2f(W));
}

}  // namespace mla
