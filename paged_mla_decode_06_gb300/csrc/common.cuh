// common.cuh -- small device helpers shared by the decode, merge and index
// kernels: async copies, warp-level matrix loads and MMAs, exp2, packing.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace mla {

constexpr int kHeadDim = 576;      // c_kv (512) || k_pe (64)
constexpr int kRank = 512;         // value width
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16-byte global -> shared copy; src_bytes == 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src),
               "r"(src_bytes)
               : "memory");
}
// 4-byte global -> shared copy; src_bytes == 0 writes zeros and reads nothing.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t& r0, uint32_t& r1,
                                            uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x2(uint32_t addr, uint32_t& r0, uint32_t& r1) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];\n"
               : "=r"(r0), "=r"(r1)
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t& r0, uint32_t& r1,
                                                  uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// D += A * B, m16n8k16, fp32 accumulate. F16 selects f16 operands, else bf16.
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (F16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// 2^x on the special-function unit (ex2.approx; 2^-inf = 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (F16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  } else {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
}

// Two e4m3 codes (low byte first) -> two f16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

// Two weights as two code pairs: hi = e4m3(p) and lo, the rest p - hi, formed
// in f16 (p rounded to 11 bits first; the difference is then exact). The rest
// is taken as e4m3 (8 bits of p, nothing below 2^-10), as e5m2 (7 bits, down to
// 2^-17), or as 32 times it in e4m3, for products that are summed apart (8
// bits, down to 2^-15; the rest is at most 8 where p <= 2^8). The last two are
// for rows of which one key outweighs a long context: with p = 2^4 at the
// largest weight, keys 2^-14 below it would be left out of the first.
enum class Rest { kE4m3, kE5m2, kE4m3Times32 };
template <Rest R>
__device__ __forceinline__ void p_terms(float p0, float p1, uint32_t& hi, uint32_t& lo) {
  const __half2 ph = __floats2half2_rn(p0, p1);
  const uint32_t phb = *reinterpret_cast<const uint32_t*>(&ph);
  uint16_t h16, l16;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(h16) : "r"(phb));
  uint32_t back;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(back) : "h"(h16));
  __half2 d = __hsub2(ph, *reinterpret_cast<const __half2*>(&back));
  if constexpr (R == Rest::kE4m3Times32) d = __hmul2(d, __floats2half2_rn(32.f, 32.f));
  const uint32_t db = *reinterpret_cast<const uint32_t*>(&d);
  if constexpr (R == Rest::kE5m2)
    asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;\n" : "=h"(l16) : "r"(db));
  else
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;\n" : "=h"(l16) : "r"(db));
  hi = h16;
  lo = l16;
}

// Four weights (in order from the low byte) as two words of codes, the rest in
// e5m2.
__device__ __forceinline__ void p_terms4(float p0, float p1, float p2, float p3, uint32_t& hi, uint32_t& lo) {
  asm("{\n .reg .b16 h0, h1, l0, l1;\n .reg .b32 a, b, c, d;\n"
      " cvt.rn.f16x2.f32 a, %3, %2;\n cvt.rn.f16x2.f32 b, %5, %4;\n"
      " cvt.rn.satfinite.e4m3x2.f16x2 h0, a;\n cvt.rn.satfinite.e4m3x2.f16x2 h1, b;\n"
      " cvt.rn.f16x2.e4m3x2 c, h0;\n cvt.rn.f16x2.e4m3x2 d, h1;\n"
      " sub.f16x2 a, a, c;\n sub.f16x2 b, b, d;\n"
      " cvt.rn.satfinite.e5m2x2.f16x2 l0, a;\n cvt.rn.satfinite.e5m2x2.f16x2 l1, b;\n"
      " mov.b32 %0, {h0, h1};\n mov.b32 %1, {l0, l1};\n}\n"
      : "=r"(hi), "=r"(lo)
      : "f"(p0), "f"(p1), "f"(p2), "f"(p3));
}

// Values with their NaNs as zeros: four e4m3 codes, or two f16 values of codes
// (infinities do not occur). For the values of keys that some rows of a tile do
// not see: 0 times a NaN would reach those rows; a row that sees such a key is
// NaN by its score.
__device__ __forceinline__ uint32_t e4m3x4_without_nan(uint32_t w) {
  return w & ~__vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}
__device__ __forceinline__ uint32_t f16x2_without_nan(uint32_t w) {
  return w & ~__vcmpeq2(w & 0x7C007C00u, 0x7C007C00u);
}

// A key of a cache with group scales, as the softmax takes it. With s the
// group's scale, s2 the key's base-2 score factor times the raw score q . c
// (c the codes), and t = s2 s + log2 s, the weights 2^(t - m) multiply the
// codes themselves in P.V and, divided by s, sum to the denominator:
//   out = sum 2^(t - m) c / sum 2^(t - m) / s,  lse = ln 2 (m + log2 sum).
// So the values' scale costs one addition in the exponent, P.V keeps 8-bit
// operands, and the largest 2^(t - m) |c| of a row decides the range of P.
struct KeyScale {
  float mul;  // score factor times s
  float add;  // log2 s
  float inv;  // 1 / s
};
__device__ __forceinline__ KeyScale key_scale(float s, float score_scale_log2) {
  KeyScale k;
  k.mul = s * score_scale_log2;
  k.add = log2f(s);
  k.inv = 1.f / s;
  return k;
}

// The (max, sum) of a partial for the merge, which passes over sums that are not
// positive: a sum that is no number (a key or a query with a NaN) goes on as
// (inf, 1), whose weight in the merge is NaN, as the whole row's is.
__device__ __forceinline__ float2 partial_sums(float max, float sum) {
  return sum != sum ? make_float2(INFINITY, 1.f) : make_float2(max, sum);
}

__host__ __device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

}  // namespace mla
