// fp4idx_attention_common.cuh -- what the operators of
// include/fp4idx_attention.h share: checks of the cache block, conversions
// between E4M3 codes and 16-bit elements, and small PTX wrappers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "fp4idx_attention.h"
#include "fp4idx_common.cuh"

namespace fp4idx_impl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

inline bool aligned(const void* p, uintptr_t n) {
  return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}

// The checks of a cache block that every call makes.
inline fp4idx_status check_cache(const fp4idx_kv_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return FP4IDX_ERR_NULL;
  if (c->kv_heads < 1 || c->kv_heads > 65535 || (c->head_dim != 64 && c->head_dim != 128) ||
      c->num_blocks < 1 || c->num_blocks >= (1ll << 31) ||
      c->code_block_stride < (int64_t)c->kv_heads * FP4IDX_KV_BLOCK * c->head_dim ||
      c->code_block_stride > (1ll << 62) / c->num_blocks || c->scale_block_stride < c->kv_heads ||
      c->scale_block_stride > (1ll << 59) / c->num_blocks)
    return FP4IDX_ERR_SHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4) || c->code_block_stride % 16)
    return FP4IDX_ERR_ALIGN;
  return FP4IDX_OK;
}

inline bool dtype_ok(int dtype) { return dtype == FP4IDX_BF16 || dtype == FP4IDX_FP16; }

// The two 16-bit elements of a word as fp32.
template <bool kHalf>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (kHalf)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return make_float2(bf16_lo(w), bf16_hi(w));
}

// An fp32 pair rounded to two 16-bit elements (lo in bits 0..15).
template <bool kHalf>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (kHalf) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return pack_bf16x2(lo, hi);
  }
}

// The same with the type chosen at run time (uniform, off the inner loops).
__device__ __forceinline__ float2 unpack16(int half, uint32_t w) {
  return half ? unpack16<true>(w) : unpack16<false>(w);
}
__device__ __forceinline__ uint32_t pack16(int half, float lo, float hi) {
  return half ? pack16<true>(lo, hi) : pack16<false>(lo, hi);
}

// Two E4M3 codes (low and high byte) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

// The four E4M3 codes of a word as fp16 pairs: (0, 1) and (2, 3).
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t c, uint32_t& lo, uint32_t& hi) {
  lo = e4m3x2_to_f16x2((uint16_t)c);
  hi = e4m3x2_to_f16x2((uint16_t)(c >> 16));
}

// 16 bytes read once: not kept in L1.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 2^x, flushing results below 2^-126 to zero.
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The biased exponent of the scale of a block whose largest magnitude is
// amax: ceil_pow2(max(rn32(amax / 448), 2^-126)), within [1, 254].
__device__ __forceinline__ uint32_t block_scale_exp(float amax) {
  const uint32_t b = __float_as_uint(fmaxf(__fdiv_rn(amax, 448.0f), 1.17549435e-38f));
  const uint32_t e = (b >> 23) + ((b & 0x7fffffu) != 0u);
  return e > 254u ? 254u : e;
}

// 2^(127 - e), the exact inverse of the scale with biased exponent e >= 1.
__device__ __forceinline__ float inv_scale(uint32_t e) {
  return e == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - e) << 23);
}

}  // namespace fp4idx_impl
