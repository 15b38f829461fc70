// lowbit.cuh -- device helpers of the low-bit weight and cache kernels (w4.cu, kv.cu, attn.cu): the
// quantisation rule of a group, the storage of 4-bit codes, their way into the tensor cores' operands.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace imq {

// ------------------------------------------------------------------------------------------------
// quantisation of one group: imq_rtn_quantize's rule with p = 1 (q = max |x|)
// ------------------------------------------------------------------------------------------------
// The bits of |x| order like unsigned integers, infinities and NaNs above every finite value, so one
// integer maximum finds q and any non-finite entry.
__device__ __forceinline__ uint32_t abs_key(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
__device__ __forceinline__ bool key_finite(uint32_t key) { return key < 0x7F800000u; }

// s = beta / q and the step q / beta, correctly rounded.  A group of zeros, or one so small that s would
// leave fp32, takes s = step = 1 (its codes are 0); a non-finite group's step is NaN.
__device__ __forceinline__ void group_scale(uint32_t key, float beta, float* s, float* step) {
  const float q = __uint_as_float(key);
  if (!key_finite(key)) {
    *s = 0.f;
    *step = __uint_as_float(0x7FC00000u);
    return;
  }
  *s = __fdiv_rn(beta, q);
  *step = __fdiv_rn(q, beta);
  if (q == 0.f || !key_finite(__float_as_uint(*s))) *s = *step = 1.f;
}

// Four different groups' scales with one division each way instead of four: every lane of four works out one group's
// and hands it to the others.  All lanes of an aligned quad hold the same four keys.
__device__ __forceinline__ void four_scales(const uint32_t (&key)[4], float beta, float (&s)[4], float (&step)[4]) {
  const int j = threadIdx.x & 3;
  float one_s, one_step;
  group_scale(j < 2 ? (j == 0 ? key[0] : key[1]) : (j == 2 ? key[2] : key[3]), beta, &one_s, &one_step);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s[i] = __shfl_sync(0xffffffffu, one_s, i, 4);
    step[i] = __shfl_sync(0xffffffffu, one_step, i, 4);
  }
}

// A code in the low bits of a float: round_half_even(fp32(x * s)) + bias on top of 0x4B400000, for |x * s| <= 128 and
// an even bias.  (Adding 1.5 * 2^23 rounds to an integer in the low mantissa bits; |x| <= q, so |fp32(x * s)| is at
// most beta but for the rounding of s, well below beta + 1/2.)
__device__ __forceinline__ uint32_t code_bits(float x, float s, float bias) {
  return __float_as_uint(__fadd_rn(__fmul_rn(x, s), 12582912.f + bias));
}
// Eight 4-bit codes in a word: code e in bits 4 * (e / 2 + 4 * (e % 2)), so that one mask leaves the codes 2i and
// 2i + 1 in the two halves of a register.  The codes are added up where they belong, and what the upper bits of
// their floats add up to is taken off.  s = 0 marks a non-finite group: its codes are 0 whatever x is.
__device__ __forceinline__ uint32_t pack4(const float (&x)[8], float s) {
  uint32_t w = 0u - 0x4B400000u * 0x11111111u;
#pragma unroll
  for (int e = 0; e < 8; ++e) w += code_bits(x[e], s, 8.f) << (4 * (e / 2 + 4 * (e % 2)));
  return s == 0.f ? 0x88888888u : w;
}
// Four 8-bit codes in a word.
__device__ __forceinline__ uint32_t pack8(float x0, float x1, float x2, float x3, float s) {
  const uint32_t w = code_bits(x0, s, 128.f) + (code_bits(x1, s, 128.f) << 8) + (code_bits(x2, s, 128.f) << 16) +
                     (code_bits(x3, s, 128.f) << 24) - 0x4B400000u * 0x01010101u;
  return s == 0.f ? 0x80808080u : w;
}

// ------------------------------------------------------------------------------------------------
// element types
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Eight consecutive entries, 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]), bf16_pair(x[4], x[5]),
                                            bf16_pair(x[6], x[7]));
}

// ------------------------------------------------------------------------------------------------
// warp-level tensor-core products, fp32 sums: D (16 x 8) += A (16 x 16) * B (16 x 8).  With g = lane / 4
// and c = lane % 4: a0, a2 are row g at inner positions 2c, 2c+1 and 2c+8, 2c+9; a1, a3 row g + 8; b0, b1
// column g at the same positions; d0, d1 row g and d2, d3 row g + 8 at columns 2c, 2c+1.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Signed by unsigned bytes, 32-bit integer sums: D += A (16 x 32) * B (32 x 8); a0 / b0 hold inner positions
// 4c .. 4c + 3 and a2 / b1 16 + 4c .. + 3, a byte each; a1, a3 row g + 8.
__device__ __forceinline__ void mma_s8u8(int32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes as fp16 or bf16 pairs without integer-to-float conversions: a code's bits are set into the mantissa
// of a power of two, where they count in units of one (or of 16), and the offset is subtracted; every step
// is exact.
__device__ __forceinline__ uint32_t h2_sub(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t h2_fma(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b),
                            *reinterpret_cast<const __half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// `one` is the power of two in both halves.  It comes from the kernel's arguments: an instruction has room for one
// constant, and the compiler, knowing both, would spend a second instruction on each pair of codes.
constexpr uint32_t kOneF16 = 0x64006400u;   // 1024
constexpr uint32_t kOneBf16 = 0x43004300u;  // 128
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t mask, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(mask), "r"(b));
  return r;
}
// fp16 pair of the 4-bit codes in bits 0-3 of each half (and with kHigh in bits 4-7).
template <bool kHigh>
__device__ __forceinline__ uint32_t nibbles_f16(uint32_t w, uint32_t one) {
  if (kHigh) return h2_fma(and_or(w, 0x00F000F0u, one), 0x2C002C00u /* 1/16 */, 0xD480D480u /* -72 */);
  return h2_sub(and_or(w, 0x000F000Fu, one), 0x64086408u /* 1032 */);
}
// fp16 pair of the 8-bit codes in the bytes of x that `sel` names (0-3), as a __byte_perm selector 0x5y5x (5: the high byte of
// `one`).
__device__ __forceinline__ uint32_t bytes_f16(uint32_t x, uint32_t sel, uint32_t one) {
  return h2_sub(__byte_perm(x, one, sel), 0x64806480u /* 1152 */);
}
// Codes 2i and 2i + 1 of a word of eight 4-bit codes, and bytes 2i and 2i + 1 of a word, as fp32.
__device__ __forceinline__ float2 nibble_pair(uint32_t w, int i, uint32_t one) {
  const uint32_t h = i == 0   ? nibbles_f16<false>(w, one)
                     : i == 1 ? nibbles_f16<true>(w, one)
                     : i == 2 ? nibbles_f16<false>(w >> 8, one)
                              : nibbles_f16<true>(w >> 8, one);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float2 byte_pair(uint32_t w, int i, uint32_t one) {
  const uint32_t h = bytes_f16(w, i == 0 ? 0x5150 : 0x5352, one);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// bf16 pair of the 4-bit codes in bits 0-3 of each half.
__device__ __forceinline__ uint32_t nibbles_bf16(uint32_t w, uint32_t one) {
  const uint32_t v = and_or(w, 0x000F000Fu, one);
  const uint32_t k = 0x43084308u;  // 136
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&k));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Two 8 x 8 blocks of 16-bit elements and the next two, transposed on the way: lane i gives the address of row
// i % 8 of block i / 8 (16 bytes), and gets of each block the elements of rows 2c and 2c + 1 in column g.
__device__ __forceinline__ void ldmatrix_trans4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// ------------------------------------------------------------------------------------------------
// asynchronous copies, each thread's own bytes
// ------------------------------------------------------------------------------------------------
template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
// src_bytes 0 writes zeros and reads nothing.
template <int kBytes>
__device__ __forceinline__ void cp_async_part(uint32_t dst, const void* src, uint32_t src_bytes) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(src_bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

}  // namespace imq
