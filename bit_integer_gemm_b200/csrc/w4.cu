// w4.cu -- weights of 4 bits with a step per group of inputs: quantiser, its inverse, and the product of a
// few tokens with such a weight (sm_100a).
//
// Storage of output channel n (a row): K inputs in blocks of 128, 64 bytes each; input r of a block is code
// e = r % 8 of word 4 * ((r % 32) / 8) + r / 32 of the block's 16.  A lane that takes the 16 bytes at
// 16 * c of a block holds the inputs 32h + 8c .. 32h + 8c + 7 for h = 0..3: one word per 32 inputs, so a
// group of 32 ends at a word, and the inputs it needs from a token are 16 contiguous bytes of bf16 per word.
#include "lowbit.cuh"
#include "internal.h"

namespace imq {
namespace {

constexpr int kBlock = 128;      // inputs of a storage block
constexpr int kBlockBytes = 64;

// Word of a block that holds its inputs 8i .. 8i + 7.
__device__ __forceinline__ int word_of(int i) { return 4 * (i & 3) + (i >> 2); }

struct QuantArgs {
  const void* W;
  int64_t K, N, ldw;
  uint8_t* codes;
  int64_t ldc;
  float* steps;
  int64_t lds;
  int group;
  int aligned;  // rows of W may be read 16 bytes at a time
  int32_t* status;
};

// Quantises the 8 entries x of lane's part of a block: `lanes` lanes (4, 8 or 16, aligned) share a group.
// Returns the packed word; *step is the group's.
__device__ __forceinline__ uint32_t quantise_word(const float (&x)[8], int lanes, float* step, bool* bad) {
  uint32_t key = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) key = max(key, abs_key(x[e]));
  for (int o = 1; o < lanes; o <<= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  float s;
  group_scale(key, 7.f, &s, step);
  *bad = !key_finite(key);
  uint32_t u[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) u[e] = code_of(x[e], s, 8u) & 15u;
  return pack_nibbles(u);
}

// W stored N x K: half a warp takes a block of 128 inputs of one row, 8 inputs a lane.
template <typename T>
__global__ void __launch_bounds__(256) k_w4_quantize_rows(QuantArgs a) {
  const int64_t nb = (a.K + kBlock - 1) / kBlock;
  const int lane = threadIdx.x & 31, i = lane & 15;
  const int64_t unit = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * 2 + (lane >> 4);
  const int64_t total = a.N * nb;
  const bool live = unit < total;
  const int64_t n = live ? unit / nb : 0, kb = live ? unit % nb : 0;
  const int64_t k0 = kb * kBlock + 8 * i;
  float x[8];
  if (live && a.aligned && k0 + 8 <= a.K) {
    load8(static_cast<const T*>(a.W) + n * a.ldw + k0, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = live && k0 + e < a.K ? to_f32(static_cast<const T*>(a.W)[n * a.ldw + k0 + e]) : 0.f;
  }
  float step;
  bool bad;
  const uint32_t w = quantise_word(x, a.group / 8, &step, &bad);
  if (!live) return;
  reinterpret_cast<uint32_t*>(a.codes + n * a.ldc + kb * kBlockBytes)[word_of(i)] = w;
  if ((8 * i) % a.group == 0 && k0 < a.K) {
    a.steps[n * a.lds + k0 / a.group] = step;
    if (bad) set_status(a.status, IMQ_ERR_NONFINITE);
  }
}

// W stored K x N: a CTA takes 128 inputs of 32 channels through shared memory.
template <typename T>
__global__ void __launch_bounds__(256) k_w4_quantize_cols(QuantArgs a) {
  __shared__ float tile[32][kBlock + 1];
  const int64_t kb = blockIdx.y, n0 = (int64_t)blockIdx.x * 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = warp; r < kBlock; r += 8) {
    const int64_t k = kb * kBlock + r, n = n0 + lane;
    tile[lane][r] = k < a.K && n < a.N ? to_f32(static_cast<const T*>(a.W)[k * a.ldw + n]) : 0.f;
  }
  __syncthreads();
  const int i = lane & 15;
  const int64_t k0 = kb * kBlock + 8 * i;
  for (int r = 2 * warp + (lane >> 4); r < 32; r += 16) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = tile[r][8 * i + e];
    float step;
    bool bad;
    const uint32_t w = quantise_word(x, a.group / 8, &step, &bad);
    const int64_t n = n0 + r;
    if (n >= a.N) continue;
    reinterpret_cast<uint32_t*>(a.codes + n * a.ldc + kb * kBlockBytes)[word_of(i)] = w;
    if ((8 * i) % a.group == 0 && k0 < a.K) {
      a.steps[n * a.lds + k0 / a.group] = step;
      if (bad) set_status(a.status, IMQ_ERR_NONFINITE);
    }
  }
}

struct DequantArgs {
  const uint8_t* codes;
  int64_t ldc;
  const float* steps;
  int64_t lds;
  int64_t K, N;
  int group;
  void* W;
  int64_t ldw;
  int aligned;
};

template <typename T>
__global__ void __launch_bounds__(256) k_w4_dequantize_rows(DequantArgs a) {
  const int64_t nb = (a.K + kBlock - 1) / kBlock;
  const int64_t unit = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;
  const int i = threadIdx.x & 15;
  if (unit >= a.N * nb) return;
  const int64_t n = unit / nb, kb = unit % nb, k0 = kb * kBlock + 8 * i;
  if (k0 >= a.K) return;
  const uint32_t w = reinterpret_cast<const uint32_t*>(a.codes + n * a.ldc + kb * kBlockBytes)[word_of(i)];
  const float step = a.steps[n * a.lds + k0 / a.group];
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(nibble_value(w, e), step);
  T* out = static_cast<T*>(a.W) + n * a.ldw + k0;
  if (a.aligned && k0 + 8 <= a.K) {
    store8(out, x);
  } else {
    for (int e = 0; e < 8 && k0 + e < a.K; ++e) out[e] = from_f32<T>(x[e]);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) k_w4_dequantize_cols(DequantArgs a) {
  __shared__ float tile[32][kBlock + 1];
  const int64_t kb = blockIdx.y, n0 = (int64_t)blockIdx.x * 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane & 15;
  const int64_t k0 = kb * kBlock + 8 * i;
  for (int r = 2 * warp + (lane >> 4); r < 32; r += 16) {
    const int64_t n = n0 + r;
    if (n < a.N && k0 < a.K) {
      const uint32_t w = reinterpret_cast<const uint32_t*>(a.codes + n * a.ldc + kb * kBlockBytes)[word_of(i)];
      const float step = a.steps[n * a.lds + k0 / a.group];
#pragma unroll
      for (int e = 0; e < 8; ++e) tile[r][8 * i + e] = __fmul_rn(nibble_value(w, e), step);
    }
  }
  __syncthreads();
  for (int r = warp; r < kBlock; r += 8) {
    const int64_t k = kb * kBlock + r, n = n0 + lane;
    if (k < a.K && n < a.N) static_cast<T*>(a.W)[k * a.ldw + n] = from_f32<T>(tile[lane][r]);
  }
}

// ------------------------------------------------------------------------------------------------
// Y = X * W for a few tokens
// ------------------------------------------------------------------------------------------------
struct MatvecArgs {
  const uint8_t* codes;
  int64_t ldc;
  const float* steps;
  int64_t lds;
  int64_t K, N;
  const void* X;
  int64_t ldx;
  int64_t M;
  void* Y;
  int64_t ldy;
  int y_bf16;
  int aligned;  // rows of X may be read 16 bytes at a time
};

constexpr int kTokens = 16;  // tokens of a CTA
constexpr int kMvWarps = 8;

// The B operand of 8 inputs of one token (or part of one): four bf16 pairs.  bf16 entries go as they are;
// an fp32 entry is cut into three bf16 parts of 8 bits, exact together, `part` of which this column holds.
__device__ __forceinline__ uint4 x_pairs(const __nv_bfloat16* p, int64_t k0, int64_t K, bool vec, int) {
  if (vec && k0 + 8 <= K) return *reinterpret_cast<const uint4*>(p + k0);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t k = k0 + 2 * i;
    const uint32_t lo = k < K ? __bfloat16_as_ushort(p[k]) : 0u, hi = k + 1 < K ? __bfloat16_as_ushort(p[k + 1]) : 0u;
    w[i] = lo | (hi << 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 x_pairs(const float* p, int64_t k0, int64_t K, bool vec, int part) {
  float x[8];
  if (vec && k0 + 8 <= K) {
    load8(p + k0, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = k0 + e < K ? p[k0 + e] : 0.f;
  }
  const uint32_t m1 = part >= 1 ? 0xFFFF0000u : 0u, m2 = part >= 2 ? 0xFFFF0000u : 0u;
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] -= __uint_as_float(__float_as_uint(x[e]) & m1);
    x[e] -= __uint_as_float(__float_as_uint(x[e]) & m2);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __byte_perm(__float_as_uint(x[2 * i]), __float_as_uint(x[2 * i + 1]), 0x7632);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA: 16 output channels, up to 16 tokens.  Its warps take the blocks of 128 inputs in turn; the codes
// become bf16 in registers (exact) and are the A operand, the tokens' entries the B operand, so up to 8
// columns cost no more than one.  A group's sum is scaled by its step in fp32.  The warps' sums meet in
// shared memory in a fixed order.
template <typename T, int kGroup, int kTiles>
__global__ void __launch_bounds__(kMvWarps * 32) k_w4_matvec(MatvecArgs a) {
  constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
  __shared__ float red[kMvWarps][16][kTiles * 8 + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * kTokens;
  const int tokens = (int)min((int64_t)kTokens, a.M - m0);
  // rows behind the last one read the last one; their sums are not stored
  const int64_t r0 = min(n0 + g, a.N - 1), r1 = min(n0 + g + 8, a.N - 1);
  const uint8_t* w0 = a.codes + r0 * a.ldc + 16 * c;
  const uint8_t* w1 = a.codes + r1 * a.ldc + 16 * c;
  const float* s0 = a.steps + r0 * a.lds;
  const float* s1 = a.steps + r1 * a.lds;
  const T* xp[kTiles];
  int part[kTiles];
  bool has[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int col = 8 * t + g, tok = col / kParts;
    part[t] = col % kParts;
    has[t] = tok < tokens;
    xp[t] = static_cast<const T*>(a.X) + (m0 + (has[t] ? tok : 0)) * a.ldx;
  }
  float total[kTiles][4] = {}, acc[kTiles][4] = {};
  const int64_t nb = (a.K + kBlock - 1) / kBlock;
  for (int64_t kb = warp; kb < nb; kb += kMvWarps) {
    const uint4 v0 = __ldg(reinterpret_cast<const uint4*>(w0 + kb * kBlockBytes));
    const uint4 v1 = __ldg(reinterpret_cast<const uint4*>(w1 + kb * kBlockBytes));
    const uint32_t p0[4] = {v0.x, v0.y, v0.z, v0.w}, p1[4] = {v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int64_t k0 = kb * kBlock + 32 * h + 8 * c;
      uint32_t q0[4], q1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        q0[i] = nibbles_bf16(p0[h] >> (4 * i));
        q1[i] = nibbles_bf16(p1[h] >> (4 * i));
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const uint4 x = has[t] ? x_pairs(xp[t], k0, a.K, a.aligned, part[t]) : make_uint4(0u, 0u, 0u, 0u);
        mma_bf16(acc[t], q0[0], q1[0], q0[1], q1[1], x.x, x.y);
        mma_bf16(acc[t], q0[2], q1[2], q0[3], q1[3], x.z, x.w);
      }
      if ((h + 1) * 32 % kGroup == 0) {
        const int64_t gi = (kb * kBlock + 32 * h) / kGroup;
        if (gi * kGroup < a.K) {
          const float d0 = __ldg(s0 + gi), d1 = __ldg(s1 + gi);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            total[t][0] += d0 * acc[t][0], total[t][1] += d0 * acc[t][1];
            total[t][2] += d1 * acc[t][2], total[t][3] += d1 * acc[t][3];
          }
        }
#pragma unroll
        for (int t = 0; t < kTiles; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    red[warp][g][8 * t + 2 * c] = total[t][0], red[warp][g][8 * t + 2 * c + 1] = total[t][1];
    red[warp][g + 8][8 * t + 2 * c] = total[t][2], red[warp][g + 8][8 * t + 2 * c + 1] = total[t][3];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < 16 * tokens; o += kMvWarps * 32) {
    const int r = o & 15, tok = o >> 4;
    if (n0 + r >= a.N) continue;
    float y = 0.f;
#pragma unroll
    for (int p = kParts - 1; p >= 0; --p)  // the smallest parts first
      for (int w = 0; w < kMvWarps; ++w) y += red[w][r][tok * kParts + p];
    const int64_t at = (m0 + tok) * a.ldy + n0 + r;
    if (a.y_bf16)
      static_cast<__nv_bfloat16*>(a.Y)[at] = __float2bfloat16_rn(y);
    else
      static_cast<float*>(a.Y)[at] = y;
  }
}

template <typename T, int kTiles>
void matvec_group(const MatvecArgs& a, int group, dim3 grid, cudaStream_t st) {
  if (group == 32)
    k_w4_matvec<T, 32, kTiles><<<grid, kMvWarps * 32, 0, st>>>(a);
  else if (group == 64)
    k_w4_matvec<T, 64, kTiles><<<grid, kMvWarps * 32, 0, st>>>(a);
  else
    k_w4_matvec<T, 128, kTiles><<<grid, kMvWarps * 32, 0, st>>>(a);
}

bool is_float(imq_dtype t) { return t == IMQ_F32 || t == IMQ_BF16; }
int size_of(imq_dtype t) { return t == IMQ_F32 ? 4 : 2; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// What every call on a 4-bit weight checks.
imq_status check_weight(const void* codes, int64_t ldc, const void* steps, int64_t lds, int64_t K, int64_t N, int32_t group) {
  if (K < 0 || N < 0 || (group != 32 && group != 64 && group != 128)) return IMQ_ERR_ARG;
  if (K > INT32_MAX || N > INT32_MAX) return IMQ_ERR_UNSUPPORTED;
  if (ldc < (K + kBlock - 1) / kBlock * kBlockBytes || ldc % 16 != 0 || lds < (K + group - 1) / group) return IMQ_ERR_ARG;
  if (K > 0 && N > 0 && (!codes || !steps || !aligned16(codes) || (reinterpret_cast<uintptr_t>(steps) & 3)))
    return IMQ_ERR_ARG;
  return IMQ_OK;
}

imq_status launched() { return cudaGetLastError() == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA; }
}  // namespace

imq_status launch_w4_quantize(const void* W, imq_dtype wt, int64_t K, int64_t N, int64_t ldw, int32_t transW, int32_t group,
                              uint8_t* codes, int64_t ldc, float* steps, int64_t lds, cudaStream_t st) {
  imq_status s = check_weight(codes, ldc, steps, lds, K, N, group);
  if (s != IMQ_OK) return s;
  if (!is_float(wt) || (transW != 0 && transW != 1) || ldw < (transW ? K : N)) return IMQ_ERR_ARG;
  if (K == 0 || N == 0) return IMQ_OK;
  if (!W || (reinterpret_cast<uintptr_t>(W) & (size_of(wt) - 1))) return IMQ_ERR_ARG;
  DeviceState* ds;
  s = device_state(&ds);
  if (s != IMQ_OK) return s;
  QuantArgs a{W, K, N, ldw, codes, ldc, steps, lds, group, aligned16(W) && ldw * size_of(wt) % 16 == 0, ds->status};
  const int64_t nb = (K + kBlock - 1) / kBlock;
  if (transW) {
    const int64_t ctas = (N * nb + 15) / 16;
    if (ctas > INT32_MAX) return IMQ_ERR_UNSUPPORTED;
    if (wt == IMQ_F32)
      k_w4_quantize_rows<float><<<(unsigned)ctas, 256, 0, st>>>(a);
    else
      k_w4_quantize_rows<__nv_bfloat16><<<(unsigned)ctas, 256, 0, st>>>(a);
  } else {
    if (nb > 65535) return IMQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)((N + 31) / 32), (unsigned)nb);
    if (wt == IMQ_F32)
      k_w4_quantize_cols<float><<<grid, 256, 0, st>>>(a);
    else
      k_w4_quantize_cols<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  }
  return launched();
}

imq_status launch_w4_dequantize(const uint8_t* codes, int64_t ldc, const float* steps, int64_t lds, int64_t K, int64_t N,
                                int32_t group, void* W, imq_dtype wt, int64_t ldw, int32_t transW, cudaStream_t st) {
  imq_status s = check_weight(codes, ldc, steps, lds, K, N, group);
  if (s != IMQ_OK) return s;
  if (!is_float(wt) || (transW != 0 && transW != 1) || ldw < (transW ? K : N)) return IMQ_ERR_ARG;
  if (K == 0 || N == 0) return IMQ_OK;
  if (!W || (reinterpret_cast<uintptr_t>(W) & (size_of(wt) - 1))) return IMQ_ERR_ARG;
  DequantArgs a{codes, ldc, steps, lds, K, N, group, W, ldw, aligned16(W) && ldw * size_of(wt) % 16 == 0};
  const int64_t nb = (K + kBlock - 1) / kBlock;
  if (transW) {
    const int64_t ctas = (N * nb + 15) / 16;
    if (ctas > INT32_MAX) return IMQ_ERR_UNSUPPORTED;
    if (wt == IMQ_F32)
      k_w4_dequantize_rows<float><<<(unsigned)ctas, 256, 0, st>>>(a);
    else
      k_w4_dequantize_rows<__nv_bfloat16><<<(unsigned)ctas, 256, 0, st>>>(a);
  } else {
    if (nb > 65535) return IMQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)((N + 31) / 32), (unsigned)nb);
    if (wt == IMQ_F32)
      k_w4_dequantize_cols<float><<<grid, 256, 0, st>>>(a);
    else
      k_w4_dequantize_cols<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
  }
  return launched();
}

imq_status launch_w4_matvec(const uint8_t* codes, int64_t ldc, const float* steps, int64_t lds, int64_t K, int64_t N,
                            int32_t group, const void* X, imq_dtype xt, int64_t M, int64_t ldx, void* Y, imq_dtype yt,
                            int64_t ldy, cudaStream_t st) {
  imq_status s = check_weight(codes, ldc, steps, lds, K, N, group);
  if (s != IMQ_OK) return s;
  if (!is_float(xt) || !is_float(yt) || M < 0 || ldx < K || ldy < N) return IMQ_ERR_ARG;
  if (M > 65535 * (int64_t)kTokens) return IMQ_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return IMQ_OK;
  if ((K > 0 && !X) || !Y || (reinterpret_cast<uintptr_t>(X) & (size_of(xt) - 1)) ||
      (reinterpret_cast<uintptr_t>(Y) & (size_of(yt) - 1)))
    return IMQ_ERR_ARG;
  MatvecArgs a{codes, ldc, steps, lds, K, N, X, ldx, M, Y, ldy, yt == IMQ_BF16,
               aligned16(X) && (M == 1 || ldx * size_of(xt) % 16 == 0)};
  const dim3 grid((unsigned)((N + 15) / 16), (unsigned)((M + kTokens - 1) / kTokens));
  const int cols = (int)(M < kTokens ? M : kTokens) * (xt == IMQ_F32 ? 3 : 1), tiles = (cols + 7) / 8;
  if (xt == IMQ_BF16) {
    if (tiles == 1)
      matvec_group<__nv_bfloat16, 1>(a, group, grid, st);
    else
      matvec_group<__nv_bfloat16, 2>(a, group, grid, st);
  } else if (tiles == 1) {
    matvec_group<float, 1>(a, group, grid, st);
  } else if (tiles <= 3) {
    matvec_group<float, 3>(a, group, grid, st);
  } else {
    matvec_group<float, 6>(a, group, grid, st);
  }
  return launched();
}

}  // namespace imq
