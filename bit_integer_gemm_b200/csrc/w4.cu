// w4.cu -- weights of 4 bits with a step per group of inputs: quantiser, its inverse, and the product of a
// few tokens with such a weight (sm_100a).
//
// Storage of output channel n (a row): K inputs in blocks of 128, 64 bytes each; input r of a block is code
// e = r % 8 of word 4 * ((r % 32) / 8) + r / 32 of the block's 16.  A lane that takes the 16 bytes at
// 16 * c of a block holds the inputs 32h + 8c .. 32h + 8c + 7 for h = 0..3: one word per 32 inputs, so a
// group of 32 ends at a word, and the inputs it needs from a token are 16 contiguous bytes of bf16 per word.
#include <atomic>

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
  int log_group;
  int vec;  // rows of W may be read 16 bytes (stored N x K) or two entries (K x N) at a time
  int32_t* status;
};

__device__ __forceinline__ uint32_t max_key(const float (&x)[8]) {
  uint32_t key = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) key = max(key, abs_key(x[e]));
  return key;
}

// Row kernels (W stored N x K): a warp takes 256 inputs (two blocks) of four rows, 8 inputs of each a lane.  Bound: memory
// for fp32 (11003 x 4097 in 36.4 us, 5.7 TB/s, and back in 34.1), the quantiser's instructions for bf16 (4096 x 4096 in
// 11.9 us, 3.6 TB/s; back 9.1).
constexpr int kRows = 4;
constexpr int kQuantWarps = 4;  // of the quantiser's CTAs (8: 37.6 us and 12.0)

// x[e] = entry e * 32 + lane of 256 consecutive ones, becomes entry 8 * lane + e: turned in shared memory (`turn`, 288
// floats of the warp's own, a float of padding every 8 entries).
__device__ __forceinline__ void turn256(float* turn, int lane, float (&x)[8]) {
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 8; ++e) turn[e * 36 + lane + lane / 8] = x[e];
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = turn[9 * lane + e];
}

template <typename T>
__global__ void __launch_bounds__(kQuantWarps * 32) k_w4_quantize_rows(QuantArgs a) {
  __shared__ float s_turn[kQuantWarps][288];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane & 15;
  const uint32_t per_row = ((uint32_t)a.K + 255) / 256, unit = blockIdx.x * kQuantWarps + warp;
  const int n0 = (int)(unit / per_row) * kRows, k0 = (int)(unit % per_row) * 256, k = k0 + 8 * lane;
  const int N = (int)a.N, K = (int)a.K;
  if (n0 >= N) return;
  const T* const p = static_cast<const T*>(a.W) + n0 * a.ldw + k0;
  float x[kRows][8];
  if (a.vec && k0 + 256 <= K) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) load8(p + (n0 + j < N ? j : 0) * a.ldw + 8 * lane, x[j]);
  } else {  // rows that begin anywhere, and their ends: read in order, all of them before the first is turned
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const T* const row = p + (n0 + j < N ? j : 0) * a.ldw + lane;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = k0 + e * 32 + lane < K ? to_f32(row[e * 32]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) turn256(s_turn[warp], lane, x[j]);
  }
  uint32_t key[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) key[j] = max_key(x[j]);
  const int lanes = 1 << (a.log_group - 3);  // of a group: 4, 8 or 16
#pragma unroll
  for (int o = 1; o < 16; o <<= 1)
    if (o < lanes) {
#pragma unroll
      for (int j = 0; j < kRows; ++j) key[j] = max(key[j], __shfl_xor_sync(0xffffffffu, key[j], o));
    }
  float s[kRows], step[kRows];
  four_scales(key, 7.f, s, step);
  if (k - 8 * i >= K) return;  // the row's last block was the other half's
  const int rows = min(kRows, N - n0);
  uint8_t* to = a.codes + n0 * a.ldc + k0 / kBlock * kBlockBytes + (lane >> 4) * kBlockBytes + 4 * word_of(i);
#pragma unroll
  for (int j = 0; j < kRows; ++j, to += a.ldc)
    if (j < rows) *reinterpret_cast<uint32_t*>(to) = pack4(x[j], s[j]);
  if ((i & (lanes - 1)) == 0 && k < K) {
    float* to_step = a.steps + n0 * a.lds + (k >> a.log_group);
    bool finite = true;
#pragma unroll
    for (int j = 0; j < kRows; ++j, to_step += a.lds)
      if (j < rows) *to_step = step[j], finite &= key_finite(key[j]);
    if (!finite) set_status(a.status, IMQ_ERR_NONFINITE);
  }
}

// Column kernels (W stored K x N): a CTA takes 128 inputs of 64 channels, a warp 32 of the inputs, a lane two channels:
// what it reads in order, 32 loads under way together, is four of its words a channel.  Only the words, and of groups
// above 32 the largest entries, pass through shared memory.  Bound: memory; 4096 x 4096 bf16 in 9.2 us (4.6 TB/s) and
// back in 9.4, 11008 x 4096 fp32 in 34.9 (5.9) and 35.7.  (A quarter of the inputs a lane, in four times the warps,
// had too few bytes under way: 13.7 and 12.4 us for the first.)
constexpr int kColChannels = 64;
// Two channels' entries of 32 inputs as they lie in memory.
template <typename T>
struct Column;
template <>
struct Column<__nv_bfloat16> {
  uint32_t w[32];
  __device__ __forceinline__ void load(int e, const __nv_bfloat16* p) { w[e] = __ldcs(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ void load(int e, const __nv_bfloat16* p, bool first, bool second) {
    w[e] = (first ? (uint32_t)__bfloat16_as_ushort(p[0]) : 0u) | (second ? (uint32_t)__bfloat16_as_ushort(p[1]) << 16 : 0u);
  }
  __device__ __forceinline__ float entry(int e, int channel) const { return __uint_as_float(channel ? w[e] & 0xFFFF0000u : w[e] << 16); }
  // abs_key of each channel's largest entry, both at a time
  __device__ __forceinline__ uint2 key() const {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) m = __vmaxu2(m, w[e] & 0x7FFF7FFFu);
    return make_uint2(m << 16, m & 0xFFFF0000u);
  }
};
template <>
struct Column<float> {
  float2 w[32];
  __device__ __forceinline__ void load(int e, const float* p) { w[e] = __ldcs(reinterpret_cast<const float2*>(p)); }
  __device__ __forceinline__ void load(int e, const float* p, bool first, bool second) {
    w[e] = make_float2(first ? p[0] : 0.f, second ? p[1] : 0.f);
  }
  __device__ __forceinline__ float entry(int e, int channel) const { return channel ? w[e].y : w[e].x; }
  __device__ __forceinline__ uint2 key() const {
    uint2 m = make_uint2(0u, 0u);
#pragma unroll
    for (int e = 0; e < 32; ++e) m.x = max(m.x, abs_key(w[e].x)), m.y = max(m.y, abs_key(w[e].y));
    return m;
  }
};
// Where word i of a channel of the CTA lies in shared memory.
__device__ __forceinline__ int col_word(int channel, int i) { return (channel % 2 * 32 + channel / 2) * 17 + i; }

template <typename T>
__global__ void __launch_bounds__(128) k_w4_quantize_cols(QuantArgs a) {
  __shared__ uint2 s_key[4][32];
  __shared__ uint32_t s_word[kColChannels * 17];
  const int k0 = blockIdx.y * kBlock, n0 = blockIdx.x * kColChannels, K = (int)a.K, N = (int)a.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = k0 + 32 * warp, n = n0 + 2 * lane;
  const T* const p = static_cast<const T*>(a.W) + k * a.ldw + n;
  Column<T> x;
  if (a.vec && k + 32 <= K && n + 1 < N) {
#pragma unroll
    for (int e = 0; e < 32; ++e) x.load(e, p + e * a.ldw);
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) x.load(e, p + e * a.ldw, k + e < K && n < N, k + e < K && n + 1 < N);
  }
  uint2 key = x.key();
  const int warps = 1 << (a.log_group - 5);  // of a group
  if (warps > 1) {
    s_key[warp][lane] = key;
    __syncthreads();
    const int first = warp & ~(warps - 1);
    for (int w = first; w < first + warps; ++w) key.x = max(key.x, s_key[w][lane].x), key.y = max(key.y, s_key[w][lane].y);
  }
  float s[2], step[2];
  group_scale(key.x, 7.f, &s[0], &step[0]);
  group_scale(key.y, 7.f, &s[1], &step[1]);
  if ((warp & (warps - 1)) == 0 && k < K) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (n + j < N) {
        a.steps[(n + j) * a.lds + (k >> a.log_group)] = step[j];
        if (!key_finite(j ? key.y : key.x)) set_status(a.status, IMQ_ERR_NONFINITE);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = x.entry(8 * i + e, j);
      s_word[col_word(2 * lane + j, 4 * i + warp)] = pack4(y, s[j]);
    }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int c = threadIdx.x / 4 + 32 * q, i = threadIdx.x % 4 * 4;
    const uint32_t* const w = s_word + col_word(c, i);
    if (n0 + c < N)
      *reinterpret_cast<uint4*>(a.codes + (n0 + c) * a.ldc + (int64_t)blockIdx.y * kBlockBytes + 4 * i) =
          make_uint4(w[0], w[1], w[2], w[3]);
  }
}

struct DequantArgs {
  const uint8_t* codes;
  int64_t ldc;
  const float* steps;
  int64_t lds;
  int64_t K, N;
  int log_group;
  void* W;
  int64_t ldw;
  int vec;
  uint32_t one;  // kOneF16
};

__device__ __forceinline__ void word_values(uint32_t w, float step, uint32_t one, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = nibble_pair(w, i, one);
    x[2 * i] = __fmul_rn(v.x, step), x[2 * i + 1] = __fmul_rn(v.y, step);
  }
}

// The row and column kernels of the quantiser the other way round.
template <typename T>
__global__ void __launch_bounds__(256) k_w4_dequantize_rows(DequantArgs a) {
  __shared__ float s_turn[8][288];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = lane & 15;
  const uint32_t per_row = ((uint32_t)a.K + 255) / 256, unit = blockIdx.x * 8 + warp;
  const int n0 = (int)(unit / per_row) * kRows, k0 = (int)(unit % per_row) * 256, k = k0 + 8 * lane;
  const int N = (int)a.N, K = (int)a.K;
  if (n0 >= N) return;
  const uint8_t* const from = a.codes + n0 * a.ldc + k0 / kBlock * kBlockBytes + (lane >> 4) * kBlockBytes + 4 * word_of(i);
  const float* const from_step = a.steps + n0 * a.lds + (k >> a.log_group);
  uint32_t w[kRows];
  float step[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const bool on = n0 + j < N && k < K;
    w[j] = on ? *reinterpret_cast<const uint32_t*>(from + j * a.ldc) : 0u;
    step[j] = on ? from_step[j * a.lds] : 0.f;
  }
  T* const out = static_cast<T*>(a.W) + n0 * a.ldw + k0;
  float* const turn = s_turn[warp];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    if (n0 + j >= N) break;
    float x[8];
    word_values(w[j], step[j], a.one, x);
    const bool whole = a.vec && k0 + 256 <= K;
    if constexpr (sizeof(T) == 2) {
      if (whole) {  // 16 bytes a lane, in order
        store8(out + j * a.ldw + 8 * lane, x);
        continue;
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) turn[9 * lane + e] = x[e];
    __syncwarp();
    if (whole) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float* const t = turn + q * 144 + 4 * lane + lane / 2;
        *reinterpret_cast<float4*>(out + j * a.ldw + q * 128 + 4 * lane) = make_float4(t[0], t[1], t[2], t[3]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k0 + e * 32 + lane < K) out[j * a.ldw + e * 32 + lane] = from_f32<T>(turn[e * 36 + lane + lane / 8]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(128) k_w4_dequantize_cols(DequantArgs a) {
  __shared__ uint32_t s_word[kColChannels * 17];
  const int k0 = blockIdx.y * kBlock, n0 = blockIdx.x * kColChannels, K = (int)a.K, N = (int)a.N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = k0 + 32 * warp, n = n0 + 2 * lane;
  uint4 w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int c = min(threadIdx.x / 4 + 32 * q, N - 1 - n0);  // (channels behind the last one: not stored)
    w[q] = *reinterpret_cast<const uint4*>(a.codes + (n0 + c) * a.ldc + (int64_t)blockIdx.y * kBlockBytes + threadIdx.x % 4 * 16);
  }
  float step[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) step[j] = n + j < N && k < K ? a.steps[(n + j) * a.lds + (k >> a.log_group)] : 0.f;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t* const to = s_word + col_word(threadIdx.x / 4 + 32 * q, threadIdx.x % 4 * 4);
    to[0] = w[q].x, to[1] = w[q].y, to[2] = w[q].z, to[3] = w[q].w;
  }
  __syncthreads();
  T* const out = static_cast<T*>(a.W) + k * a.ldw + n;
  const bool whole = a.vec && k + 32 <= K && n + 1 < N;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[2][8];
#pragma unroll
    for (int j = 0; j < 2; ++j) word_values(s_word[col_word(2 * lane + j, 4 * i + warp)], step[j], a.one, x[j]);
    T* const to = out + 8 * i * a.ldw;
    if (whole) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(to + e * a.ldw) = make_float2(x[0][e], x[1][e]);
        else *reinterpret_cast<uint32_t*>(to + e * a.ldw) = bf16_pair(x[0][e], x[1][e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (k + 8 * i + e < K && n < N) to[e * a.ldw] = from_f32<T>(x[0][e]);
        if (k + 8 * i + e < K && n + 1 < N) to[e * a.ldw + 1] = from_f32<T>(x[1][e]);
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------
// Y = X * W for a few tokens
// ------------------------------------------------------------------------------------------------
// The weight is read once per 16 tokens, N K / 2 bytes and the steps, for 2 M N K operations.  Memory does not bound it:
// turning codes into operands takes eleven instructions for eight codes (seven of them integer).  So the product runs on
// the warp-level tensor core instruction with the weight as the 16-row operand: a conversion serves 8 tokens at once.
// No unit is full either (issue slots 37 to 58 %, integer pipe 34 to 52 %, 12 to 24 % of the warps): the warps are few and
// wait on their own chains, and sets of channels come in whole rounds (688 sets on 296 CTAs: three rounds for 2.3).
// One bf16 token: 4096 x 4096 in 4.3 us, 11008 x 4096 in 8.6 (2.9 TB/s); 8 tokens, 4096 x 22016: 16.0 us (3.0 TB/s), 16: 22.8,
// 24: 42; 3 fp32 tokens, 4099 x 11007: 20.1 us.
//   - Codes in -7 .. 7 are exact in bf16, and bf16 entries of X are operands as they are.
//   - An fp32 entry is cut into three bf16 parts of 8 bits, exact together: a column of the other operand for each
//     part with up to 2 tokens, an operand for each part with more.
//   - The sums of a group are scaled by its step in fp32.
// A CTA takes 16 kR output channels at a time; its eight warps take the blocks of 128 inputs in turn, each with its own
// ring of asynchronous copies that runs on from one set of channels to the next.  The warps' sums meet in shared
// memory, in a fixed order.  (X read straight into registers, a block ahead, cost 17.1 us for the 8 tokens; 16.3 then.)
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
  int aligned;   // bytes at which every row of X begins a multiple: 16, 4 or 2
  uint32_t one;  // kOneBf16
};

constexpr int kTokens = 16;  // tokens of a CTA
constexpr int kMvWarps = 8;

// kTiles: operands of 8 columns.  bf16: tokens 8t + g.  fp32: 1: part g % 3 of token g / 3; 3 (6): parts 0-2 of token g
// (and of token g + 8).
template <typename T, int kGroup, int kTiles, int kR>
struct MvShape {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr bool kPacked = kF32 && kTiles == 1;
  static constexpr int kParts = kF32 ? 3 : 1;
  static constexpr int kTok = kPacked ? 1 : kTiles / kParts;  // tokens of a lane
  // X of a stage: a row of 128 entries a token.  In odd rows kSwap bytes change places with the next kSwap (an exclusive
  // or of the place), so that the eight lanes that read 16 bytes together, from two rows, meet other banks.
  static constexpr int kXRows = kPacked ? 2 : 8 * kTok, kXPitch = kBlock * (int)sizeof(T), kSwap = kF32 ? 16 : 64;
  static constexpr int kPerBlock = kBlock / kGroup;           // steps of a row and block
  static constexpr int kXAt = 2 * kR * 512, kStepsAt = kXAt + kXRows * kXPitch;
  static constexpr int kStage = kStepsAt + 2 * kR * 8 * kPerBlock * 4;
  // CTAs an SM: two where registers allow (8 tokens, 4096 x 22016: 16.0 us; with one and rings twice as long 18.8)
  static constexpr int kPerSm = kTiles * kR <= 2 ? 2 : 1;
  static constexpr int kCols = kTiles * 8;
  static constexpr int kRed = kMvWarps * 16 * kR * kCols * 4;
  // where a row's and column's sum of a warp lies: turned by a place every four rows, against bank conflicts
  static __device__ __forceinline__ int sum_at(int warp, int row, int col) {
    return ((warp * 16 * kR + row) * kTiles + col / 8) * 8 + ((col % 8 + row / 4) & 7);
  }
  // as many stages as shared memory holds (227 KB an SM, 1 KB a CTA of it reserved)
  static constexpr int kFit = ((kPerSm == 2 ? 112 : 225) * 1024 - kRed) / (kMvWarps * kStage);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kSmem = kMvWarps * kStages * kStage + kRed;
  static_assert(kStages >= 2, "a ring needs two stages");
};

template <typename T, int kGroup, int kTiles, int kR>
__global__ void __launch_bounds__(kMvWarps * 32, MvShape<T, kGroup, kTiles, kR>::kPerSm) k_w4_matvec(const __grid_constant__ MatvecArgs a) {
  using S = MvShape<T, kGroup, kTiles, kR>;
  constexpr int kStages = S::kStages, kPer16 = 16 / sizeof(T);
  extern __shared__ __align__(16) uint8_t smem[];
  float* const red = reinterpret_cast<float*>(smem + kMvWarps * kStages * S::kStage);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int K = (int)a.K, N = (int)a.N, nb = (K + kBlock - 1) / kBlock;
  const int64_t m0 = (int64_t)blockIdx.y * kTokens;
  const int tokens = (int)min((int64_t)kTokens, a.M - m0);
  const int sets = (N + 16 * kR - 1) / (16 * kR);
  const int per_set = (nb - warp + kMvWarps - 1) / kMvWarps;  // this warp's blocks of a set (0 for K below its first)
  const int groups = (K + kGroup - 1) / kGroup;
  constexpr int kPerBlock = S::kPerBlock;
  uint8_t* const mine = smem + warp * kStages * S::kStage;

  // Copies of X take its rows in order: a row's 128 entries are kRowLanes copies of 16 bytes.  Columns without a token
  // hold what lies in shared memory: a column's sums depend on no other column, and theirs are not stored.
  constexpr int kRowLanes = kBlock / kPer16, kRowsAtOnce = 32 / kRowLanes;
  const int64_t row_bytes = a.ldx * (int)sizeof(T);
  const uint8_t* const x0 = static_cast<const uint8_t*>(a.X) + m0 * row_bytes;
  const uint8_t* const x16 = x0 + lane / kRowLanes * row_bytes + lane % kRowLanes * 16;
  const uint32_t to16 = S::kXAt + lane / kRowLanes * S::kXPitch + (lane % kRowLanes * 16 ^ lane / kRowLanes % 2 * S::kSwap);
  const int whole = K / kBlock, whole16 = a.aligned == 16 ? whole : 0;  // blocks copied whole, and 16 bytes at a time
  // where this lane's entries lie in a stage
  const int x_row = S::kPacked ? min(g / 3, 1) : g, swap = x_row % 2 * S::kSwap;
  const uint32_t x_at = S::kXAt + x_row * S::kXPitch + (S::kF32 ? 32 * c : 16 * c);

  // the next block to copy: set, its block, ring stage, and where the set's rows lie
  int set_in = blockIdx.x, kb_in = warp, stage_in = 0;
  // The steps of a stage are copied in order too: kStepCopies of them a lane.
  constexpr int kStepCopies = (16 * kR * kPerBlock + 31) / 32;
  const uint8_t* code_row[2 * kR];
  const float* step_row[kStepCopies];
  auto open_set = [&]() {
    // rows behind the last one read the last one; their sums are not stored
    const int last = N - 1 - set_in * 16 * kR;
    const uint8_t* const code0 = a.codes + (int64_t)set_in * (16 * kR) * a.ldc + 16 * c;
    const float* const step0 = a.steps + (int64_t)set_in * (16 * kR) * a.lds + lane % kPerBlock;
#pragma unroll
    for (int r = 0; r < 2 * kR; ++r) code_row[r] = code0 + min(8 * r + g, last) * a.ldc;
#pragma unroll
    for (int q = 0; q < kStepCopies; ++q) step_row[q] = step0 + min((q * 32 + lane) / kPerBlock, last) * a.lds;
  };
  if (set_in < sets) open_set();
  auto issue = [&]() {
    if (set_in < sets && per_set > 0) {
      uint8_t* const to = mine + stage_in * S::kStage;
      const uint32_t dst = smem_addr(to), dst_x = dst + S::kXAt;
#pragma unroll
      for (int r = 0; r < 2 * kR; ++r) cp_async<16>(dst + lane * 16 + r * 512, code_row[r] + (uint32_t)kb_in * kBlockBytes);
      // zeros for groups behind the last one: no stale step meets their sums of 0
      const uint32_t step_bytes = kb_in * kPerBlock + lane % kPerBlock < groups ? 4u : 0u;
#pragma unroll
      for (int q = 0; q < kStepCopies; ++q)
        if (16 * kR * kPerBlock >= 32 || lane < 16 * kR * kPerBlock)
          cp_async_part<4>(dst + S::kStepsAt + (q * 32 + lane) * 4, step_bytes ? step_row[q] + (uint32_t)kb_in * kPerBlock : a.steps,
                           step_bytes);
      const uint32_t k_bytes = (uint32_t)kb_in * (kBlock * (int)sizeof(T));
      if (kb_in < whole16) {
        const uint8_t* row = x16 + k_bytes;
#pragma unroll
        for (int q = 0; q < S::kXRows / kRowsAtOnce; ++q) {
          if (q * kRowsAtOnce >= tokens) break;
          const uint32_t at = (to16 ^ (kRowsAtOnce == 1 ? q % 2 * S::kSwap : 0)) + q * kRowsAtOnce * S::kXPitch;
          if (kRowsAtOnce == 1 || q * kRowsAtOnce + lane / kRowLanes < tokens) cp_async<16>(dst + at, row);
          row += kRowsAtOnce * row_bytes;
        }
      } else if (a.aligned >= 4 && kb_in < whole) {  // rows that begin anywhere: four bytes at a time
        const uint8_t* row = x0 + k_bytes + lane * 4;
        uint32_t at = dst_x;
        for (int t = 0; t < tokens; ++t, row += row_bytes, at += S::kXPitch) {
          const uint32_t to4 = at + (lane * 4 ^ t % 2 * S::kSwap);  // (stages begin at multiples of 64 bytes: not at ^ ...)
#pragma unroll
          for (int q = 0; q < kBlock * (int)sizeof(T) / 128; ++q) cp_async<4>(to4 + q * 128, row + q * 128);
        }
      } else if (a.aligned >= 4) {  // the end of a row, zeros behind it
        const int left = (K - kb_in * kBlock) * (int)sizeof(T);  // bytes
        for (int t = 0; t < tokens; ++t) {
          for (int q = 0; q < kBlock * (int)sizeof(T) / 128; ++q) {
            const int at = q * 128 + lane * 4, n = min(max(left - at, 0), 4);
            cp_async_part<4>(dst_x + t * S::kXPitch + (at ^ t % 2 * S::kSwap), n ? x0 + t * row_bytes + k_bytes + at : a.codes, n);
          }
        }
      } else if constexpr (!S::kF32) {  // bf16 rows on 2-byte boundaries
        const int k0 = kb_in * kBlock + lane;
        for (int t = 0; t < tokens; t += 2) {  // (loads of two rows under way together)
          T v[2][4];
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[j][q] = k0 + 32 * q < K ? reinterpret_cast<const T*>(x0 + min(t + j, tokens - 1) * row_bytes)[k0 + 32 * q]
                                        : from_f32<T>(0.f);
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int at = (32 * q + lane) * (int)sizeof(T) ^ j * S::kSwap;
              *reinterpret_cast<T*>(to + S::kXAt + (t + j) * S::kXPitch + at) = v[j][q];
            }
        }
      }
      stage_in = stage_in + 1 == kStages ? 0 : stage_in + 1;
      kb_in += kMvWarps;
      if (kb_in >= nb) {
        kb_in = warp, set_in += gridDim.x;
        if (set_in < sets) open_set();
      }
    }
    cp_async_commit();
  };
  for (int i = 0; i < kStages - 1; ++i) issue();

  int stage = 0;
  for (int set = blockIdx.x; set < sets; set += gridDim.x) {
    float total[kR][kTiles][4] = {};
    for (int i = 0; i < per_set; ++i) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // other lanes copied X and the steps; every lane is done with the stage that is overwritten now
      issue();
      const uint8_t* const from = mine + stage * S::kStage;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      uint4 v[kR][2];
#pragma unroll
      for (int r = 0; r < kR; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) v[r][j] = *reinterpret_cast<const uint4*>(from + (2 * r + j) * 512 + lane * 16);
      const float* const st = reinterpret_cast<const float*>(from + S::kStepsAt) + g * kPerBlock;
      float acc[kR][kTiles][4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        // the other operand: per tile, the pairs of this half's first four inputs and of its second four
        uint32_t x[kTiles][4];
#pragma unroll
        for (int t = 0; t < S::kTok; ++t) {
          if constexpr (!S::kF32) {
            const uint4 q = *reinterpret_cast<const uint4*>(from + x_at + t * 8 * S::kXPitch + (h * 64 ^ swap));
            x[t][0] = q.x, x[t][1] = q.y, x[t][2] = q.z, x[t][3] = q.w;
          } else {
            float f[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float4 y = *reinterpret_cast<const float4*>(from + x_at + t * 8 * S::kXPitch + h * 128 + (q * 16 ^ swap));
              f[4 * q] = y.x, f[4 * q + 1] = y.y, f[4 * q + 2] = y.z, f[4 * q + 3] = y.w;
            }
            if constexpr (S::kPacked) {
              const uint32_t m1 = g % 3 >= 1 ? 0xFFFF0000u : 0u, m2 = g % 3 >= 2 ? 0xFFFF0000u : 0u;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                f[e] -= __uint_as_float(__float_as_uint(f[e]) & m1);
                f[e] -= __uint_as_float(__float_as_uint(f[e]) & m2);
              }
            }
#pragma unroll
            for (int part = 0; part < (S::kPacked ? 1 : 3); ++part) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[t * (S::kPacked ? 1 : 3) + part][e] = __byte_perm(__float_as_uint(f[2 * e]), __float_as_uint(f[2 * e + 1]), 0x7632);
              if (part < 2) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] -= __uint_as_float(__float_as_uint(f[e]) & 0xFFFF0000u);
              }
            }
          }
        }
        const bool opens = h * 32 % kGroup == 0, closes = (h + 1) * 32 % kGroup == 0;
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const uint32_t p0 = h == 0 ? v[r][0].x : h == 1 ? v[r][0].y : h == 2 ? v[r][0].z : v[r][0].w;
          const uint32_t p1 = h == 0 ? v[r][1].x : h == 1 ? v[r][1].y : h == 2 ? v[r][1].z : v[r][1].w;
          uint32_t q0[4], q1[4];
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) q0[i4] = nibbles_bf16(p0 >> (4 * i4), a.one), q1[i4] = nibbles_bf16(p1 >> (4 * i4), a.one);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            if (opens) acc[r][t][0] = acc[r][t][1] = acc[r][t][2] = acc[r][t][3] = 0.f;
            mma_bf16(acc[r][t], q0[0], q1[0], q0[1], q1[1], x[t][0], x[t][1]);
            mma_bf16(acc[r][t], q0[2], q1[2], q0[3], q1[3], x[t][2], x[t][3]);
          }
          if (closes) {
            const int gi = h * 32 / kGroup;
            const float d0 = st[2 * r * 8 * kPerBlock + gi], d1 = st[(2 * r + 1) * 8 * kPerBlock + gi];
#pragma unroll
            for (int t = 0; t < kTiles; ++t) {
              total[r][t][0] += d0 * acc[r][t][0], total[r][t][1] += d0 * acc[r][t][1];
              total[r][t][2] += d1 * acc[r][t][2], total[r][t][3] += d1 * acc[r][t][3];
            }
          }
        }
      }
    }
    // ---- the warps' sums of this set
#pragma unroll
    for (int r = 0; r < kR; ++r)
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int j = 0; j < 4; ++j) red[S::sum_at(warp, 16 * r + g + 8 * (j >> 1), 8 * t + 2 * c + (j & 1))] = total[r][t][j];
      }
    __syncthreads();
    for (int o = threadIdx.x; o < 16 * kR * tokens; o += kMvWarps * 32) {
      const int row = o % (16 * kR), tok = o / (16 * kR), n = set * 16 * kR + row;
      float y = 0.f;
#pragma unroll
      for (int p = S::kParts - 1; p >= 0; --p) {  // the smallest parts first
        const int col = S::kPacked ? 3 * tok + p : S::kF32 ? (tok / 8 * 3 + p) * 8 + tok % 8 : tok;
#pragma unroll
        for (int w = 0; w < kMvWarps; ++w) y += red[S::sum_at(w, row, col)];
      }
      if (n < N) {
        const int64_t at = (m0 + tok) * a.ldy + n;
        if (a.y_bf16)
          static_cast<__nv_bfloat16*>(a.Y)[at] = __float2bfloat16_rn(y);
        else
          static_cast<float*>(a.Y)[at] = y;
      }
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

template <typename T, int kGroup, int kTiles, int kR>
imq_status matvec_shape(const MatvecArgs& a, int num_sms, cudaStream_t st) {
  constexpr int kSmem = MvShape<T, kGroup, kTiles, kR>::kSmem;
  const void* fn = reinterpret_cast<const void*>(&k_w4_matvec<T, kGroup, kTiles, kR>);
  static std::atomic<int> resident[64];  // CTAs an SM holds, per device; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return IMQ_ERR_CUDA;
  int per_sm = resident[dev].load(std::memory_order_acquire);
  if (per_sm == 0) {
    if (ensure_smem(fn, kSmem) != cudaSuccess || blocks_per_sm(fn, kMvWarps * 32, kSmem, &per_sm) != cudaSuccess || per_sm < 1)
      return IMQ_ERR_CUDA;
    resident[dev].store(per_sm, std::memory_order_release);
  }
  const int64_t sets = (a.N + 16 * kR - 1) / (16 * kR), most = (int64_t)per_sm * num_sms;
  const dim3 grid((unsigned)(sets < most ? sets : most), (unsigned)((a.M + kTokens - 1) / kTokens));
  k_w4_matvec<T, kGroup, kTiles, kR><<<grid, kMvWarps * 32, kSmem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA;
}

// 32 channels a CTA where 16 would put a second CTA on some SMs: X is read and cut up half as often, and the SMs have
// the same work.  Below that 16: twice the CTAs.  bf16, one token, K = 11008: N = 2560 in 8.3 us with 32 and 8.8 with 16,
// N = 2048 in 8.2 and 6.4; fp32, four tokens: 14.3 and 19.7, 14.2 and 10.6.
template <typename T, int kGroup, int kTiles>
imq_status matvec_rows(const MatvecArgs& a, int num_sms, cudaStream_t st) {
  return a.N > 16 * num_sms ? matvec_shape<T, kGroup, kTiles, 2>(a, num_sms, st) : matvec_shape<T, kGroup, kTiles, 1>(a, num_sms, st);
}

template <typename T, int kGroup>
imq_status matvec_tokens(const MatvecArgs& a, int num_sms, cudaStream_t st) {
  const int64_t tokens = a.M < kTokens ? a.M : kTokens;
  if constexpr (sizeof(T) == 2)
    return tokens <= 8 ? matvec_rows<T, kGroup, 1>(a, num_sms, st) : matvec_rows<T, kGroup, 2>(a, num_sms, st);
  else
    return tokens <= 2   ? matvec_rows<T, kGroup, 1>(a, num_sms, st)
           : tokens <= 8 ? matvec_rows<T, kGroup, 3>(a, num_sms, st)
                         : matvec_rows<T, kGroup, 6>(a, num_sms, st);
}

template <typename T>
imq_status matvec_group(const MatvecArgs& a, int group, int num_sms, cudaStream_t st) {
  return group == 32   ? matvec_tokens<T, 32>(a, num_sms, st)
         : group == 64 ? matvec_tokens<T, 64>(a, num_sms, st)
                       : matvec_tokens<T, 128>(a, num_sms, st);
}

bool is_float(imq_dtype t) { return t == IMQ_F32 || t == IMQ_BF16; }
int size_of(imq_dtype t) { return t == IMQ_F32 ? 4 : 2; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Whether W may be read or written 16 bytes at a time along its rows (stored N x K), two entries (K x N).
int vectors(const void* W, int64_t ldw, imq_dtype t, int32_t transW) {
  const uintptr_t unit = transW ? 16 : 2 * size_of(t);
  return ((reinterpret_cast<uintptr_t>(W) | (uintptr_t)(ldw * size_of(t))) & (unit - 1)) == 0;
}

int log2_of(int32_t group) { return group == 32 ? 5 : group == 64 ? 6 : 7; }

int row_alignment(const void* p, int64_t row_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p) | (uintptr_t)row_bytes;
  return x % 16 == 0 ? 16 : x % 4 == 0 ? 4 : 2;
}

// What every call on a 4-bit weight checks.
imq_status check_weight(const void* codes, int64_t ldc, const void* steps, int64_t lds, int64_t K, int64_t N, int32_t group) {
  if (K < 0 || N < 0 || (group != 32 && group != 64 && group != 128)) return IMQ_ERR_ARG;
  if (K > (1 << 30) || N > (1 << 30)) return IMQ_ERR_UNSUPPORTED;
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
  QuantArgs a{W, K, N, ldw, codes, ldc, steps, lds, log2_of(group), vectors(W, ldw, wt, transW), ds->status};
  if (transW) {
    const int64_t ctas = ((N + kRows - 1) / kRows * ((K + 255) / 256) + kQuantWarps - 1) / kQuantWarps;
    if (ctas > INT32_MAX / 8) return IMQ_ERR_UNSUPPORTED;
    if (wt == IMQ_F32)
      k_w4_quantize_rows<float><<<(unsigned)ctas, kQuantWarps * 32, 0, st>>>(a);
    else
      k_w4_quantize_rows<__nv_bfloat16><<<(unsigned)ctas, kQuantWarps * 32, 0, st>>>(a);
  } else {
    const int64_t nb = (K + kBlock - 1) / kBlock;
    if (nb > 65535) return IMQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)((N + kColChannels - 1) / kColChannels), (unsigned)nb);
    if (wt == IMQ_F32)
      k_w4_quantize_cols<float><<<grid, 128, 0, st>>>(a);
    else
      k_w4_quantize_cols<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
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
  DequantArgs a{codes, ldc, steps, lds, K, N, log2_of(group), W, ldw, vectors(W, ldw, wt, transW), kOneF16};
  if (transW) {
    const int64_t ctas = ((N + kRows - 1) / kRows * ((K + 255) / 256) + 7) / 8;
    if (ctas > INT32_MAX / 8) return IMQ_ERR_UNSUPPORTED;
    if (wt == IMQ_F32)
      k_w4_dequantize_rows<float><<<(unsigned)ctas, 256, 0, st>>>(a);
    else
      k_w4_dequantize_rows<__nv_bfloat16><<<(unsigned)ctas, 256, 0, st>>>(a);
  } else {
    const int64_t nb = (K + kBlock - 1) / kBlock;
    if (nb > 65535) return IMQ_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)((N + kColChannels - 1) / kColChannels), (unsigned)nb);
    if (wt == IMQ_F32)
      k_w4_dequantize_cols<float><<<grid, 128, 0, st>>>(a);
    else
      k_w4_dequantize_cols<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
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
  DeviceState* ds;
  s = device_state(&ds);
  if (s != IMQ_OK) return s;
  MatvecArgs a{codes, ldc, steps, lds, K, N, X, ldx, M, Y, ldy, yt == IMQ_BF16,
               row_alignment(X, M == 1 ? 0 : ldx * size_of(xt)), kOneBf16};
  return xt == IMQ_BF16 ? matvec_group<__nv_bfloat16>(a, group, ds->num_sms, st) : matvec_group<float>(a, group, ds->num_sms, st);
}

}  // namespace imq
