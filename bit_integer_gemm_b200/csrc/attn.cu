// attn.cu -- attention of one new token per sequence over the paged low-bit cache (sm_100a).
//
//   s_t = scale * dk_t * sum_d q_d ck[t, d]      p = softmax of s over the sequence's tokens
//   o_d = sum_t p_t dv_t cv[t, d]                lse = log sum_t exp(s_t)
// with ck, cv the codes and dk, dv the steps of the cache.
//
// Bound: the cache is read once, 2 D bits / 8 + 8 bytes a token and key head, for 4 G D operations of G
// query heads -- memory, far below the tensor cores' rate, but above what the fp32 units do at 8 query heads a
// key head.  So both products run on warp-level tensor-core instructions, whose operands are registers: the
// codes go from the copy to the operand without another trip through shared memory.
//   - q * k runs on integers, exactly: a query row is scaled by a power of two so that its largest entry lies between
//     2^30 and 2^31, and rounded to integers of four digits of radix 256 in -128 .. 127 (the unpacking of this library,
//     applied to the query), and the stored bytes or nibbles are the other operand as they lie, offset and
//     all: the offset times the sum of a row's digits is what the sums start from.  8-bit codes need no
//     conversion, 4-bit codes three instructions for eight.  Rows g and g + 8 of one 16-row operand hold the
//     first two digits of up to 8 query heads, a second operand the others; for 9 to 16 heads each digit has
//     an operand.  (One query entry 1000 times as large as the others, on keys that are small there, costs
//     the output 3e-7; with three digits it cost 4e-5.)
//   - p * v runs on fp16 with fp32 sums: codes are exact in fp16; a probability times its value's step, the weight
//     of a code, is cut into two fp16 parts, 22 bits together, in units of the query head's largest weight so far and
//     of 2^-11.  So what a weight loses is at most 2^-36 of the largest of its head.  With up to 8 query heads both
//     parts share one 16-row operand, so the second costs no further instruction.
// The inner axis of a product may be permuted at will if both operands agree, so a lane's 16 (or 8) bytes of a
// key are contiguous ones.  Values are transposed on the way from shared memory (pairs of bytes, or four
// nibbles, of two tokens to a register), and the columns they make are sorted out when the sums are written.
//
// The softmax keeps a reference instead of the running maximum, and so does the unit of the weights: they are raised
// (and the sums rescaled) only when an exponential exceeds the reference's 8 times, or a weight the unit 16 times (the
// room that fp16 leaves above 2^11), so most runs need no exchange between lanes.  A vector of zeros has the step 1
// whatever the others have; it adds nothing, and the unit leaves it out.
//
// Split: the work of all sequences and key heads lies in one line of units of 64 tokens, cut into equal parts, one
// for each CTA that the SMs hold at once; so lengths may differ as they will.  A row (one sequence's tokens of one key
// head) counts four units more than it has, for its queries and its end: without them a CTA whose part is made of many
// short rows came last (64 sequences of 1 to 4097 tokens, 8 key heads of 64: 50.1 us, with them 34.6; 16 of up to 8192
// at 4 bits: 38.8 and 29.7; 64 of up to 2048, 4 key heads of 256: 44.5 and 30.9; 256 of up to 600: 76 and 52.  Of
// thirteen such mixes one takes 25 % more with 2 units, 7 % with 6, 13 % with 8, and one, of 16 heads a key head, 6 % less
// with 6).  A CTA's four warps take runs of 16 tokens in turn, each with its own ring of asynchronous copies (so that a run waits for
// no barrier but the warp's), and join in shared memory.  Rows that several CTAs share join in k_attn_join from partial
// sums in the workspace, in a fixed order.
//
// Measured, both kernels: 64 sequences of 2048 tokens, 32 key heads of 128 at 8 bits, 175 us (6.3 TB/s); one of 131072, 8
// heads, 52 us (5.3 TB/s: memory, and about 8 us of start, ends and join); 64 of 8192 at 4 bits 154 us (3.7 TB/s: a code
// takes as many instructions as at 8 bits, 337 to 356 for 16 tokens and 128 entries, and half the bytes); head size 64
// at 8 query heads a key head 57 us for 64 of 4096 (5.0 TB/s), size 256 94 us for 64 of 2048 (5.8 TB/s); 16 query heads a
// key head, 64 of 4096, 4 key heads of 128: 80 us (3.5 TB/s; twice the matrix instructions, spills); one sequence of 2048
// tokens and 32 heads 10.0 us, which is two dependent launches and a CTA's chain of dependent loads.
#include <atomic>
#include <type_traits>

#include "lowbit.cuh"
#include "internal.h"

namespace imq {
namespace {

constexpr int kWarps = 4;
constexpr int kRun = 16;              // tokens that a warp copies at a time; they lie in one page (pages are multiples of it)
constexpr int kUnit = kWarps * kRun;  // tokens: the grain of the split
constexpr uint32_t kRowCost = 4;      // what a row costs besides its units, in units
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.f;          // how many times an exponential may exceed the reference's
constexpr float kPScale = 2048.f;      // the unit of the weights in fp16,
constexpr float kPMost = 32768.f;      // and the largest weight
constexpr float kUnitFloor = 1e-33f;   // the unit of the weights starts here
constexpr int kDigits = 4;              // of a query entry

struct AttnArgs {
  imq_kv_cache c;
  const void* Q;
  int64_t q_batch, q_head;
  int q_bf16, q_vec;  // q_vec: four entries of a row may be read at once
  int o_bf16, o_vec;
  int group;          // query heads of a key head
  int page_shift;     // page_size = 2^page_shift, or -1
  int head_chunks;    // blocks of up to 8 * kM query heads per key head
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int batch;
  int limit;          // longest sequence the call covers
  int ctas;           // of k_attn
  float scale;
  void* out;
  int64_t o_batch, o_head;
  float* lse;
  int64_t lse_batch;
  float* part;        // [CTA][2][head of the row][D]: sums of rows that several CTAs share
  float2* ml;         // [CTA][2][head of the row]: reference (a power of two's exponent) and sum of the weights
  int32_t* status;
  uint32_t one;       // kOneF16
  uint32_t k_stride16, v_stride16, s_stride16;  // of pages, in 16 bytes
};

// Bytes a lane holds of a token's key (a quarter of the vector), as 16-byte pieces and an 8-byte one.  Piece p of the
// four lanes of a token together is a contiguous part of the vector; in shared memory a piece of a warp is 32
// consecutive slots.
template <int kBits, int kD>
struct Pieces {
  static constexpr int kBytes = kD * kBits / 32, n16 = kBytes / 16, n8 = kBytes % 16 / 8;
  // entry d of a vector (d a multiple of 4): the lane column that holds it and its word among the lane's
  static __device__ __forceinline__ void find(int d, int* column, int* word) {
    const int at = d * kBits / 8;
    if (at < n16 * 64) *column = at % 64 / 16, *word = at / 64 * 4 + at % 16 / 4;
    else *column = (at - n16 * 64) / 8, *word = n16 * 4 + (at - n16 * 64) % 8 / 4;
  }
};
template <typename P>
__device__ __forceinline__ void read_pieces(const uint8_t* src, int lane, uint32_t (&w)[P::kBytes / 4]) {
#pragma unroll
  for (int j = 0; j < P::n16; ++j) {
    const uint4 v = *reinterpret_cast<const uint4*>(src + (j * 32 + lane) * 16);
    w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
  }
  if (P::n8) {
    const uint2 v = *reinterpret_cast<const uint2*>(src + P::n16 * 512 + lane * 8);
    w[4 * P::n16] = v.x, w[4 * P::n16 + 1] = v.y;
  }
}

// Four consecutive entries; vec: they are aligned to their size together.
__device__ __forceinline__ void load4(const float* p, bool vec, float (&x)[4]) {
  if (vec) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = p[j];
  }
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, bool vec, float (&x)[4]) {
  if (vec) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __bfloat162float(p[j]);
  }
}
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t at, float v) {
  if (a.o_bf16)
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(a.out)[at] = v;
}
// Four consecutive entries of out.
__device__ __forceinline__ void store_out4(const AttnArgs& a, int64_t at, const float4& v) {
  if (a.o_bf16) {
    __nv_bfloat16* const p = static_cast<__nv_bfloat16*>(a.out) + at;
    if (a.o_vec) {
      *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
    } else {
      p[0] = __float2bfloat16_rn(v.x), p[1] = __float2bfloat16_rn(v.y), p[2] = __float2bfloat16_rn(v.z), p[3] = __float2bfloat16_rn(v.w);
    }
  } else {
    float* const p = static_cast<float*>(a.out) + at;
    if (a.o_vec) {
      *reinterpret_cast<float4*>(p) = v;
    } else {
      p[0] = v.x, p[1] = v.y, p[2] = v.z, p[3] = v.w;
    }
  }
}

// x as two fp16 parts (hi, lo), pairs packed.
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t* hi, uint32_t* lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / x to the last bit or so: the hardware's approximation and a step of Newton's method.
__device__ __forceinline__ float inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return fmaf(y, fmaf(-x, y, 1.f), y);
}
__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xFF800000u); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

// Units of a sequence (0 for one that has no tokens or that the call does not cover).
__device__ __forceinline__ uint32_t units_of(const AttnArgs& a, int len) {
  return len <= 0 || len > a.limit ? 0u : (uint32_t)(len + kUnit - 1) / kUnit;
}
// A row's length in the line: its units, behind kRowCost places that stand for its start and end.
__device__ __forceinline__ uint32_t cost_of(const AttnArgs& a, int len) {
  const uint32_t n = units_of(a, len);
  return n ? n + kRowCost : 0u;
}
// The parts of the line: `all` places over `n` CTAs, the first all % n take one more.
struct Parts {
  uint32_t each, more;
  __device__ __forceinline__ Parts(uint32_t all, uint32_t n) : each(all / n), more(all % n) {}
  __device__ __forceinline__ uint32_t begin(uint32_t i) const { return each * i + min(i, more); }
  __device__ __forceinline__ uint32_t cta_of(uint32_t u) const {
    const uint32_t big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};

// kM: 1 for up to 8 query heads a key head, 2 for 9 to 16.
template <int kBits, int kD, int kM>
struct Shape {
  using KP = Pieces<kBits, kD>;
  static constexpr int kRow = kD * kBits / 8, kChunks = kRow / 16;
  static constexpr uint32_t kZeros = kBits == 8 ? 0x80808080u : 0x88888888u;  // codes of 0
  // Values lie in rows of 16-byte chunks; eight rows' chunks of one column are in different banks: by an exclusive or
  // of the chunk with the row where a row is a power of two, by a chunk of padding where it is not.
  static constexpr bool kPadded = (kRow & (kRow - 1)) != 0;
  static constexpr int kPitch = kRow + (kPadded ? 16 : 0);
  static __device__ __forceinline__ int chunk_at(int row, int chunk) {
    const int mix = kPadded ? 0 : kRow >= 128 ? row & 7 : kRow == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
    return row * kPitch + (chunk ^ mix) * 16;
  }
  static constexpr int kSteps = kD / 32;               // inner steps of q * k
  static constexpr int kCols = kD / 8;                 // 8-column blocks of p * v
  static constexpr int kValues = 16 * kRow, kStepsAt = kValues + 16 * kPitch;
  static constexpr int kRunBytes = kStepsAt + 128;     // keys, values, steps of 16 tokens
  // about 13 KB for a warp's ring: three CTAs an SM have about 100 KB of copies under way
  static constexpr int kStages = 13000 / kRunBytes < 2 ? 2 : 13000 / kRunBytes > 8 ? 8 : 13000 / kRunBytes;
  static constexpr int kRing = kStages * kRunBytes;
  // CTAs an SM, by the registers of the sums.  At 128 a fourth would cost spills: three take 52 us for 131072 tokens of
  // 8 key heads at 8 bits, four 73.
  static constexpr int kPerSm = kD <= 64 ? 4 : kD <= 128 ? 3 : 2;
  static constexpr int kHeads = 8 * kM;
  static constexpr int kQOps = kDigits / 2 * kM;       // operands of the digits, 512 bytes each a step
  static constexpr int kQBytes = kSteps * kQOps * 512;
  static constexpr int kPad = kD + 4;
  static constexpr int kJoin = kWarps * kHeads * kPad * 4;  // the warps' sums, over the ring
  static constexpr int kSmem = kQBytes + (kWarps * kRing > kJoin ? kWarps * kRing : kJoin);
};

// The query operands of a row's heads.  A warp takes every fourth head, a lane its entries 4i .. 4i + 3 (and 128 further
// on).  Entry (step, operand, lane) is {row g at the step's first four inner positions of column c, row g + 8 at them,
// row g at the second four, row g + 8}; the positions are the ones whose codes a lane's words hold.
template <int kBits, int kD, int kM>
struct Query {
  using S = Shape<kBits, kD, kM>;
  static constexpr int kParts = (kD + 127) / 128, kMine = 8 * kM / kWarps;
  float x[kMine][kParts][4];

  template <typename T>
  __device__ __forceinline__ void load(const T* q, int64_t head_stride, bool vec, int heads, int warp, int lane) {
#pragma unroll
    for (int n = 0; n < kMine; ++n)
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const int h = warp + n * kWarps, d = 4 * lane + 128 * p;
        if (h < heads && d < kD) load4(q + h * head_stride + d, vec, x[n][p]);
        else x[n][p][0] = x[n][p][1] = x[n][p][2] = x[n][p][3] = 0.f;
      }
  }

  __device__ __forceinline__ void write(uint8_t* qs, int32_t (*s_dig)[8 * kM], float* s_mul, int heads, float scale, int warp, int lane) {
#pragma unroll
    for (int n = 0; n < kMine; ++n) {
      const int h = warp + n * kWarps;
      if (h >= heads) break;
      uint32_t key = 0;
#pragma unroll
      for (int p = 0; p < kParts; ++p)
#pragma unroll
        for (int j = 0; j < 4; ++j) key = max(key, abs_key(x[n][p][j]));
      key = __reduce_max_sync(0xffffffffu, key);
      // a row of (almost) zeros, and one that is not finite (its scores' factor is NaN), have digits of 0
      const float top = __uint_as_float(key);
      const bool use = key_finite(key) && top > 1e-30f;
      // e: the exponent (and its offset of 127) of the largest entry, one more where its first digit would pass 127.  The
      // entries are scaled by 2^(30 - (e - 127)) in two factors that fp32 has, without rounding.
      const int e = (int)((key + 0x20000u) >> 23);
      const float r = __int_as_float((260 - e) << 23);
      int32_t sum[kDigits] = {};
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const int d = 4 * lane + 128 * p;
        if (kD % 128 != 0 && d >= kD) continue;
        // v + 128 * (2^24 + 2^16 + 2^8 + 1) has the digits, each plus 128, as its bytes
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = (uint32_t)__float2int_rn(use ? x[n][p][j] * r * 16777216.f : 0.f) + 0x80808080u;
        const uint32_t a = __byte_perm(u[0], u[1], 0x5140), b = __byte_perm(u[2], u[3], 0x5140);
        const uint32_t y = __byte_perm(u[0], u[1], 0x7362), z = __byte_perm(u[2], u[3], 0x7362);
        // first to fourth digits of the four entries
        const uint32_t dig[kDigits] = {__byte_perm(y, z, 0x7632) ^ 0x80808080u, __byte_perm(y, z, 0x5410) ^ 0x80808080u,
                                       __byte_perm(a, b, 0x7632) ^ 0x80808080u, __byte_perm(a, b, 0x5410) ^ 0x80808080u};
        int c, w;
        S::KP::find(d, &c, &w);
#pragma unroll
        for (int k = 0; k < kDigits; ++k) {
          sum[k] = __dp4a((int)dig[k], 0x01010101, sum[k]);
          // kM = 1: operand 0 holds the first digit in row g and the second in row g + 8, operand 1 the third and fourth;
          // kM = 2: an operand a digit, heads g and g + 8
          const int op = kM == 1 ? k / 2 : k, high = kM == 1 ? k % 2 : h / 8, g = kM == 1 ? h : h % 8;
          if constexpr (kBits == 8) {
            // four entries are one word of a key: inner step w / 2, its first or second four positions
            reinterpret_cast<uint32_t*>(qs)[((w / 2 * S::kQOps + op) * 32 + g * 4 + c) * 4 + (w % 2) * 2 + high] = dig[k];
          } else {
            // a word of a key is eight entries, its even nibbles (codes 0, 4, 1, 5) the first four positions of the
            // step and its odd ones (codes 2, 6, 3, 7) the second; these four entries are codes 0-3 or 4-7
            uint8_t* const to = qs + (((w * S::kQOps + op) * 32 + g * 4 + c) * 4 + high) * 4 + d % 8 / 4;
            to[0] = dig[k] & 255, to[2] = dig[k] >> 8 & 255;     // codes 0 and 1 (4 and 5)
            to[8] = dig[k] >> 16 & 255, to[10] = dig[k] >> 24;   // codes 2 and 3 (6 and 7)
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kDigits; ++k) sum[k] = __reduce_add_sync(0xffffffffu, sum[k]);
      // the offset of the stored codes times a row's digits: of the first two digits together, and of the others.  The
      // factor of the scores (as exponents of 2) is scale * 2^(e - 127 - 30) * log2(e), the power again in two factors.
      if (lane == 0) {
        s_mul[h] = !key_finite(key) ? quiet_nan() : use ? scale * __int_as_float((e - 22) << 23) * (kLog2e / 256.f) : 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) s_dig[k][h] = -(1 << (kBits - 1)) * (256 * sum[2 * k] + sum[2 * k + 1]);
      }
    }
  }
};

// A bit for each of a run's 16 value vectors that has a code other than 0.
template <typename S>
__device__ __forceinline__ uint32_t nonzero_rows(const uint8_t* values, int lane) {
  uint32_t rows = 0;
#pragma unroll
  for (int q = 0; q < S::kChunks / 2; ++q) {
    const int at = q * 32 + lane, row = at / S::kChunks;
    const uint4 v = *reinterpret_cast<const uint4*>(values + S::chunk_at(row, at % S::kChunks));
    if (((v.x ^ S::kZeros) | (v.y ^ S::kZeros) | (v.z ^ S::kZeros) | (v.w ^ S::kZeros)) != 0u) rows |= 1u << row;
  }
  return __reduce_or_sync(0xffffffffu, rows);
}

template <int kBits, int kD, int kM>
__global__ void __launch_bounds__(kWarps * 32, Shape<kBits, kD, kM>::kPerSm) k_attn(const __grid_constant__ AttnArgs a) {
  using S = Shape<kBits, kD, kM>;
  using KP = typename S::KP;
  constexpr int kStages = S::kStages, kRow = S::kRow;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* const qs = reinterpret_cast<uint4*>(smem);
  uint8_t* const ring = smem + S::kQBytes;
  __shared__ float s_mul[S::kHeads];
  __shared__ int32_t s_dig[2][S::kHeads];
  __shared__ float s_m[kWarps][S::kHeads], s_l[kWarps][S::kHeads];
  __shared__ __align__(16) int s_part[8];  // the part of a row that the CTA works on

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;");
  // the scores of rows without a head become 0 (their digits are whatever the shared memory holds)
  if (threadIdx.x < S::kHeads) s_mul[threadIdx.x] = 0.f, s_dig[0][threadIdx.x] = s_dig[1][threadIdx.x] = 0;

  // sequences without tokens, and those longer than the call covers, are answered here
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int len = __ldg(a.lens + b);
    if (units_of(a, len)) continue;
    const bool over = len > a.limit;
    if (over && threadIdx.x == 0) set_status(a.status, IMQ_ERR_BOUNDS);
    for (int i = threadIdx.x; i < a.c.n_heads * a.group * kD; i += kWarps * 32)
      store_out(a, b * a.o_batch + i / kD * a.o_head + i % kD, over ? quiet_nan() : 0.f);
    if (a.lse)
      for (int i = threadIdx.x; i < a.c.n_heads * a.group; i += kWarps * 32)
        a.lse[b * a.lse_batch + i] = over ? quiet_nan() : minus_inf();
  }

  // ---- the first warp keeps the CTA's part of the line, u0 .. u1 - 1, the sequence that u0 lies in, and the places before
  // that
  uint32_t u0 = 0, u1 = 0, base = 0;
  int b_now = 0;
  const uint32_t rows = a.c.n_heads * a.head_chunks;
  if (warp == 0) {
    // inclusive sums of the first 32 sequences' places, and the sum of all
    const uint32_t mine = lane < a.batch ? cost_of(a, __ldg(a.lens + lane)) * rows : 0u;
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
      sum += lane >= o ? x : 0u;
    }
    uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
    if (a.batch > 32) {
      uint32_t more = 0;
      for (int i = 32 + lane; i < a.batch; i += 32) more += cost_of(a, __ldg(a.lens + i));
      all += __reduce_add_sync(0xffffffffu, more) * rows;
    }
    const uint32_t ctas = min((uint32_t)a.ctas, all);
    if (blockIdx.x < ctas) {
      const Parts parts(all, ctas);
      u0 = parts.begin(blockIdx.x), u1 = parts.begin(blockIdx.x + 1);
      uint32_t own = mine;
      for (;;) {
        const unsigned behind = __ballot_sync(0xffffffffu, base + sum > u0);
        if (behind) {
          const int l = __ffs(behind) - 1;
          b_now += l;
          base += __shfl_sync(0xffffffffu, sum - own, l);
          break;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
        b_now += 32;
        own = b_now + lane < a.batch ? cost_of(a, __ldg(a.lens + b_now + lane)) * rows : 0u;
        sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
          sum += lane >= o ? x : 0u;
        }
      }
    }
  }

  // ---- a row's part after the other
  for (;;) {
    if (warp == 0) {
      uint32_t take = 0, per_row = 0, row = 0, unit = 0;
      int len = 0;
      while (u0 < u1 && take == 0) {
        len = __ldg(a.lens + b_now);
        const uint32_t cost = cost_of(a, len);
        if (u0 - base >= cost * rows) {
          base += cost * rows;
          ++b_now;
          continue;
        }
        per_row = units_of(a, len);
        row = (u0 - base) / cost;
        const uint32_t at = (u0 - base) - row * cost, to = min(cost, at + (u1 - u0));  // this CTA's places of the row
        unit = at > kRowCost ? at - kRowCost : 0u;
        take = to > kRowCost ? to - kRowCost - unit : 0u;
        u0 += to - at;
      }
      if (lane == 0) {
        *reinterpret_cast<int4*>(s_part) = make_int4(b_now, (int)row, (int)unit, (int)take);
        *reinterpret_cast<int2*>(s_part + 4) = make_int2(len, (int)per_row);
      }
    }
    __syncthreads();
    const int4 part = *reinterpret_cast<const int4*>(s_part);
    const int b = part.x, row = part.y, unit = part.z, take = part.w, len = s_part[4], per_row = s_part[5];
    if (take == 0) return;
    const int begin = unit * kUnit, end = min(len, begin + take * kUnit), first = begin + warp * kRun;
    const int kv = a.head_chunks == 1 ? row : row / a.head_chunks;
    const int h0 = kv * a.group + (row - kv * a.head_chunks) * S::kHeads, heads = min(S::kHeads, (kv + 1) * a.group - h0);
    const int32_t* const table = a.table + b * a.table_stride;
    const int n_runs = first < end ? (end - first + kUnit - 1) / kUnit : 0;

    Query<kBits, kD, kM> query;
    {
      const int64_t q0 = b * a.q_batch + h0 * a.q_head;
      if (a.q_bf16) query.load(static_cast<const __nv_bfloat16*>(a.Q) + q0, a.q_head, a.q_vec, heads, warp, lane);
      else query.load(static_cast<const float*>(a.Q) + q0, a.q_head, a.q_vec, heads, warp, lane);
    }

    // Where the warp's runs u .. u + 31 lie, one a lane: the offsets of their page and place in the cache's keys, values
    // and steps, in 16 bytes; kNowhere for a page outside the cache.
    constexpr uint32_t kNowhere = 0xFFFFFFFFu;
    struct Place {
      uint32_t k, v, s;
    };
    auto locate = [&](int u) {
      Place at{kNowhere, 0u, 0u};
      u += lane;
      if (u < n_runs) {
        const uint32_t t = first + u * kUnit, j = a.page_shift >= 0 ? t >> a.page_shift : t / (uint32_t)a.c.page_size;
        const int32_t page = __ldg(table + j);
        const uint32_t place = t - j * (uint32_t)a.c.page_size + kv * (uint32_t)a.c.page_size;
        if (page >= 0 && page < a.c.n_pages)
          at = {page * a.k_stride16 + place * (kRow / 16), page * a.v_stride16 + place * (kRow / 16), page * a.s_stride16 + place / 2};
      }
      return at;
    };
    Place now = locate(0), next{kNowhere, 0u, 0u};
    if (n_runs > 32) next = locate(32);

    // ---- the warp's copies
    const uint32_t mine = smem_addr(ring) + warp * S::kRing;
    bool bad = false;
    uint32_t fill = mine;  // the stage that is filled next
    auto issue = [&](int u) {
      if (u < n_runs) {
        const int left = end - (first + u * kUnit);
        if ((u & 31) == 0 && u > 0) {
          now = next;
          next = locate(u + 32);
        }
        const uint32_t ko = __shfl_sync(0xffffffffu, now.k, u & 31), vo = __shfl_sync(0xffffffffu, now.v, u & 31);
        const uint32_t so = __shfl_sync(0xffffffffu, now.s, u & 31);
        const uint8_t* const kp = a.c.k + (uint64_t)ko * 16 + (g * kRow + c * 16);
        const uint8_t* const vp = a.c.v + (uint64_t)vo * 16 + lane * 16;
        const uint8_t* const sp = reinterpret_cast<const uint8_t*>(a.c.steps) + (uint64_t)so * 16 + lane * 16;
        const uint32_t to16 = fill + lane * 16, to8 = fill + lane * 8 + KP::n16 * 512;
        if (left >= kRun && ko != kNowhere) {
          // keys: tokens g and g + 8, this lane's quarter; values: the run's bytes in order
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int q = 0; q < KP::n16; ++q) cp_async<16>(to16 + j * 8 * kRow + q * 512, kp + j * 8 * kRow + q * 64);
            if (KP::n8) cp_async<8>(to8 + j * 8 * kRow, kp - 8 * c + j * 8 * kRow + 64 * KP::n16);
          }
#pragma unroll
          for (int q = 0; q < S::kChunks / 2; ++q) {
            const int at = q * 32 + lane;
            cp_async<16>(fill + S::kValues + S::chunk_at(at / S::kChunks, at % S::kChunks), vp + q * 512);
          }
          if (lane < 8) cp_async<16>(to16 + S::kStepsAt, sp);
        } else {
          // the end of the sequence, or a page outside the cache: what is not read is zero-filled (steps of 0: no
          // stale value meets a weight of 0), with an address that is not read either
          const int valid = ko == kNowhere ? 0 : min(left, kRun);
          bad |= ko == kNowhere;
#pragma unroll 1
          for (int j = 0; j < 2; ++j) {
            const bool on = 8 * j + g < valid;
            const uint8_t* from = on ? kp + j * 8 * kRow : a.c.k;
#pragma unroll
            for (int q = 0; q < KP::n16; ++q) cp_async_part<16>(to16 + j * 8 * kRow + q * 512, from + (on ? q * 64 : 0), on ? 16u : 0u);
            if (KP::n8) cp_async_part<8>(to8 + j * 8 * kRow, from + (on ? 64 * KP::n16 - 8 * c : 0), on ? 8u : 0u);
          }
#pragma unroll 1
          for (int q = 0; q < S::kChunks / 2; ++q) {
            const int at = q * 32 + lane;
            const bool on = at / S::kChunks < valid;
            cp_async_part<16>(fill + S::kValues + S::chunk_at(at / S::kChunks, at % S::kChunks), on ? vp + q * 512 : a.c.v, on ? 16u : 0u);
          }
          const int n = min(max(valid - 2 * lane, 0), 2);
          if (lane < 8) cp_async_part<16>(to16 + S::kStepsAt, n ? sp : reinterpret_cast<const uint8_t*>(a.c.steps), 8u * n);
        }
        fill = fill + S::kRunBytes == mine + S::kRing ? mine : fill + S::kRunBytes;
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // ---- the query operands, while the first copies are under way
    query.write(smem, s_dig, s_mul, heads, a.scale, warp, lane);
    __syncthreads();
    float mul[kM];
    int32_t start[2][kM];  // the offset's part of the first two digits' sums together, and of the others'
#pragma unroll
    for (int r = 0; r < kM; ++r) {
      mul[r] = s_mul[g + 8 * r];
#pragma unroll
      for (int k = 0; k < 2; ++k) start[k][r] = s_dig[k][g + 8 * r];
    }

    constexpr bool kQInRegs = kM == 1 && kD <= 128;  // at most 32 registers
    uint4 qr[kQInRegs ? S::kSteps * S::kQOps : 1];
    if constexpr (kQInRegs) {
#pragma unroll
      for (int i = 0; i < S::kSteps * S::kQOps; ++i) qr[i] = qs[i * 32 + lane];
    }

    // ---- the warp's runs
    float o[S::kCols][4] = {};
    // of a head: the reference's exponent, the sum of the exponentials, and the unit of the weights (of an exponential of 1
    // and a step of 1)
    float m[kM], l[kM], wunit[kM], winv[kM];
#pragma unroll
    for (int r = 0; r < kM; ++r) m[r] = minus_inf(), l[r] = 0.f, wunit[r] = kUnitFloor, winv[r] = kPScale / kUnitFloor;
    const uint8_t* run = ring + warp * S::kRing;

#pragma unroll 1
    for (int u = 0; u < n_runs; ++u) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // other lanes copied parts of the run; and every lane is done with the run that is overwritten now
      issue(u + kStages - 1);
      // ---- scores, two blocks of eight tokens; this lane's tokens are 2c, 2c + 1, 2c + 8, 2c + 9, its heads g (and g + 8)
      constexpr int kMine = 4;
      float x[kM][kMine];
      {
        int32_t acc[2][S::kQOps][4] = {};
        uint32_t w[2][KP::kBytes / 4];
#pragma unroll
        for (int j = 0; j < 2; ++j) read_pieces<KP>(run + j * 8 * kRow, lane, w[j]);
#pragma unroll
        for (int st = 0; st < S::kSteps; ++st) {
#pragma unroll
          for (int op = 0; op < S::kQOps; ++op) {
            const uint4 q = kQInRegs ? qr[kQInRegs ? st * S::kQOps + op : 0] : qs[(st * S::kQOps + op) * 32 + lane];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t b0 = kBits == 8 ? w[j][kBits == 8 ? 2 * st : 0] : w[j][kBits == 8 ? 0 : st] & 0x0F0F0F0Fu;
              const uint32_t b1 = kBits == 8 ? w[j][kBits == 8 ? 2 * st + 1 : 0] : w[j][kBits == 8 ? 0 : st] >> 4 & 0x0F0F0F0Fu;
              mma_s8u8(acc[j][op], q.x, q.y, q.z, q.w, b0, b1);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < kM; ++r)
#pragma unroll
          for (int j = 0; j < kMine; ++j) {
            const auto& sum = acc[j >> 1];
            int32_t d[kDigits];
#pragma unroll
            for (int k = 0; k < kDigits; ++k)
              d[k] = kM == 1 ? sum[k / 2][k % 2 * 2 + (j & 1)] : sum[kM == 1 ? 0 : k][2 * r + (j & 1)];
            // at 256 dimensions 256 * d[0] + d[1] still lies within 2^31
            x[r][j] = fmaf((float)(d[0] * 256 + d[1] + start[0][r]), 65536.f, (float)(d[2] * 256 + d[3] + start[1][r]));
          }
      }
      float ks[kMine], vs[kMine];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 st = *reinterpret_cast<const float4*>(run + S::kStepsAt + j * 64 + c * 16);
        ks[2 * j] = st.x, vs[2 * j] = st.y, ks[2 * j + 1] = st.z, vs[2 * j + 1] = st.w;
      }
#pragma unroll
      for (int r = 0; r < kM; ++r)
#pragma unroll
        for (int j = 0; j < kMine; ++j) x[r][j] *= ks[j] * mul[r];
      const int left = end - (first + u * kUnit);
      if (left < kRun) {
#pragma unroll
        for (int j = 0; j < kMine; ++j)
          if (8 * (j >> 1) + 2 * c + (j & 1) >= left) {
#pragma unroll
            for (int r = 0; r < kM; ++r) x[r][j] = minus_inf();
          }
      }
      // ---- exponentials, and the weights of the codes
      float p[kM][kMine], wt[kM][kMine];
      bool raise = false;
#pragma unroll
      for (int r = 0; r < kM; ++r) {
        float pmax = 0.f, wmax = 0.f;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          p[r][j] = ex2(x[r][j] - m[r]);
          wt[r][j] = p[r][j] * vs[j] * winv[r];
          pmax = fmaxf(pmax, p[r][j]), wmax = fmaxf(wmax, wt[r][j]);
        }
        raise |= pmax > kSlack || wmax > kPMost;
      }
      if (__any_sync(0xffffffffu, raise)) {
        // vectors of zeros: their step of 1 is no weight
        bool one = false;
#pragma unroll
        for (int j = 0; j < kMine; ++j) one |= vs[j] == 1.f;
        if (__any_sync(0xffffffffu, one)) {
          const uint32_t live = nonzero_rows<S>(run + S::kValues, lane);
#pragma unroll
          for (int j = 0; j < kMine; ++j)
            if (vs[j] == 1.f && !(live >> (8 * (j >> 1) + 2 * c + (j & 1)) & 1)) vs[j] = 0.f;
        }
        // new references and units, the largest so far, and the sums in their terms
        float fix[kM];
#pragma unroll
        for (int r = 0; r < kM; ++r) {
          float top = x[r][0];
#pragma unroll
          for (int j = 1; j < kMine; ++j) top = fmaxf(top, x[r][j]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)), m[r]);
          const float alpha = top == minus_inf() ? 1.f : ex2(m[r] - top);  // (no score yet but NaN)
          m[r] = top;
          l[r] *= alpha;
          float most = 0.f;
#pragma unroll
          for (int j = 0; j < kMine; ++j) {
            p[r][j] = ex2(x[r][j] - top);
            wt[r][j] = p[r][j] * vs[j];
            most = fmaxf(most, wt[r][j]);
          }
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const float old = wunit[r] * alpha;
          wunit[r] = fmaxf(fmaxf(most, old), kUnitFloor);
          fix[r] = __fdividef(old, wunit[r]);
          winv[r] = __fdividef(kPScale, wunit[r]);
#pragma unroll
          for (int j = 0; j < kMine; ++j) wt[r][j] *= winv[r];
        }
        if (u > 0) {
#pragma unroll
          for (int n = 0; n < S::kCols; ++n) {
            o[n][0] *= fix[0], o[n][1] *= fix[0];
            o[n][2] *= fix[kM - 1], o[n][3] *= fix[kM - 1];
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kM; ++r)
#pragma unroll
        for (int j = 0; j < kMine; ++j) l[r] += p[r][j];
      uint32_t hi[kM][2], lo[kM][2];  // weights as operands
#pragma unroll
      for (int r = 0; r < kM; ++r) {
        split_f16(wt[r][0], wt[r][1], &hi[r][0], &lo[r][0]);
        split_f16(wt[r][2], wt[r][3], &hi[r][1], &lo[r][1]);
      }
      auto product = [&](float (&acc)[4], uint32_t b0, uint32_t b1) {
        if (kM == 1) {
          mma_f16(acc, hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
        } else {
          mma_f16(acc, hi[0][0], hi[kM - 1][0], hi[0][1], hi[kM - 1][1], b0, b1);
          mma_f16(acc, lo[0][0], lo[kM - 1][0], lo[0][1], lo[kM - 1][1], b0, b1);
        }
      };
#pragma unroll
      for (int q = 0; q < S::kChunks; q += 2) {
        // chunks q and q + 1 of tokens 0-7 and 8-15; a register holds two bytes (four nibbles) of tokens 2c and 2c + 1
        uint32_t w[4];
        ldmatrix_trans4(smem_addr(run) + S::kValues + S::chunk_at(lane % 16, q + lane / 16), w);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = w[2 * e], y = w[2 * e + 1];
          if constexpr (kBits == 8) {
            product(o[2 * (q + e)], bytes_f16(x, 0x5250, a.one), bytes_f16(y, 0x5250, a.one));
            product(o[2 * (q + e) + 1], bytes_f16(x, 0x5351, a.one), bytes_f16(y, 0x5351, a.one));
          } else {
            product(o[4 * (q + e)], nibbles_f16<false>(x, a.one), nibbles_f16<false>(y, a.one));
            product(o[4 * (q + e) + 1], nibbles_f16<true>(x, a.one), nibbles_f16<true>(y, a.one));
            product(o[4 * (q + e) + 2], nibbles_f16<false>(x >> 8, a.one), nibbles_f16<false>(y >> 8, a.one));
            product(o[4 * (q + e) + 3], nibbles_f16<true>(x >> 8, a.one), nibbles_f16<true>(y >> 8, a.one));
          }
        }
      }
      run = run + S::kRunBytes == ring + (warp + 1) * S::kRing ? ring + warp * S::kRing : run + S::kRunBytes;
    }
    cp_async_wait<0>();

    // ---- join the warps' sums
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) set_status(a.status, IMQ_ERR_BOUNDS);
#pragma unroll
    for (int r = 0; r < kM; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (c == 0) s_m[warp][g + 8 * r] = m[r];
    }
    __syncthreads();  // the rings are done with: they hold the sums from here
    float* const sums = reinterpret_cast<float*>(ring);  // [warp][head][kPad]
#pragma unroll
    for (int r = 0; r < kM; ++r) {
      float top = s_m[0][g + 8 * r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][g + 8 * r]);
      const float weight = top == minus_inf() ? 1.f : ex2(m[r] - top), f = weight * (wunit[r] * (1.f / kPScale));
      if (c == 0) s_l[warp][g + 8 * r] = bad ? quiet_nan() : l[r] * weight;
      float* const row = sums + (warp * S::kHeads + g + 8 * r) * S::kPad;
#pragma unroll
      for (int n = 0; n < S::kCols; n += 8 / kBits * 2) {
        // 8 bits: block 2q + e, column i is entry 16q + 2i + e, so this lane's two columns of two blocks are entries
        // 16q + 4c .. + 3.  4 bits: block 4q + i, column 2j + e is entry 32q + 8j + 2i + e, so two blocks give four
        // entries from 32q + 8c + 2i.
        auto sum = [&](int k, int e) { return (kM == 1 ? o[k][e] + o[k][2 + e] : o[k][2 * r + e]) * f; };
        if constexpr (kBits == 8) {
          *reinterpret_cast<float4*>(row + 8 * n + 4 * c) = make_float4(sum(n, 0), sum(n + 1, 0), sum(n, 1), sum(n + 1, 1));
        } else {
#pragma unroll
          for (int i = 0; i < 4; i += 2)
            *reinterpret_cast<float4*>(row + 8 * n + 8 * c + 2 * i) =
                make_float4(sum(n + i, 0), sum(n + i, 1), sum(n + i + 1, 0), sum(n + i + 1, 1));
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < heads * (kD / 4); i += kWarps * 32) {
      const int h = i / (kD / 4), d = i % (kD / 4) * 4;
      float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(sums + (w * S::kHeads + h) * S::kPad + d);
        num.x += x.x, num.y += x.y, num.z += x.z, num.w += x.w;
        den += s_l[w][h];
      }
      const bool shared = take < per_row;  // part of a row: the one that begins it in the second place
      const int64_t at = (blockIdx.x * 2 + (unit == 0 ? 1 : 0)) * S::kHeads + h;
      if (shared) {
        *reinterpret_cast<float4*>(a.part + at * kD + d) = num;
      } else {
        const float f = inverse(den);
        store_out4(a, b * a.o_batch + (h0 + h) * a.o_head + d, make_float4(num.x * f, num.y * f, num.z * f, num.w * f));
      }
      if (d == 0 && (shared || a.lse)) {
        const float top = fmaxf(fmaxf(s_m[0][h], s_m[1][h]), fmaxf(s_m[2][h], s_m[3][h]));
        if (shared) a.ml[at] = make_float2(top, den);
        else a.lse[b * a.lse_batch + h0 + h] = kLn2 * ((top == minus_inf() ? 0.f : top) + lg2(den));
      }
    }
    __syncthreads();  // before the next part's copies and operands
  }
}

constexpr int kJoinWarps = 8;

// Joins the parts of a row that several CTAs hold.  A lane has four entries (and four more at 128).  Few parts: a warp
// takes a head; many: all warps share a head's parts (always: 43.5 us for 64 sequences of 1 to 4097 tokens, 34.6 as it
// is).  A CTA takes a row; a head where that makes no more CTAs than two to one of k_attn's (one sequence of 131072: 51.7
// us, by rows 58.0; the 64 sequences by heads: 47.1 us).
__global__ void __launch_bounds__(kJoinWarps * 32, 4) k_attn_join(const __grid_constant__ AttnArgs a, int heads_of_cta, int per_head) {
  __shared__ float s_num[kJoinWarps][256], s_den[kJoinWarps], s_top[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
  const int D = a.c.head_dim;
  // per_head: a CTA a head; else a CTA a row
  const uint32_t rows = a.c.n_heads * a.head_chunks;
  const uint32_t row = per_head ? blockIdx.x / a.group * a.head_chunks + blockIdx.x % a.group / heads_of_cta : blockIdx.x;
  const uint32_t per_row = units_of(a, __ldg(a.lens + b));
  uint32_t before = 0, all = 0;  // places of the sequences before b, and of all
  for (int i = lane; i < a.batch; i += 32) {
    const uint32_t n = cost_of(a, __ldg(a.lens + i));
    all += n;
    if (i < b) before += n;
  }
  before = __reduce_add_sync(0xffffffffu, before) * rows;
  all = __reduce_add_sync(0xffffffffu, all) * rows;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // by every thread: this grid ends after k_attn's
  if (per_row <= 1) return;
  const Parts parts(all, min((uint32_t)a.ctas, all));
  const uint32_t first = before + row * (per_row + kRowCost) + kRowCost;  // the row's first unit
  const uint32_t c0 = parts.cta_of(first), c1 = parts.cta_of(first + per_row - 1);
  if (c0 == c1) return;  // one CTA had the whole row and has written it
  const int n = (int)(c1 - c0 + 1);
  const int kv = row / a.head_chunks, h0 = kv * a.group + row % a.head_chunks * heads_of_cta;
  const int h_from = per_head ? (int)blockIdx.x - h0 : 0, heads = per_head ? h_from + 1 : min(heads_of_cta, (kv + 1) * a.group - h0);

  float top, den;
  float4 num[2];
  // parts s, s + every, ...: four at a time, so that their loads are under way together
  auto add = [&](int h, int s, int every) {
    top = minus_inf(), den = 0.f;
    num[0] = num[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (; s < n; s += 4 * every) {
      float2 ml[4];
      float4 x[4];
      auto at = [&](int j) {
        const int t = min(s + j * every, n - 1);  // behind the last part: read, and not used
        return ((int64_t)(c0 + t) * 2 + (t == 0 ? 1 : 0)) * heads_of_cta + h;
      };
      auto load = [&](int k) {
        if (4 * lane + 128 * k < D)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const float4*>(a.part + at(j) * D + 4 * lane + 128 * k);
      };
#pragma unroll
      for (int j = 0; j < 4; ++j) ml[j] = a.ml[at(j)];
      load(0);
      float up = top;
#pragma unroll
      for (int j = 0; j < 4; ++j) up = fmaxf(up, ml[j].x);
      const float ref = up == minus_inf() ? 0.f : up, f = ex2(top - ref);
      float w[4];
      top = up;
      den *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool on = s + j * every < n;
        w[j] = on ? ex2(ml[j].x - ref) : 0.f;
        den += on ? w[j] * ml[j].y : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (4 * lane + 128 * k >= D) break;
        if (k) load(k);
        num[k].x *= f, num[k].y *= f, num[k].z *= f, num[k].w *= f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          num[k].x += w[j] * x[j].x, num[k].y += w[j] * x[j].y, num[k].z += w[j] * x[j].z, num[k].w += w[j] * x[j].w;
      }
    }
  };
  auto write_lse = [&](int h, float ref, float sum) {
    if (a.lse) a.lse[b * a.lse_batch + h0 + h] = kLn2 * ((ref == minus_inf() ? 0.f : ref) + lg2(sum));
  };
  if (n <= kJoinWarps && !per_head) {
    for (int h = warp; h < heads; h += kJoinWarps) {
      add(h, 0, 1);
      const float f = 1.f / den;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (4 * lane + 128 * k < D)
          store_out4(a, b * a.o_batch + (h0 + h) * a.o_head + 4 * lane + 128 * k,
                     make_float4(num[k].x * f, num[k].y * f, num[k].z * f, num[k].w * f));
      if (lane == 0) write_lse(h, top, den);
    }
    return;
  }
  for (int h = h_from; h < heads; ++h) {
    add(h, warp, kJoinWarps);
    if (lane == 0) s_den[warp] = den, s_top[warp] = top;
#pragma unroll
    for (int k = 0; k < 2; ++k) *reinterpret_cast<float4*>(&s_num[warp][4 * lane + 128 * k]) = num[k];
    __syncthreads();
    top = s_top[0];
    for (int w = 1; w < kJoinWarps; ++w) top = fmaxf(top, s_top[w]);
    const float ref = top == minus_inf() ? 0.f : top;
    const int d = threadIdx.x;
    float sum = 0.f;
    den = 0.f;
    for (int w = 0; w < kJoinWarps; ++w) {
      const float f = ex2(s_top[w] - ref);
      sum += f * s_num[w][d];
      den += f * s_den[w];
    }
    if (d < D) store_out(a, b * a.o_batch + (h0 + h) * a.o_head + d, sum / den);
    if (d == 0) write_lse(h, top, den);
    __syncthreads();
  }
}

int heads_of_cta(int group) { return group > 8 ? 16 : 8; }

// CTAs of k_attn: as many as the SMs hold at once (each takes an equal part of the line), or one a place.
int64_t most_places(int64_t batch, int64_t rows, int64_t limit) { return batch * rows * ((limit + kUnit - 1) / kUnit + kRowCost); }
bool has_parts(int64_t limit) { return limit > kUnit; }

// What launch_main does: fill in a.ctas only; launch with room for `bytes` of workspace (IMQ_ERR_BUFFER if that is
// too little).
struct Launch {
  bool only_count;
  void* workspace;
  size_t bytes;
  cudaStream_t st;
};

size_t workspace_of(const AttnArgs& a) {
  return has_parts(a.limit) ? (size_t)a.ctas * 2 * heads_of_cta(a.group) * ((size_t)a.c.head_dim * 4 + 8) : 0;
}

template <int kBits, int kD, int kM>
imq_status launch_shape(AttnArgs& a, int num_sms, int64_t rows, const Launch& l) {
  constexpr int kSmem = Shape<kBits, kD, kM>::kSmem;
  const void* fn = reinterpret_cast<const void*>(&k_attn<kBits, kD, kM>);
  static std::atomic<int> resident[64];  // CTAs an SM holds, per device; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return IMQ_ERR_CUDA;
  int per_sm = resident[dev].load(std::memory_order_acquire);
  if (per_sm == 0) {
    if (ensure_smem(fn, kSmem) != cudaSuccess || blocks_per_sm(fn, kWarps * 32, kSmem, &per_sm) != cudaSuccess || per_sm < 1)
      return IMQ_ERR_CUDA;
    resident[dev].store(per_sm, std::memory_order_release);
  }
  const int64_t most = most_places(a.batch, rows, a.limit);
  a.ctas = (int)(most < 1 ? 1 : most < (int64_t)per_sm * num_sms ? most : (int64_t)per_sm * num_sms);
  if (l.only_count) return IMQ_OK;
  if (has_parts(a.limit)) {
    if (!l.workspace || l.bytes < workspace_of(a)) return IMQ_ERR_BUFFER;
    a.part = static_cast<float*>(l.workspace);
    a.ml = reinterpret_cast<float2*>(a.part + (size_t)a.ctas * 2 * (8 * kM) * kD);
  }
  k_attn<kBits, kD, kM><<<a.ctas, kWarps * 32, kSmem, l.st>>>(a);
  return cudaGetLastError() == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA;
}

template <int kBits, int kM>
imq_status launch_dim(AttnArgs& a, int num_sms, int64_t rows, const Launch& l) {
  switch (a.c.head_dim) {
    case 64: return launch_shape<kBits, 64, kM>(a, num_sms, rows, l);
    case 128: return launch_shape<kBits, 128, kM>(a, num_sms, rows, l);
    case 192: return launch_shape<kBits, 192, kM>(a, num_sms, rows, l);
    default: return launch_shape<kBits, 256, kM>(a, num_sms, rows, l);
  }
}

imq_status launch_main(AttnArgs& a, const Launch& l) {
  DeviceState* ds;
  const imq_status s = device_state(&ds);
  if (s != IMQ_OK) return s;
  a.status = ds->status, a.one = kOneF16;
  const int64_t rows = (int64_t)a.head_chunks * a.c.n_heads;
  const bool wide = heads_of_cta(a.group) == 16;
  if (a.c.bits == 4) return wide ? launch_dim<4, 2>(a, ds->num_sms, rows, l) : launch_dim<4, 1>(a, ds->num_sms, rows, l);
  return wide ? launch_dim<8, 2>(a, ds->num_sms, rows, l) : launch_dim<8, 1>(a, ds->num_sms, rows, l);
}

imq_status check_shape(const imq_kv_cache* c, int64_t batch, int32_t q_heads, int64_t max_len) {
  imq_status s = check_cache(c);
  if (s != IMQ_OK) return s;
  if (batch < 0 || q_heads < 1 || max_len < 0 || q_heads % c->n_heads != 0) return IMQ_ERR_ARG;
  const int64_t group = q_heads / c->n_heads, per = heads_of_cta((int)group), rows = (group + per - 1) / per * c->n_heads;
  if (batch > 65535 || q_heads > 65535 || max_len > (1 << 30) || most_places(batch, rows, max_len) > INT32_MAX)
    return IMQ_ERR_UNSUPPORTED;
  return IMQ_OK;
}
}  // namespace

imq_status paged_attention_workspace(const imq_kv_cache* c, int64_t batch, int32_t q_heads, int64_t max_len, size_t* bytes) {
  if (!bytes) return IMQ_ERR_ARG;
  imq_status s = check_shape(c, batch, q_heads, max_len);
  if (s != IMQ_OK) return s;
  AttnArgs a = {};
  a.c = *c, a.batch = (int)batch, a.limit = (int)max_len, a.group = q_heads / c->n_heads;
  const int per = heads_of_cta(a.group);
  a.head_chunks = (a.group + per - 1) / per;
  s = launch_main(a, {true, nullptr, 0, nullptr});
  if (s == IMQ_OK) *bytes = workspace_of(a);
  return s;
}

imq_status launch_paged_attention(const imq_kv_cache* c, const void* Q, imq_dtype qt, int64_t q_batch, int64_t q_head,
                                  int64_t batch, int32_t q_heads, const int32_t* table, int64_t table_stride,
                                  int64_t table_width, const int32_t* lens, int64_t max_len, float scale, void* out,
                                  imq_dtype ot, int64_t o_batch, int64_t o_head, float* lse, int64_t lse_batch,
                                  void* workspace, size_t workspace_bytes, cudaStream_t st) {
  imq_status s = check_shape(c, batch, q_heads, max_len);
  if (s != IMQ_OK) return s;
  if ((qt != IMQ_F32 && qt != IMQ_BF16) || (ot != IMQ_F32 && ot != IMQ_BF16)) return IMQ_ERR_ARG;
  if (q_batch < 0 || q_head < 0 || o_batch < 0 || o_head < 0 || lse_batch < 0 || table_width < 0 || table_stride < 0 ||
      max_len > table_width * c->page_size)
    return IMQ_ERR_ARG;
  if (batch == 0) return IMQ_OK;
  if (!Q || !lens || !out || (table_width > 0 && !table)) return IMQ_ERR_ARG;
  const uintptr_t qp = reinterpret_cast<uintptr_t>(Q);
  if ((qp & (qt == IMQ_F32 ? 3 : 1)) || (reinterpret_cast<uintptr_t>(out) & (ot == IMQ_F32 ? 3 : 1)) ||
      ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(table)) & 3) ||
      (reinterpret_cast<uintptr_t>(workspace) & 15))
    return IMQ_ERR_ARG;
  if (!vectors_apart(batch, o_batch, q_heads, o_head, c->head_dim) || (lse && batch > 1 && lse_batch < q_heads)) return IMQ_ERR_ARG;
  AttnArgs a = {};
  a.c = *c;
  a.k_stride16 = (uint32_t)(c->k_page_stride / 16), a.v_stride16 = (uint32_t)(c->v_page_stride / 16);
  a.s_stride16 = (uint32_t)(c->steps_page_stride / 4);
  a.Q = Q, a.q_batch = q_batch, a.q_head = q_head, a.q_bf16 = qt == IMQ_BF16;
  const int64_t q_size = qt == IMQ_F32 ? 4 : 2;
  a.q_vec = ((qp | (uintptr_t)(q_batch * q_size) | (uintptr_t)(q_head * q_size)) & (4 * q_size - 1)) == 0;
  a.group = q_heads / c->n_heads;
  const int per = heads_of_cta(a.group);
  a.head_chunks = (a.group + per - 1) / per;
  a.page_shift = (c->page_size & (c->page_size - 1)) == 0 ? __builtin_ctz(c->page_size) : -1;
  a.table = table, a.table_stride = table_stride, a.lens = lens, a.batch = (int)batch, a.limit = (int)max_len;
  a.scale = scale;
  a.out = out, a.o_batch = o_batch, a.o_head = o_head, a.o_bf16 = ot == IMQ_BF16;
  const int64_t o_size = ot == IMQ_F32 ? 4 : 2;
  a.o_vec = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(o_batch * o_size) | (uintptr_t)(o_head * o_size)) & (4 * o_size - 1)) == 0;
  a.lse = lse, a.lse_batch = lse_batch;
  s = launch_main(a, {false, workspace, workspace_bytes, st});
  if (s != IMQ_OK || !has_parts(max_len)) return s;
  // launched before k_attn has finished; it waits for it on the device
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int rows = a.head_chunks * c->n_heads, per_head = batch * q_heads <= 2 * a.ctas;
  cfg.gridDim = dim3((unsigned)(per_head ? q_heads : rows), (unsigned)batch);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attn_join, a, per, per_head) == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA;
}

}  // namespace imq
