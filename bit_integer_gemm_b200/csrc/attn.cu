// attn.cu -- attention of one new token per sequence over the paged low-bit cache (sm_100a).
//
//   s_t = scale * dk_t * sum_d q_d ck[t, d]      p = softmax of s over the sequence's tokens
//   o_d = sum_t p_t dv_t cv[t, d]                lse = log sum_t exp(s_t)
// with ck, cv the codes and dk, dv the steps of the cache.
//
// Bound: the cache is read once, 2 D bits / 8 + 8 bytes a token and key head, for 4 G D operations of G
// query heads -- memory, far below the tensor cores' rate, but above what fp32 units do at 8 query heads a
// key head.  So the products run on the warp-level tensor-core instruction (16 x 8 x 16, fp16 with fp32
// sums), whose operands are registers: the codes go from the copy to the operand without another trip
// through shared memory, and every fp16 value on the way is exact.
//   - Codes in -127..127 are exact in fp16.
//   - A query is scaled by a power of two to put its largest entry near 2^15 and cut into two fp16 parts, 22
//     bits together.  With up to 8 query heads a key head both parts share one 16-row operand (rows g and
//     g + 8), so the second part costs no further instruction; 9 to 16 heads take a product per part.
//   - A probability is weighted with its value's step relative to the largest step so far, scaled by 2^15
//     and cut into two fp16 parts in the same way.  The running maxima of the scores and of the steps
//     rescale the sums when they grow.
// The inner axis of a product may be permuted at will if both operands agree, so a lane's 16 (8, 4) bytes
// of a key are contiguous ones, and a lane's bytes of four values make the columns of the second product.
//
// Split: a CTA of four warps takes a chunk of one sequence and one key head; its warps take tiles of 16
// tokens in turn, each with its own ring of asynchronous copies (every lane copies what it will use
// itself, so a tile waits for no barrier but the warp's).  The warps join in shared memory; chunks of one
// sequence join in k_attn_join from partial sums in the workspace, in a fixed order.
#include "lowbit.cuh"
#include "internal.h"

namespace imq {
namespace {

constexpr int kWarps = 4;
constexpr int kTile = 16;      // tokens of a warp's tile
constexpr int kStages = 4;     // tiles in a warp's ring
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kPScale = 32768.f;
constexpr float kStepFloor = 1e-30f;

struct AttnArgs {
  imq_kv_cache c;
  const void* Q;
  int64_t q_batch, q_head;
  int q_bf16;
  int group;       // query heads of a key head
  int head_chunks; // blocks of up to 8 * kM query heads per key head
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  int64_t limit;   // longest sequence the call covers
  int64_t chunk;   // tokens of a split
  int splits;
  float scale;
  void* out;
  int64_t o_batch, o_head;
  int o_bf16;
  float* lse;
  int64_t lse_batch;
  float* part;     // [batch][split][query head][D]
  float2* ml;      // [batch][split][query head]: maximum (in log2 units) and sum
  int32_t* status;
};

// Bytes a lane holds of a token's key (a quarter of the vector) and of a value (an eighth), as 16-, 8- and
// 4-byte pieces.  Piece p of the lanes of a token together is a contiguous part of the vector.
template <int kBits, int kD, int kShare>
struct Pieces {
  static constexpr int kBytes = kD * kBits / 8 / kShare;
  static constexpr int n16 = kBytes / 16, n8 = kBytes % 16 / 8, n4 = kBytes % 8 / 4;
};

// Copies lane `i` of kShare lanes' pieces of the vector at src to dst + 16 * lane, laid out so that each
// piece of a warp is 32 consecutive slots.
template <typename P, int kShare>
__device__ __forceinline__ void copy_pieces(uint32_t dst, int lane, const uint8_t* src, int i, uint32_t on) {
#pragma unroll
  for (int j = 0; j < P::n16; ++j) cp_async<16>(dst + (j * 32 + lane) * 16, src + (j * kShare + i) * 16, on ? 16u : 0u);
  if (P::n8) cp_async<8>(dst + P::n16 * 512 + lane * 8, src + P::n16 * kShare * 16 + i * 8, on ? 8u : 0u);
  if (P::n4)
    cp_async<4>(dst + P::n16 * 512 + P::n8 * 256 + lane * 4, src + P::n16 * kShare * 16 + P::n8 * kShare * 8 + i * 4, on ? 4u : 0u);
}
// The lane's words of those pieces.
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
  if (P::n4) w[4 * P::n16 + 2 * P::n8] = *reinterpret_cast<const uint32_t*>(src + P::n16 * 512 + P::n8 * 256 + lane * 4);
}
// Byte of the vector at which word i of lane `l` of kShare lanes lies.
template <typename P, int kShare>
__device__ __forceinline__ int word_byte(int i, int l) {
  if (i < 4 * P::n16) return (i / 4 * kShare + l) * 16 + i % 4 * 4;
  i -= 4 * P::n16;
  int base = P::n16 * kShare * 16;
  if (i < 2 * P::n8) return base + l * 8 + i * 4;
  base += P::n8 * kShare * 8;
  return base + l * 4;
}

__device__ __forceinline__ float load_q(const AttnArgs& a, int64_t at) {
  return a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.Q)[at]) : static_cast<const float*>(a.Q)[at];
}
__device__ __forceinline__ void store_out(const AttnArgs& a, int64_t at, float v) {
  if (a.o_bf16)
    static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(a.out)[at] = v;
}

// x as two fp16 parts (hi, lo), pairs packed.
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t* hi, uint32_t* lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
  *hi = *reinterpret_cast<const uint32_t*>(&h);
  *lo = *reinterpret_cast<const uint32_t*>(&l);
}

// kM 16-row operands per product: 1 for up to 8 query heads a key head (rows g: first parts, rows g + 8:
// second parts), 2 for 9 to 16 (an operand per part).
template <int kBits, int kD, int kM>
struct Shape {
  using KP = Pieces<kBits, kD, 4>;
  using VP = Pieces<kBits, kD, 8>;
  static constexpr int kSteps = kD / 16;                       // inner steps of q * k
  static constexpr int kCols = kD / 8;                         // 8-column blocks of p * v
  static constexpr int kKeyBytes = kTile * KP::kBytes * 4;     // of a tile
  static constexpr int kTileBytes = 2 * kKeyBytes + kTile * 8; // keys, values, steps
  static constexpr int kRing = kStages * kTileBytes;           // of a warp
  static constexpr int kHeads = 8 * kM;
  static constexpr int kQBytes = kSteps * 32 * 16 * kM;        // query operands
  static constexpr int kJoin = kWarps * kHeads * (kD + 4) * 4; // the warps' sums, over the ring
  static constexpr int kSmem = kQBytes + (kWarps * kRing > kJoin ? kWarps * kRing : kJoin);
};

template <int kBits, int kD, int kM>
__global__ void __launch_bounds__(kWarps * 32) k_attn(const __grid_constant__ AttnArgs a) {
  using S = Shape<kBits, kD, kM>;
  using KP = typename S::KP;
  using VP = typename S::VP;
  extern __shared__ __align__(16) uint8_t smem[];
  uint4* const qs = reinterpret_cast<uint4*>(smem);
  uint8_t* const ring = smem + S::kQBytes;
  __shared__ float s_mul[S::kHeads];
  __shared__ float s_m[kWarps][S::kHeads], s_l[kWarps][S::kHeads];

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, split = blockIdx.x;
  const int kv = blockIdx.y / a.head_chunks, h0 = kv * a.group + (blockIdx.y % a.head_chunks) * S::kHeads;
  const int heads = min(S::kHeads, (kv + 1) * a.group - h0);
  const int q_heads = a.c.n_heads * a.group;
  const int64_t len = a.lens[b];
  const bool over = len > a.limit;
  const int64_t begin = split * a.chunk, end = over ? 0 : min(len, begin + a.chunk);
  asm volatile("griddepcontrol.launch_dependents;");

  if (begin >= end) {  // nothing here; a sequence without tokens, or one longer than the call covers, is answered
    if (over && split == 0 && threadIdx.x == 0) set_status(a.status, IMQ_ERR_BOUNDS);
    const float nan = __uint_as_float(0x7FC00000u), minus_inf = __uint_as_float(0xFF800000u);
    if (a.splits > 1) {
      if (threadIdx.x < heads)
        a.ml[((int64_t)b * a.splits + split) * q_heads + h0 + threadIdx.x] = make_float2(minus_inf, over ? nan : 0.f);
    } else {
      for (int i = threadIdx.x; i < heads * kD; i += kWarps * 32)
        store_out(a, b * a.o_batch + (h0 + i / kD) * a.o_head + i % kD, over ? nan : 0.f);
      if (a.lse && threadIdx.x < heads) a.lse[b * a.lse_batch + h0 + threadIdx.x] = over ? nan : minus_inf;
    }
    return;
  }

  // ---- the query operands, shared by the warps: each warp prepares a part of the rows' scales first
  for (int h = warp; h < S::kHeads; h += kWarps) {
    uint32_t key = 0;
    if (h < heads)
      for (int d = lane; d < kD; d += 32) key = max(key, abs_key(load_q(a, b * a.q_batch + (h0 + h) * a.q_head + d)));
    key = __reduce_max_sync(0xffffffffu, key);
    if (lane == 0) s_mul[h] = __uint_as_float(key);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < S::kSteps * 32 * kM; i += kWarps * 32) {
    // entry (step, lane): with one operand {first part 0-1, second part 0-1, first 2-3, second 2-3} of head
    // g; with two, the first (second) parts of heads g and g + 8 at entries 2 * step (+ 1)
    const int l = i & 31, gg = l >> 2, cc = l & 3, st = (i >> 5) / kM, part = (i >> 5) % kM;
    // four entries of the inner step: 8-bit codes are one word a step, 4-bit codes half a word
    const int d = kBits == 8 ? word_byte<KP, 4>(st, cc) : 2 * word_byte<KP, 4>(st / 2, cc) + 4 * (st & 1);
    uint32_t hi[kM][2], lo[kM][2];
#pragma unroll
    for (int r = 0; r < kM; ++r) {
      const int h = gg + 8 * r;
      float x[4] = {};
      if (h < heads) {
        const uint32_t key = __float_as_uint(s_mul[h]);
        // 2^e with the largest entry in [2^14, 2^15); nothing for a non-finite row, whose scores become NaN
        const int e = min(14 + 127 - (int)(key >> 23), 126);
        const float up = key_finite(key) ? __uint_as_float((uint32_t)(e + 127) << 23) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float q = load_q(a, b * a.q_batch + (h0 + h) * a.q_head + d + j);
          x[j] = up != 0.f ? q * up : 0.f;
        }
      }
      split_f16(x[0], x[1], &hi[r][0], &lo[r][0]);
      split_f16(x[2], x[3], &hi[r][1], &lo[r][1]);
    }
    if (kM == 1)
      qs[i] = make_uint4(hi[0][0], lo[0][0], hi[0][1], lo[0][1]);
    else
      qs[i] = part == 0 ? make_uint4(hi[0][0], hi[kM - 1][0], hi[0][1], hi[kM - 1][1])
                        : make_uint4(lo[0][0], lo[kM - 1][0], lo[0][1], lo[kM - 1][1]);
  }
  // the factor of a row's integer scores: scale * log2(e) / 2^e
  float mul[kM];
#pragma unroll
  for (int r = 0; r < kM; ++r) {
    const uint32_t key = __float_as_uint(s_mul[g + 8 * r]);
    const int e = min(14 + 127 - (int)(key >> 23), 126);
    mul[r] = key_finite(key) ? a.scale * kLog2e * __uint_as_float((uint32_t)(127 - e) << 23) : __uint_as_float(0x7FC00000u);
  }
  __syncthreads();

  // ---- the warp's tiles
  const int64_t first = begin + warp * kTile;
  const int n_tiles = first < end ? (int)((end - first + kWarps * kTile - 1) / (kWarps * kTile)) : 0;
  uint8_t* const mine = ring + warp * S::kRing;
  const uint32_t mine_addr = smem_addr(mine);
  const int32_t* const table = a.table + b * a.table_stride;
  bool bad = false;
  int32_t pages = 0;  // page of tile (i & ~31) + lane

  auto issue = [&](int i) {
    if (i < n_tiles) {
      if ((i & 31) == 0) {
        const int64_t t = first + (int64_t)(i + lane) * (kWarps * kTile);
        pages = t < end ? table[t / a.c.page_size] : 0;
        if (pages < 0 || pages >= a.c.n_pages) pages = -1;
      }
      const int32_t page = __shfl_sync(0xffffffffu, pages, i & 31);
      bad |= page < 0;
      const int64_t t0 = first + (int64_t)i * (kWarps * kTile);
      const int in_page = (int)(t0 % a.c.page_size), valid = page < 0 ? 0 : (int)min((int64_t)kTile, end - t0);
      const int64_t vec = kv * (int64_t)a.c.page_size + in_page, p = max(page, 0);
      constexpr int kRow = kD * kBits / 8;
      const uint8_t* kp = a.c.k + p * a.c.k_page_stride + vec * kRow;
      const uint8_t* vp = a.c.v + p * a.c.v_page_stride + vec * kRow;
      const uint32_t dst = mine_addr + (i % kStages) * S::kTileBytes;
      // tokens that are not read keep the address of the tile's first one and are zero-filled
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = 8 * j + g, on = t < valid;
        copy_pieces<KP, 4>(dst + j * (S::kKeyBytes / 2), lane, kp + (on ? t : 0) * kRow, c, on);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 8 * (j >> 1) + 2 * c + (j & 1), on = t < valid;
        copy_pieces<VP, 8>(dst + S::kKeyBytes + j * (S::kKeyBytes / 4), lane, vp + (on ? t : 0) * kRow, g, on);
      }
      if (lane < 8) {
        const int n = min(max(valid - 2 * lane, 0), 2);
        cp_async<16>(dst + 2 * S::kKeyBytes + lane * 16,
                     a.c.steps + p * a.c.steps_page_stride + (vec + (n ? 2 * lane : 0)) * 2, 8u * n);
      }
    }
    cp_async_commit();
  };

  float o[S::kCols][4] = {};
  float m[kM], l[kM], vref = kStepFloor, winv = kPScale / kStepFloor;
#pragma unroll
  for (int r = 0; r < kM; ++r) m[r] = __uint_as_float(0xFF800000u), l[r] = 0.f;

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);
  for (int i = 0; i < n_tiles; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    issue(i + kStages - 1);
    const uint8_t* tile = mine + (i % kStages) * S::kTileBytes;
    // scores: two blocks of eight tokens
    float sc[2][4] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[KP::kBytes / 4];
      read_pieces<KP>(tile + j * (S::kKeyBytes / 2), lane, w);
#pragma unroll
      for (int st = 0; st < S::kSteps; ++st) {
        uint32_t b0, b1;
        if (kBits == 8) {
          b0 = bytes_f16(w[st], 0x4140), b1 = bytes_f16(w[st], 0x4342);
        } else {
          const uint32_t x = (st & 1) ? w[st / 2] >> 8 : w[st / 2];
          b0 = nibbles_f16<false>(x), b1 = nibbles_f16<true>(x);
        }
#pragma unroll
        for (int r = 0; r < kM; ++r) {
          const uint4 q = qs[(st * kM + r) * 32 + lane];
          mma_f16(sc[j], q.x, q.y, q.z, q.w, b0, b1);
        }
      }
    }
    const float4 st0 = *reinterpret_cast<const float4*>(tile + 2 * S::kKeyBytes + c * 16);
    const float4 st1 = *reinterpret_cast<const float4*>(tile + 2 * S::kKeyBytes + 64 + c * 16);
    const float ks[4] = {st0.x, st0.z, st1.x, st1.z}, vs[4] = {st0.y, st0.w, st1.y, st1.w};
    const int64_t left = end - (first + (int64_t)i * (kWarps * kTile));
    // this lane's tokens 2c, 2c + 1, 2c + 8, 2c + 9; heads g (and g + 8)
    float p[kM][4], fix[kM];
    float vmax = fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]));
    vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 1));
    vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
    float ratio = 1.f;
    if (vmax > vref) {
      ratio = vref / vmax;
      vref = vmax;
      winv = kPScale / vmax;
    }
    bool change = false;
#pragma unroll
    for (int r = 0; r < kM; ++r) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float dot = kM == 1 ? sc[j >> 1][j & 1] + sc[j >> 1][2 + (j & 1)] : sc[j >> 1][2 * r + (j & 1)];
        p[r][j] = 8 * (j >> 1) + 2 * c + (j & 1) < left ? dot * ks[j] * mul[r] : __uint_as_float(0xFF800000u);
      }
      float top = fmaxf(fmaxf(p[r][0], p[r][1]), fmaxf(p[r][2], p[r][3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = fmaxf(top, m[r]);
      const float ref = top == __uint_as_float(0xFF800000u) ? 0.f : top;
      const float alpha = exp2f(m[r] - ref);
      m[r] = top;
      fix[r] = alpha * ratio;
      change |= fix[r] != 1.f;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[r][j] = exp2f(p[r][j] - ref);
        sum += p[r][j];
        p[r][j] *= vs[j] * winv;
      }
      l[r] = l[r] * alpha + sum;
    }
    if (__any_sync(0xffffffffu, change)) {
#pragma unroll
      for (int n = 0; n < S::kCols; ++n) {
        o[n][0] *= fix[0], o[n][1] *= fix[0];
        if (kM == 2) o[n][2] *= fix[kM - 1], o[n][3] *= fix[kM - 1];
        else o[n][2] *= fix[0], o[n][3] *= fix[0];
      }
    }
    // probabilities as operands
    uint32_t hi[kM][2], lo[kM][2];
#pragma unroll
    for (int r = 0; r < kM; ++r) {
      split_f16(p[r][0], p[r][1], &hi[r][0], &lo[r][0]);
      split_f16(p[r][2], p[r][3], &hi[r][1], &lo[r][1]);
    }
    uint32_t w[4][VP::kBytes / 4];
#pragma unroll
    for (int j = 0; j < 4; ++j) read_pieces<VP>(tile + S::kKeyBytes + j * (S::kKeyBytes / 4), lane, w[j]);
    auto product = [&](float (&acc)[4], uint32_t b0, uint32_t b1) {
      if (kM == 1) {
        mma_f16(acc, hi[0][0], lo[0][0], hi[0][1], lo[0][1], b0, b1);
      } else {
        mma_f16(acc, hi[0][0], hi[kM - 1][0], hi[0][1], hi[kM - 1][1], b0, b1);
        mma_f16(acc, lo[0][0], lo[kM - 1][0], lo[0][1], lo[kM - 1][1], b0, b1);
      }
    };
#pragma unroll
    for (int n = 0; n < VP::kBytes / 4; ++n) {
      if constexpr (kBits == 8) {
        const uint32_t x0 = __byte_perm(w[0][n], w[1][n], 0x5140), x1 = __byte_perm(w[0][n], w[1][n], 0x7362);
        const uint32_t y0 = __byte_perm(w[2][n], w[3][n], 0x5140), y1 = __byte_perm(w[2][n], w[3][n], 0x7362);
        product(o[4 * n], bytes_f16(x0, 0x4140), bytes_f16(y0, 0x4140));
        product(o[4 * n + 1], bytes_f16(x0, 0x4342), bytes_f16(y0, 0x4342));
        product(o[4 * n + 2], bytes_f16(x1, 0x4140), bytes_f16(y1, 0x4140));
        product(o[4 * n + 3], bytes_f16(x1, 0x4342), bytes_f16(y1, 0x4342));
      } else {
        // byte k of a word holds codes (0, 2), (4, 6), (1, 3), (5, 7) in its low and high half
        constexpr int kSel[4] = {0x0400, 0x0501, 0x0602, 0x0703}, kLow[4] = {0, 4, 1, 5}, kUp[4] = {2, 6, 3, 7};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = __byte_perm(w[0][n], w[1][n], kSel[k]), y = __byte_perm(w[2][n], w[3][n], kSel[k]);
          product(o[8 * n + kLow[k]], nibbles_f16<false>(x), nibbles_f16<false>(y));
          product(o[8 * n + kUp[k]], nibbles_f16<true>(x), nibbles_f16<true>(y));
        }
      }
    }
  }
  cp_async_wait<0>();

  // ---- join the warps' sums
#pragma unroll
  for (int r = 0; r < kM; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (__any_sync(0xffffffffu, bad)) l[r] = __uint_as_float(0x7FC00000u);
    if (c == 0) s_m[warp][g + 8 * r] = m[r], s_l[warp][g + 8 * r] = l[r];
  }
  if (bad && lane == 0) set_status(a.status, IMQ_ERR_BOUNDS);
  __syncthreads();  // the rings are done with: they hold the sums from here
  float* const sums = reinterpret_cast<float*>(ring);  // [warp][head][kD + 4]
  const float down = vref / kPScale;
#pragma unroll
  for (int n = 0; n < S::kCols; ++n) {
    constexpr int kCodes = 32 / kBits;  // codes of a word
    // column 2c (+ 1) of block n is code n of lane 2c's (2c + 1's) eighth of the vector
    const int d0 = word_byte<VP, 8>(n / kCodes, 2 * c) * 8 / kBits + n % kCodes;
    const int d1 = word_byte<VP, 8>(n / kCodes, 2 * c + 1) * 8 / kBits + n % kCodes;
    float* row = sums + (warp * S::kHeads + g) * (kD + 4);
    if (kM == 1) {
      row[d0] = (o[n][0] + o[n][2]) * down, row[d1] = (o[n][1] + o[n][3]) * down;
    } else {
      row[d0] = o[n][0] * down, row[d1] = o[n][1] * down;
      row += 8 * (kD + 4);
      row[d0] = o[n][2] * down, row[d1] = o[n][3] * down;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < heads * kD; i += kWarps * 32) {
    const int h = i / kD, d = i % kD;
    float top = s_m[0][h];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_m[w][h]);
    const float ref = top == __uint_as_float(0xFF800000u) ? 0.f : top;
    float num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = exp2f(s_m[w][h] - ref);
      num += f * sums[(w * S::kHeads + h) * (kD + 4) + d];
      den += f * s_l[w][h];
    }
    if (a.splits > 1) {
      const int64_t at = ((int64_t)b * a.splits + split) * q_heads + h0 + h;
      a.part[at * kD + d] = num;
      if (d == 0) a.ml[at] = make_float2(top, den);
    } else {
      store_out(a, b * a.o_batch + (h0 + h) * a.o_head + d, num / den);
      if (d == 0 && a.lse) a.lse[b * a.lse_batch + h0 + h] = kLn2 * (ref + log2f(den));
    }
  }
}

// Joins the chunks of one sequence and query head: a thread per output entry.
__global__ void k_attn_join(const __grid_constant__ AttnArgs a, int D) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x, q_heads = gridDim.x;
  const int64_t at = (int64_t)b * a.splits * q_heads + h;
  float top = __uint_as_float(0xFF800000u);
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.ml[at + (int64_t)s * q_heads].x);
  const float ref = top == __uint_as_float(0xFF800000u) ? 0.f : top;
  float num = 0.f, den = 0.f;
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = a.ml[at + (int64_t)s * q_heads];
    if (ml.y == 0.f) continue;  // an empty chunk wrote no sums
    const float f = exp2f(ml.x - ref);
    num += f * a.part[(at + (int64_t)s * q_heads) * D + d];
    den += f * ml.y;
  }
  // den = 0: no token at all
  store_out(a, b * a.o_batch + h * a.o_head + d, den == 0.f ? 0.f : num / den);
  if (d == 0 && a.lse) a.lse[b * a.lse_batch + h] = den == 0.f ? __uint_as_float(0xFF800000u) : kLn2 * (ref + log2f(den));
}

// Tokens of a split: chunks that fill the SMs once, none below 128 tokens.
void plan_splits(int num_sms, int64_t batch, int64_t rows, int64_t limit, int64_t* chunk, int* splits) {
  const int64_t ctas = batch * rows, want = 3ll * num_sms;
  int64_t n = ctas > 0 ? want / ctas : 1;
  if (n < 1) n = 1;
  int64_t c = (limit + n - 1) / n;
  c = (c + kWarps * kTile - 1) / (kWarps * kTile) * (kWarps * kTile);
  if (c < 128) c = 128;
  *chunk = c;
  *splits = (int)(limit > 0 ? (limit + c - 1) / c : 1);
}

int heads_of_cta(int group) { return group > 8 ? 16 : 8; }

template <int kBits, int kD, int kM>
imq_status launch_shape(const AttnArgs& a, dim3 grid, cudaStream_t st) {
  constexpr int kSmem = Shape<kBits, kD, kM>::kSmem;
  const void* fn = reinterpret_cast<const void*>(&k_attn<kBits, kD, kM>);
  if (ensure_smem(fn, kSmem) != cudaSuccess) return IMQ_ERR_CUDA;
  k_attn<kBits, kD, kM><<<grid, kWarps * 32, kSmem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA;
}

template <int kBits, int kM>
imq_status launch_dim(const AttnArgs& a, dim3 grid, cudaStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch_shape<kBits, 64, kM>(a, grid, st);
    case 128: return launch_shape<kBits, 128, kM>(a, grid, st);
    case 192: return launch_shape<kBits, 192, kM>(a, grid, st);
    default: return launch_shape<kBits, 256, kM>(a, grid, st);
  }
}

imq_status check_shape(const imq_kv_cache* c, int64_t batch, int32_t q_heads, int64_t max_len) {
  imq_status s = check_cache(c);
  if (s != IMQ_OK) return s;
  if (batch < 0 || q_heads < 1 || max_len < 0 || q_heads % c->n_heads != 0) return IMQ_ERR_ARG;
  const int64_t group = q_heads / c->n_heads, per = heads_of_cta((int)group);
  if (batch > 65535 || (group + per - 1) / per * c->n_heads > 65535 || q_heads > 65535 || max_len > INT32_MAX)
    return IMQ_ERR_UNSUPPORTED;
  return IMQ_OK;
}
}  // namespace

imq_status paged_attention_workspace(const imq_kv_cache* c, int64_t batch, int32_t q_heads, int64_t max_len, size_t* bytes) {
  if (!bytes) return IMQ_ERR_ARG;
  imq_status s = check_shape(c, batch, q_heads, max_len);
  if (s != IMQ_OK) return s;
  DeviceState* ds;
  s = device_state(&ds);
  if (s != IMQ_OK) return s;
  const int group = q_heads / c->n_heads, per = heads_of_cta(group);
  int64_t chunk;
  int splits;
  plan_splits(ds->num_sms, batch, (int64_t)((group + per - 1) / per) * c->n_heads, max_len, &chunk, &splits);
  *bytes = splits > 1 ? (size_t)batch * splits * q_heads * ((size_t)c->head_dim * 4 + 8) : 0;
  return IMQ_OK;
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
  if ((reinterpret_cast<uintptr_t>(Q) & (qt == IMQ_F32 ? 3 : 1)) || (reinterpret_cast<uintptr_t>(out) & (ot == IMQ_F32 ? 3 : 1)) ||
      (reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(workspace) & 15))
    return IMQ_ERR_ARG;
  DeviceState* ds;
  s = device_state(&ds);
  if (s != IMQ_OK) return s;
  AttnArgs a;
  a.c = *c;
  a.Q = Q, a.q_batch = q_batch, a.q_head = q_head, a.q_bf16 = qt == IMQ_BF16;
  a.group = q_heads / c->n_heads;
  const int per = heads_of_cta(a.group);
  a.head_chunks = (a.group + per - 1) / per;
  a.table = table, a.table_stride = table_stride, a.lens = lens, a.limit = max_len;
  plan_splits(ds->num_sms, batch, (int64_t)a.head_chunks * c->n_heads, max_len, &a.chunk, &a.splits);
  a.scale = scale;
  a.out = out, a.o_batch = o_batch, a.o_head = o_head, a.o_bf16 = ot == IMQ_BF16;
  a.lse = lse, a.lse_batch = lse_batch;
  a.part = nullptr, a.ml = nullptr;
  a.status = ds->status;
  if (a.splits > 1) {
    const size_t rows = (size_t)batch * a.splits * q_heads;
    if (!workspace || workspace_bytes < rows * ((size_t)c->head_dim * 4 + 8)) return IMQ_ERR_BUFFER;
    a.part = static_cast<float*>(workspace);
    a.ml = reinterpret_cast<float2*>(a.part + rows * c->head_dim);
  }
  const dim3 grid((unsigned)a.splits, (unsigned)(a.head_chunks * c->n_heads), (unsigned)batch);
  if (c->bits == 4)
    s = per == 8 ? launch_dim<4, 1>(a, grid, st) : launch_dim<4, 2>(a, grid, st);
  else
    s = per == 8 ? launch_dim<8, 1>(a, grid, st) : launch_dim<8, 2>(a, grid, st);
  if (s != IMQ_OK || a.splits == 1) return s;
  // launched before k_attn has finished; it waits for it on the device
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)q_heads, (unsigned)batch);
  cfg.blockDim = dim3((unsigned)c->head_dim);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attn_join, a, (int)c->head_dim) == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA;
}

}  // namespace imq
