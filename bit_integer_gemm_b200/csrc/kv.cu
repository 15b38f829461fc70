// kv.cu -- the paged low-bit cache of keys and values: quantising vectors as they are written, and reading
// them back (sm_100a).
//
// A vector (one head's key or value of one token) is one quantisation group.  D / 8 lanes take a vector, 8
// entries each: the largest |x| by shuffles, the codes packed to one word (4 bits) or two (8 bits) a lane.
// A lane group does a token's key and value of a head together, so their two steps are one 8-byte store.
// Bound: memory; every entry is read and written once.  65536 tokens of 8 heads of 128, bf16 and 8 bits: written in 69.0 us
// (5.9 TB/s, keys and values two tensors), read back in 64.9 (6.3 TB/s).  Writing has the instructions of the quantiser
// besides, seven an entry: 8191 tokens at 4 bits take 12.4 us (3.4 TB/s), issue slots 62 % busy in 42 % of the warps.
#include <type_traits>

#include "lowbit.cuh"
#include "internal.h"

namespace imq {
namespace {

struct VecArgs {
  imq_kv_cache c;
  void* K;  // only read by the write kernel
  void* V;
  int64_t n, k_tok, k_head, v_tok, v_head;
  const int64_t* slots;
  int aligned;
  int head_shift, page_shift;  // heads = 2^head_shift, page_size = 2^page_shift, or -1
  int32_t* status;
  uint32_t one;  // kOneF16
  int64_t slots_of_cache;
  uint32_t k_stride16, v_stride16, s_stride16;  // of pages, in 16 bytes
  uint32_t vec16;                               // of a vector, in 16 bytes
};

// Tokens a lane group takes, their loads under way together: four where that still fills the SMs twice (65536 tokens of
// 8 heads at 8 bits: 69.0 us written and 64.9 read; with one 79.8 and 75.9), one below (32 tokens of 32 heads: 2.0 us
// written, 1.8 read; with four 3.3 and 2.7).
constexpr int kManyTokens = 4;

// Where a token's vectors of a head lie: in the keys and the values, and their page in the steps, in 16 bytes (every
// offset of a legal cache fits); and which vector of its page it is.
struct Place {
  uint32_t k, v, s_page, vec;
};
__device__ __forceinline__ float2* steps_at(const imq_kv_cache& c, const Place& at) {
  return reinterpret_cast<float2*>(c.steps + (uint64_t)at.s_page * 4) + at.vec;
}
// False for a token that is skipped.  A legal cache has fewer than 2^32 slots.
__device__ __forceinline__ bool locate(const VecArgs& a, int64_t slot, int head, bool report, Place* at) {
  if (slot < 0) return false;
  if (slot >= a.slots_of_cache) {
    if (report) set_status(a.status, IMQ_ERR_BOUNDS);
    return false;
  }
  const uint32_t x = (uint32_t)slot, size = a.c.page_size;
  const uint32_t p = a.page_shift >= 0 ? x >> a.page_shift : x / size, vec = head * size + (x - p * size);
  *at = {p * a.k_stride16 + vec * a.vec16, p * a.v_stride16 + vec * a.vec16, p * a.s_stride16, vec};
  return true;
}

// Eight entries as they lie in memory.
template <typename T>
struct Raw {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];

  template <bool kVec>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kVec) {
#pragma unroll
      for (int q = 0; q < kWords / 4; ++q) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[q];
        w[4 * q] = v.x, w[4 * q + 1] = v.y, w[4 * q + 2] = v.z, w[4 * q + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(p[e]);
        else if (e % 2 == 0) w[e / 2] = __bfloat16_as_ushort(p[e]) | (uint32_t)__bfloat16_as_ushort(p[e + 1]) << 16;
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float entry(int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float(e % 2 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
  }
  // abs_key of the largest entry; two bf16 entries are compared at a time
  __device__ __forceinline__ uint32_t key() const {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7FFFFFFFu);
      return m;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
      return max(m << 16, m & 0xFFFF0000u);
    }
  }
};
// 16 bytes.
template <bool kVec>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[8]) {
  if constexpr (kVec) {
    store8(p, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = from_f32<__nv_bfloat16>(x[e]);
  }
}
template <bool kVec>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[4]) {
  if constexpr (kVec) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = x[e];
  }
}

// kLanes: lanes of a vector's group (a power of two >= D / 8; the lanes at and above D / 8 hold zeros).
// bf16: four CTAs an SM, at the price of a few spilled registers (69.0 us for the 65536 tokens; three without: 72.9).
template <typename T, int kBits, int kLanes, int kTokens>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) k_kv_write(const __grid_constant__ VecArgs a) {
  const imq_kv_cache& c = a.c;
  const int i = threadIdx.x % kLanes;
  const uint32_t unit = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  const uint32_t set = a.head_shift >= 0 ? unit >> a.head_shift : unit / (uint32_t)c.n_heads;
  const int64_t tok0 = (int64_t)set * kTokens;
  const int head = unit - set * (uint32_t)c.n_heads;
  const bool lane = 8 * i < c.head_dim;
  Raw<T> k[kTokens], v[kTokens];
  const T* const kp0 = static_cast<const T*>(a.K) + tok0 * a.k_tok + head * a.k_head + 8 * i;
  const T* const vp0 = static_cast<const T*>(a.V) + tok0 * a.v_tok + head * a.v_head + 8 * i;
  auto load = [&](auto vec) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      k[j].clear(), v[j].clear();
      if (lane && tok0 + j < a.n) k[j].template load<vec>(kp0 + j * a.k_tok), v[j].template load<vec>(vp0 + j * a.v_tok);
    }
  };
  if (a.aligned) load(std::true_type{});
  else load(std::false_type{});
  int64_t slot[kTokens];
#pragma unroll
  for (int j = 0; j < kTokens; ++j) slot[j] = tok0 + j < a.n ? a.slots[tok0 + j] : -1;
  uint32_t key[2][kTokens];
#pragma unroll
  for (int j = 0; j < kTokens; ++j) key[0][j] = k[j].key(), key[1][j] = v[j].key();
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1)
#pragma unroll
    for (int q = 0; q < 2 * kTokens; ++q)
      key[q / kTokens][q % kTokens] = max(key[q / kTokens][q % kTokens], __shfl_xor_sync(0xffffffffu, key[q / kTokens][q % kTokens], o));
  float s[2][kTokens], step[2][kTokens];
  constexpr float kBeta = (float)((1 << (kBits - 1)) - 1);
  if constexpr (kTokens == 4) {
#pragma unroll
    for (int q = 0; q < 2; ++q) four_scales(key[q], kBeta, s[q], step[q]);
  } else {
#pragma unroll
    for (int q = 0; q < 2; ++q) group_scale(key[q][0], kBeta, &s[q][0], &step[q][0]);
  }
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    Place at;
    if (!locate(a, slot[j], head, i == 0, &at) || !lane) continue;
    uint8_t* const kp = c.k + (uint64_t)at.k * 16 + kBits * i;  // eight codes are kBits bytes
    uint8_t* const vp = c.v + (uint64_t)at.v * 16 + kBits * i;
    float x[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const Raw<T>& r = q ? v[j] : k[j];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = r.entry(e);
      if constexpr (kBits == 4)
        *reinterpret_cast<uint32_t*>(q ? vp : kp) = pack4(x, s[q][j]);
      else
        *reinterpret_cast<uint2*>(q ? vp : kp) = make_uint2(pack8(x[0], x[1], x[2], x[3], s[q][j]), pack8(x[4], x[5], x[6], x[7], s[q][j]));
    }
    if (i == 0) {
      *steps_at(c, at) = make_float2(step[0][j], step[1][j]);
      if (!key_finite(key[0][j]) || !key_finite(key[1][j])) set_status(a.status, IMQ_ERR_NONFINITE);
    }
  }
}

// A lane makes 16 bytes of a vector: 8 entries of bf16, 4 of fp32 (so that a warp's stores are one piece).  kLanes: a power
// of two that covers a vector.
template <typename T, int kBits, int kLanes, int kTokens>
__global__ void __launch_bounds__(256) k_kv_read(const __grid_constant__ VecArgs a) {
  constexpr int kMine = 16 / sizeof(T), kWords = kMine * kBits > 32 ? 2 : 1;
  const imq_kv_cache& c = a.c;
  const int i = threadIdx.x % kLanes;
  const uint32_t unit = blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  const uint32_t set = a.head_shift >= 0 ? unit >> a.head_shift : unit / (uint32_t)c.n_heads;
  const int64_t tok0 = (int64_t)set * kTokens;
  const int head = unit - set * (uint32_t)c.n_heads;
  // the word (or two) of this lane's codes; at 4 bits and fp32 two lanes share a word
  const int from = i * kMine * kBits / 32 * 4;
  uint32_t kw[kTokens][kWords], vw[kTokens][kWords];
  float2 step[kTokens];
  bool on[kTokens];
  int64_t slot[kTokens];
#pragma unroll
  for (int j = 0; j < kTokens; ++j) slot[j] = tok0 + j < a.n ? a.slots[tok0 + j] : -1;
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    Place at;
    on[j] = locate(a, slot[j], head, i == 0, &at) && kMine * i < c.head_dim;
    if (!on[j]) continue;
    const uint8_t* const kp = c.k + (uint64_t)at.k * 16 + from;
    const uint8_t* const vp = c.v + (uint64_t)at.v * 16 + from;
    step[j] = *steps_at(c, at);
    if constexpr (kWords == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(kp), y = *reinterpret_cast<const uint2*>(vp);
      kw[j][0] = x.x, kw[j][1] = x.y, vw[j][0] = y.x, vw[j][1] = y.y;
    } else {
      kw[j][0] = *reinterpret_cast<const uint32_t*>(kp), vw[j][0] = *reinterpret_cast<const uint32_t*>(vp);
    }
  }
  auto values = [&](const uint32_t(&w)[kWords], float s, float(&x)[kMine]) {
#pragma unroll
    for (int q = 0; q < kMine / 2; ++q) {
      float2 v;
      if constexpr (kBits == 8) v = byte_pair(w[q / 2], q % 2, a.one);
      else if constexpr (kMine == 8) v = nibble_pair(w[0], q, a.one);
      else v = nibble_pair(i & 1 ? w[0] >> 8 : w[0], q, a.one);  // codes 4-7 lie 8 bits above codes 0-3
      x[2 * q] = __fmul_rn(v.x, s), x[2 * q + 1] = __fmul_rn(v.y, s);
    }
  };
  auto write = [&](auto vec) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      if (!on[j]) continue;
      float x[kMine];
      if (a.K) {
        values(kw[j], step[j].x, x);
        store_vec<vec>(static_cast<T*>(a.K) + (tok0 + j) * a.k_tok + head * a.k_head + kMine * i, x);
      }
      if (a.V) {
        values(vw[j], step[j].y, x);
        store_vec<vec>(static_cast<T*>(a.V) + (tok0 + j) * a.v_tok + head * a.v_head + kMine * i, x);
      }
    }
  };
  if (a.aligned) write(std::true_type{});
  else write(std::false_type{});
}

int log2_or(int32_t n) { return (n & (n - 1)) == 0 ? __builtin_ctz(n) : -1; }

template <typename T, int kBits, int kTokens>
void run_tokens(bool write, const VecArgs& a, int lanes, cudaStream_t st) {
  const int64_t units = (a.n + kTokens - 1) / kTokens * a.c.n_heads;
  const unsigned ctas = (unsigned)((units + 256 / lanes - 1) / (256 / lanes));
  if (write) {
    if (lanes == 8) k_kv_write<T, kBits, 8, kTokens><<<ctas, 256, 0, st>>>(a);
    if (lanes == 16) k_kv_write<T, kBits, 16, kTokens><<<ctas, 256, 0, st>>>(a);
    if (lanes == 32) k_kv_write<T, kBits, 32, kTokens><<<ctas, 256, 0, st>>>(a);
  } else {
    if (lanes == 8) k_kv_read<T, kBits, 8, kTokens><<<ctas, 256, 0, st>>>(a);
    if (lanes == 16) k_kv_read<T, kBits, 16, kTokens><<<ctas, 256, 0, st>>>(a);
    if (lanes == 32) k_kv_read<T, kBits, 32, kTokens><<<ctas, 256, 0, st>>>(a);
    if (lanes == 64) k_kv_read<T, kBits, 64, kTokens><<<ctas, 256, 0, st>>>(a);
  }
}

template <typename T, int kBits>
void run(bool write, const VecArgs& a, int num_sms, cudaStream_t st) {
  const int mine = write ? 8 : 16 / (int)sizeof(T), need = a.c.head_dim / mine;
  const int lanes = need <= 8 ? 8 : need <= 16 ? 16 : need <= 32 ? 32 : 64;
  if (a.n * a.c.n_heads * lanes >= (int64_t)kManyTokens * 2 * 256 * num_sms) run_tokens<T, kBits, kManyTokens>(write, a, lanes, st);
  else run_tokens<T, kBits, 1>(write, a, lanes, st);
}

imq_status launch(bool write, const imq_kv_cache* cache, void* K, int64_t k_tok, int64_t k_head, void* V, int64_t v_tok,
                  int64_t v_head, imq_dtype t, int64_t n, const int64_t* slots, cudaStream_t st) {
  imq_status s = check_cache(cache);
  if (s != IMQ_OK) return s;
  if ((t != IMQ_F32 && t != IMQ_BF16) || n < 0) return IMQ_ERR_ARG;
  if (k_tok < 0 || k_head < 0 || v_tok < 0 || v_head < 0) return IMQ_ERR_ARG;
  if (n == 0) return IMQ_OK;
  const int size = t == IMQ_F32 ? 4 : 2;
  const uintptr_t kp = reinterpret_cast<uintptr_t>(K), vp = reinterpret_cast<uintptr_t>(V);
  if (!slots || (write && (!K || !V)) || (!K && !V) || ((kp | vp) & (size - 1)) || (reinterpret_cast<uintptr_t>(slots) & 7))
    return IMQ_ERR_ARG;
  if (n > INT32_MAX / cache->n_heads) return IMQ_ERR_UNSUPPORTED;
  if (!write && ((K && !vectors_apart(n, k_tok, cache->n_heads, k_head, cache->head_dim)) ||
                 (V && !vectors_apart(n, v_tok, cache->n_heads, v_head, cache->head_dim))))
    return IMQ_ERR_ARG;
  DeviceState* ds;
  s = device_state(&ds);
  if (s != IMQ_OK) return s;
  const int64_t strides = ((K ? k_tok | k_head : 0) | (V ? v_tok | v_head : 0)) * size;
  VecArgs a{*cache, K, V, n, k_tok, k_head, v_tok, v_head, slots, ((kp | vp | (uintptr_t)strides) & 15) == 0,
            log2_or(cache->n_heads), log2_or(cache->page_size), ds->status, kOneF16,
            cache->n_pages * cache->page_size, (uint32_t)(cache->k_page_stride / 16), (uint32_t)(cache->v_page_stride / 16),
            (uint32_t)(cache->steps_page_stride / 4), (uint32_t)(cache->head_dim * cache->bits / 128)};
  if (t == IMQ_F32) {
    if (cache->bits == 4) run<float, 4>(write, a, ds->num_sms, st);
    else run<float, 8>(write, a, ds->num_sms, st);
  } else {
    if (cache->bits == 4) run<__nv_bfloat16, 4>(write, a, ds->num_sms, st);
    else run<__nv_bfloat16, 8>(write, a, ds->num_sms, st);
  }
  return cudaGetLastError() == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA;
}
}  // namespace

bool vectors_apart(int64_t n, int64_t step, int64_t heads, int64_t head_step, int64_t dim) {
  if (n <= 1 || heads <= 1) return (n <= 1 || step >= dim) && (heads <= 1 || head_step >= dim);
  if (step < dim || head_step < dim) return false;
  // one axis within the other's step: every layout of a tensor's axes
  if ((step - dim) / head_step >= heads - 1 || (head_step - dim) / step >= n - 1) return true;
  // else two vectors d heads apart are nearest where their tokens' distance is d * head_step, rounded either way
  for (int64_t d = 1; d < heads; ++d) {
    const int64_t from = head_step > INT64_MAX / d ? INT64_MAX : d * head_step, i = from / step, rest = from % step;
    if (i < n && rest < dim) return false;
    if (i + 1 < n && step - rest < dim) return false;
  }
  return true;
}

imq_status check_cache(const imq_kv_cache* c) {
  if (!c) return IMQ_ERR_ARG;
  if (c->bits != 4 && c->bits != 8) return IMQ_ERR_ARG;
  if (c->n_pages < 0 || c->n_heads < 1 || c->page_size < 1 || c->head_dim < 1) return IMQ_ERR_ARG;
  if (c->head_dim % 64 != 0 || c->head_dim > 256 || c->page_size % 16 != 0 || c->page_size > 65536 || c->n_heads > 65535 ||
      c->n_pages > INT32_MAX)
    return IMQ_ERR_UNSUPPORTED;
  const int64_t vectors = (int64_t)c->n_heads * c->page_size, bytes = vectors * (c->head_dim * c->bits / 8);
  if (c->k_page_stride < bytes || c->v_page_stride < bytes || c->steps_page_stride < 2 * vectors) return IMQ_ERR_ARG;
  if (c->k_page_stride % 16 || c->v_page_stride % 16 || c->steps_page_stride % 4) return IMQ_ERR_ARG;
  // offsets into each of the three are 32-bit numbers of 16 bytes in places
  const int64_t most = ((int64_t)1 << 36) - 16, pages = c->n_pages > 0 ? c->n_pages : 1;
  if (c->k_page_stride > most / pages || c->v_page_stride > most / pages || c->steps_page_stride > most / 4 / pages) return IMQ_ERR_UNSUPPORTED;
  if (c->n_pages > 0 && (!c->k || !c->v || !c->steps)) return IMQ_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v) | reinterpret_cast<uintptr_t>(c->steps)) & 15)
    return IMQ_ERR_ARG;
  return IMQ_OK;
}

imq_status launch_kv_write(const imq_kv_cache* c, const void* K, int64_t k_tok, int64_t k_head, const void* V, int64_t v_tok,
                           int64_t v_head, imq_dtype t, int64_t n, const int64_t* slots, cudaStream_t st) {
  return launch(true, c, const_cast<void*>(K), k_tok, k_head, const_cast<void*>(V), v_tok, v_head, t, n, slots, st);
}
imq_status launch_kv_read(const imq_kv_cache* c, const int64_t* slots, int64_t n, void* K, int64_t k_tok, int64_t k_head,
                          void* V, int64_t v_tok, int64_t v_head, imq_dtype t, cudaStream_t st) {
  return launch(false, c, K, k_tok, k_head, V, v_tok, v_head, t, n, slots, st);
}

}  // namespace imq
