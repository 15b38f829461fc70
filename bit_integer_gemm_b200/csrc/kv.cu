// kv.cu -- the paged low-bit cache of keys and values: quantising vectors as they are written, and reading
// them back (sm_100a).
//
// A vector (one head's key or value of one token) is one quantisation group.  D / 8 lanes take a vector, 8
// entries each: the largest |x| by shuffles, the codes packed to one word (4 bits) or two (8 bits) a lane.
// A lane group does a token's key and value of a head together, so their two steps are one 8-byte store.
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
  int32_t* status;
};

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, bool vec, float (&x)[8]) {
  if (vec) {
    load8(p, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = to_f32(p[e]);
  }
}
template <typename T>
__device__ __forceinline__ void store_vec(T* p, bool vec, const float (&x)[8]) {
  if (vec) {
    store8(p, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = from_f32<T>(x[e]);
  }
}

// kLanes: lanes of a vector's group (a power of two >= D / 8; the lanes at and above D / 8 hold zeros).
template <typename T, int kBits, int kLanes>
__global__ void __launch_bounds__(256) k_kv_write(VecArgs a) {
  constexpr int kBytes = kBits;  // bytes of 8 codes
  const imq_kv_cache& c = a.c;
  const int i = threadIdx.x % kLanes;
  const int64_t unit = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  const int64_t tok = unit / c.n_heads;
  const int head = (int)(unit - tok * c.n_heads);
  const int64_t slot = tok < a.n ? a.slots[tok] : -1;
  const bool inside = slot >= 0 && slot < c.n_pages * c.page_size;
  if (slot >= 0 && !inside && i == 0) set_status(a.status, IMQ_ERR_BOUNDS);
  const bool lane = inside && 8 * i < c.head_dim;
  float k[8] = {}, v[8] = {};
  if (lane) {
    load_vec(static_cast<const T*>(a.K) + tok * a.k_tok + head * a.k_head + 8 * i, a.aligned, k);
    load_vec(static_cast<const T*>(a.V) + tok * a.v_tok + head * a.v_head + 8 * i, a.aligned, v);
  }
  uint32_t kk = 0, vk = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) kk = max(kk, abs_key(k[e])), vk = max(vk, abs_key(v[e]));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    kk = max(kk, __shfl_xor_sync(0xffffffffu, kk, o));
    vk = max(vk, __shfl_xor_sync(0xffffffffu, vk, o));
  }
  if (!lane) return;
  constexpr float kBeta = (float)((1 << (kBits - 1)) - 1);
  constexpr uint32_t kBias = 1u << (kBits - 1);
  float ks, vs, kd, vd;
  group_scale(kk, kBeta, &ks, &kd);
  group_scale(vk, kBeta, &vs, &vd);
  uint32_t ku[8], vu[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) ku[e] = code_of(k[e], ks, kBias), vu[e] = code_of(v[e], vs, kBias);
  const int64_t page = slot / c.page_size, at = head * (int64_t)c.page_size + (slot - page * c.page_size);
  uint8_t* kp = c.k + page * c.k_page_stride + at * (c.head_dim * kBits / 8) + kBytes * i;
  uint8_t* vp = c.v + page * c.v_page_stride + at * (c.head_dim * kBits / 8) + kBytes * i;
  if constexpr (kBits == 4) {
    *reinterpret_cast<uint32_t*>(kp) = pack_nibbles(ku);
    *reinterpret_cast<uint32_t*>(vp) = pack_nibbles(vu);
  } else {
    *reinterpret_cast<uint2*>(kp) = make_uint2(ku[0] | ku[1] << 8 | ku[2] << 16 | ku[3] << 24,
                                               ku[4] | ku[5] << 8 | ku[6] << 16 | ku[7] << 24);
    *reinterpret_cast<uint2*>(vp) = make_uint2(vu[0] | vu[1] << 8 | vu[2] << 16 | vu[3] << 24,
                                               vu[4] | vu[5] << 8 | vu[6] << 16 | vu[7] << 24);
  }
  if (i == 0) {
    *reinterpret_cast<float2*>(c.steps + page * c.steps_page_stride + at * 2) = make_float2(kd, vd);
    if (!key_finite(kk) || !key_finite(vk)) set_status(a.status, IMQ_ERR_NONFINITE);
  }
}

template <typename T, int kBits, int kLanes>
__global__ void __launch_bounds__(256) k_kv_read(VecArgs a) {
  constexpr int kBytes = kBits;
  const imq_kv_cache& c = a.c;
  const int i = threadIdx.x % kLanes;
  const int64_t unit = (int64_t)blockIdx.x * (256 / kLanes) + threadIdx.x / kLanes;
  const int64_t tok = unit / c.n_heads;
  const int head = (int)(unit - tok * c.n_heads);
  const int64_t slot = tok < a.n ? a.slots[tok] : -1;
  const bool inside = slot >= 0 && slot < c.n_pages * c.page_size;
  if (slot >= 0 && !inside && i == 0) set_status(a.status, IMQ_ERR_BOUNDS);
  if (!inside || 8 * i >= c.head_dim) return;
  const int64_t page = slot / c.page_size, at = head * (int64_t)c.page_size + (slot - page * c.page_size);
  const uint8_t* kp = c.k + page * c.k_page_stride + at * (c.head_dim * kBits / 8) + kBytes * i;
  const uint8_t* vp = c.v + page * c.v_page_stride + at * (c.head_dim * kBits / 8) + kBytes * i;
  const float2 step = *reinterpret_cast<const float2*>(c.steps + page * c.steps_page_stride + at * 2);
  float k[8], v[8];
  if constexpr (kBits == 4) {
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(kp), vw = *reinterpret_cast<const uint32_t*>(vp);
#pragma unroll
    for (int e = 0; e < 8; ++e) k[e] = __fmul_rn(nibble_value(kw, e), step.x), v[e] = __fmul_rn(nibble_value(vw, e), step.y);
  } else {
    const uint2 kw = *reinterpret_cast<const uint2*>(kp), vw = *reinterpret_cast<const uint2*>(vp);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t ku = ((e < 4 ? kw.x : kw.y) >> (8 * (e & 3))) & 255u, vu = ((e < 4 ? vw.x : vw.y) >> (8 * (e & 3))) & 255u;
      k[e] = __fmul_rn((float)ku - 128.f, step.x), v[e] = __fmul_rn((float)vu - 128.f, step.y);
    }
  }
  if (a.K) store_vec(static_cast<T*>(a.K) + tok * a.k_tok + head * a.k_head + 8 * i, a.aligned, k);
  if (a.V) store_vec(static_cast<T*>(a.V) + tok * a.v_tok + head * a.v_head + 8 * i, a.aligned, v);
}

template <typename T, int kBits>
void run(bool write, const VecArgs& a, cudaStream_t st) {
  const int lanes = a.c.head_dim <= 64 ? 8 : a.c.head_dim <= 128 ? 16 : 32;
  const unsigned ctas = (unsigned)((a.n * a.c.n_heads + 256 / lanes - 1) / (256 / lanes));
  if (write) {
    if (lanes == 8) k_kv_write<T, kBits, 8><<<ctas, 256, 0, st>>>(a);
    if (lanes == 16) k_kv_write<T, kBits, 16><<<ctas, 256, 0, st>>>(a);
    if (lanes == 32) k_kv_write<T, kBits, 32><<<ctas, 256, 0, st>>>(a);
  } else {
    if (lanes == 8) k_kv_read<T, kBits, 8><<<ctas, 256, 0, st>>>(a);
    if (lanes == 16) k_kv_read<T, kBits, 16><<<ctas, 256, 0, st>>>(a);
    if (lanes == 32) k_kv_read<T, kBits, 32><<<ctas, 256, 0, st>>>(a);
  }
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
  if (n > (int64_t)INT32_MAX * 8 / cache->n_heads) return IMQ_ERR_UNSUPPORTED;
  DeviceState* ds;
  s = device_state(&ds);
  if (s != IMQ_OK) return s;
  const int64_t strides = ((K ? k_tok | k_head : 0) | (V ? v_tok | v_head : 0)) * size;
  VecArgs a{*cache, K, V, n, k_tok, k_head, v_tok, v_head, slots, ((kp | vp | (uintptr_t)strides) & 15) == 0, ds->status};
  if (t == IMQ_F32) {
    if (cache->bits == 4) run<float, 4>(write, a, st);
    else run<float, 8>(write, a, st);
  } else {
    if (cache->bits == 4) run<__nv_bfloat16, 4>(write, a, st);
    else run<__nv_bfloat16, 8>(write, a, st);
  }
  return cudaGetLastError() == cudaSuccess ? IMQ_OK : IMQ_ERR_CUDA;
}
}  // namespace

imq_status check_cache(const imq_kv_cache* c) {
  if (!c) return IMQ_ERR_ARG;
  if (c->bits != 4 && c->bits != 8) return IMQ_ERR_ARG;
  if (c->n_pages < 0 || c->n_heads < 1 || c->page_size < 1 || c->head_dim < 1) return IMQ_ERR_ARG;
  if (c->head_dim % 64 != 0 || c->head_dim > 256 || c->page_size % 16 != 0 || c->page_size > 65536 || c->n_heads > 65535 ||
      c->n_pages > INT32_MAX || c->k_page_stride > UINT32_MAX || c->v_page_stride > UINT32_MAX || c->steps_page_stride > UINT32_MAX)
    return IMQ_ERR_UNSUPPORTED;
  const int64_t vectors = (int64_t)c->n_heads * c->page_size, bytes = vectors * (c->head_dim * c->bits / 8);
  if (c->k_page_stride < bytes || c->v_page_stride < bytes || c->steps_page_stride < 2 * vectors) return IMQ_ERR_ARG;
  if (c->k_page_stride % 16 || c->v_page_stride % 16 || c->steps_page_stride % 4) return IMQ_ERR_ARG;
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
