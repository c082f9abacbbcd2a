// kv_cache.hip -- writing keys and values into an NVFP4 cache and reading
// them back (gfx950).
//
// Per group of 16 values of a head the encode is that of nvfp4_quantize
// (nvfp4_device.h, encode_half_group): scale = e4m3(amax/6 * 2688/g), codes =
// e2m1(x * (2688/g) / scale), bit for bit the same; the read is nvfp4_dequantize's
// T(e2m1 * (e4m3 * g/2688)).  Both move bytes only: 2 (2 + 9/16) per value
// of a 16-bit type each way, keys and values.
//
// One lane per half group (8 values), lane pairs per group as in codec.hip.
// blockIdx.y selects keys or values and the head; along x run the half groups
// of consecutive tokens of that head, so that for tokens of one page both the
// cache side (64 bytes of codes a token at dim 128, contiguous over tokens)
// and each token's values (256 contiguous bytes) are whole lines.
#include "kv_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// 8 consecutive values of type DT at element offset `e` as floats; VEC: 16-byte aligned.
template <int DT, bool VEC>
__device__ __forceinline__ void load_values(const void* base, int64_t e, float (&v)[8]) {
  if constexpr (VEC) {
    load8<DT>(base, e >> 3, v);
  } else {
    const typename Elem<DT>::T* p = reinterpret_cast<const typename Elem<DT>::T*>(base) + e;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32<DT>(p[i]);
  }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(KvCache c, const void* __restrict__ k, const void* __restrict__ v, int64_t k_token,
                int64_t k_head, int64_t v_token, int64_t v_head, const int64_t* __restrict__ slots,
                int halves, KvDiv per_token) {
  const bool values = blockIdx.y >= (unsigned)c.heads;
  const int head = values ? blockIdx.y - c.heads : blockIdx.y;
  const void* x = values ? v : k;
  const int64_t xt = values ? v_token : k_token, xh = values ? v_head : k_head;
  uint32_t* codes = reinterpret_cast<uint32_t*>(values ? c.v_codes : c.k_codes);
  uint8_t* scales = values ? c.v_scales : c.k_scales;
  const float enc = global_encode(values ? c.global_v : c.global_k);
  const int h = blockIdx.x * kThreads + threadIdx.x;  // pairs of lanes stay whole: dim/8 and `halves` are even
  if (h >= halves) return;
  const int t = kv_div(h, per_token);
  const int u = h - t * per_token.d;
  const int64_t slot = slots[t];
  if (slot < 0 || slot >= (int64_t)c.pages * c.page_size) return;  // padding
  float f[8];
  load_values<DT, VEC>(x, t * xt + head * xh + 8 * u, f);
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, __builtin_fabsf(f[i]));
  a = fmaxf(a, __shfl_xor(a, 1, 64));
  uint32_t byte;
  const uint32_t word = encode_half_group(f, a, enc, byte);
  const int page = kv_div((uint32_t)slot, c.page_div);
  const int64_t row = kv_row(c, page, head, (int)slot - page * c.page_size);
  codes[row * (c.dim / 8) + u] = word;
  if ((u & 1) == 0) scales[row * (c.dim / 16) + (u >> 1)] = (uint8_t)byte;
}

template <int DT>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(KvCache c, const int64_t* __restrict__ slots, void* __restrict__ k,
               void* __restrict__ v, int halves, KvDiv per_token) {
  const bool values = blockIdx.y >= (unsigned)c.heads;
  const int head = values ? blockIdx.y - c.heads : blockIdx.y;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(values ? c.v_codes : c.k_codes);
  const uint8_t* scales = values ? c.v_scales : c.k_scales;
  const float dec = global_decode(values ? c.global_v : c.global_k);
  const int h = blockIdx.x * kThreads + threadIdx.x;
  if (h >= halves) return;
  const int t = kv_div(h, per_token);
  const int u = h - t * per_token.d;
  const int64_t slot = slots[t];
  float q[8] = {};
  if (slot >= 0 && slot < (int64_t)c.pages * c.page_size) {
    const int page = kv_div((uint32_t)slot, c.page_div);
    const int64_t row = kv_row(c, page, head, (int)slot - page * c.page_size);
    e2m1_decode8_f32(codes[row * (c.dim / 8) + u], q);
    float sc;
    {
#pragma clang fp contract(off)
      sc = e4m3_decode(scales[row * (c.dim / 16) + (u >> 1)]) * dec;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)
      q[i] = q[i] * sc;
    }
  }
  store8<DT>(values ? v : k, ((int64_t)t * c.heads + head) * (c.dim / 8) + u, q);
}

}  // namespace

KvDiv kv_make_div(uint32_t d) {
  KvDiv r;
  r.d = d;
  r.shift = 0;
  while ((1ull << r.shift) < d) ++r.shift;
  r.mul = (uint32_t)((((1ull << r.shift) - d) << 32) / d + 1);
  return r;
}

hipError_t launch_kv_write(const KvCache& c, const void* k, const void* v, int dt, int64_t tokens,
                           int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                           const int64_t* slots, hipStream_t s) {
  const int halves = (int)(tokens * (c.dim / 8));
  const dim3 grid((halves + kThreads - 1) / kThreads, 2 * c.heads);
  const KvDiv per = kv_make_div(c.dim / 8);
  const int64_t lane_elems = dt == kF32 ? 4 : 8;
  const bool vec = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) == 0 &&
                   (k_token | k_head | v_token | v_head) % lane_elems == 0;
#define KV_WRITE(DT, VEC)                                                                          \
  kv_write_kernel<DT, VEC><<<grid, kThreads, 0, s>>>(c, k, v, k_token, k_head, v_token, v_head, slots, \
                                                     halves, per)
  if (dt == kF32) {
    if (vec) KV_WRITE(kF32, true); else KV_WRITE(kF32, false);
  } else if (dt == kF16) {
    if (vec) KV_WRITE(kF16, true); else KV_WRITE(kF16, false);
  } else {
    if (vec) KV_WRITE(kBF16, true); else KV_WRITE(kBF16, false);
  }
#undef KV_WRITE
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const int64_t* slots, int64_t tokens, void* k, void* v, int dt,
                          hipStream_t s) {
  const int halves = (int)(tokens * (c.dim / 8));
  const dim3 grid((halves + kThreads - 1) / kThreads, 2 * c.heads);
  const KvDiv per = kv_make_div(c.dim / 8);
  if (dt == kF32)
    kv_read_kernel<kF32><<<grid, kThreads, 0, s>>>(c, slots, k, v, halves, per);
  else if (dt == kF16)
    kv_read_kernel<kF16><<<grid, kThreads, 0, s>>>(c, slots, k, v, halves, per);
  else
    kv_read_kernel<kBF16><<<grid, kThreads, 0, s>>>(c, slots, k, v, halves, per);
  return hipGetLastError();
}

}  // namespace nvfp4
