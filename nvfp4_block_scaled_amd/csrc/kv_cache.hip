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
// A workgroup takes consecutive tokens of one head's keys or values, so that
// for tokens of one page both the cache side (64 bytes of codes a token at dim
// 128, contiguous over tokens) and each token's values (256 contiguous bytes)
// are whole lines; the workgroups of all heads of the same tokens follow one
// another (16,384 tokens of 8 heads of 128 out of a fused projection, 86 MB:
// 21.7 us written, 4.0 TB/s; the heads one after another 25.6; float32, 153 MB:
// 26.9, 5.7 TB/s).
#include "kv_device.h"

namespace nvfp4 {

namespace {

constexpr int kThreads = 256;

// 8 consecutive values of type DT at element offset `e` as floats; VEC: 16-byte aligned.
template <int DT, bool VEC>
__device__ __forceinline__ void load_values(const void* base, int64_t e, float (&v)[8]) {
  if constexpr (VEC) {
    load8x<DT>(base, e >> 3, v);
  } else {
    const typename Elem<DT>::T* p = reinterpret_cast<const typename Elem<DT>::T*>(base) + e;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32<DT>(p[i]);
  }
}

// Half group h of a head: its token and place there.  A lane takes so many of
// them, a workgroup's width apart, all their loads ahead of the first use.
constexpr int kWriteEach = 2, kReadEach = 4;

template <int DT, bool VEC>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(KvCache c, const void* __restrict__ k, const void* __restrict__ v, int64_t k_token,
                int64_t k_head, int64_t v_token, int64_t v_head, const int64_t* __restrict__ slots,
                int halves, KvDiv per_token) {
  const int at = blockIdx.x % (2u * c.heads);  // keys' heads, then values'
  const bool values = at >= c.heads;
  const int head = values ? at - c.heads : at;
  const void* x = values ? v : k;
  const int64_t xt = values ? v_token : k_token, xh = values ? v_head : k_head;
  uint32_t* codes = reinterpret_cast<uint32_t*>(values ? c.v_codes : c.k_codes);
  uint8_t* scales = values ? c.v_scales : c.k_scales;
  const float enc = global_encode(values ? c.global_v : c.global_k);
  const int64_t slots_held = (int64_t)c.pages * c.page_size;
  const int h0 = blockIdx.x / (2u * c.heads) * (kThreads * kWriteEach) + threadIdx.x;
  int64_t slot[kWriteEach];
  int u[kWriteEach];
  float f[kWriteEach][8];
#pragma unroll
  for (int e = 0; e < kWriteEach; ++e) {
    const int h = h0 + e * kThreads;  // pairs of lanes stay whole: dim/8 and `halves` are even
    const int t = kv_div(min(h, halves - 1), per_token);
    u[e] = h - t * per_token.d;
    slot[e] = h < halves ? slots[t] : -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[e][i] = 0.0f;
    if (h < halves) load_values<DT, VEC>(x, t * xt + head * xh + 8 * u[e], f[e]);
  }
#pragma unroll
  for (int e = 0; e < kWriteEach; ++e) {
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, __builtin_fabsf(f[e][i]));
    a = fmaxf(a, __shfl_xor(a, 1, 64));
    uint32_t byte;
    const uint32_t word = encode_half_group(f[e], a, enc, byte);
    if (slot[e] >= 0 && slot[e] < slots_held) {  // else padding
      const int page = kv_div((uint32_t)slot[e], c.page_div);
      const int64_t row = kv_row(c, page, head, (int)slot[e] - page * c.page_size);
      codes[row * (c.dim / 8) + u[e]] = word;
      if ((u[e] & 1) == 0) scales[row * (c.dim / 16) + (u[e] >> 1)] = (uint8_t)byte;
    }
  }
}

// Outputs of more than kStream bytes do not stay in the last-level cache
// anyway: stored around it.  65,536 tokens of 8 heads of 128 (268 MB out):
// 51 us, 75 with ordinary stores; 16,384 tokens (67 MB): 15 us both ways,
// and what reads them next finds them in the cache.  (float32, 537 MB out: 226
// us, 2.7 TB/s; two stores a lane, 16 bytes of 32 each.)
constexpr int64_t kStream = (int64_t)128 << 20;

template <int DT, bool STREAM>
__device__ __forceinline__ void store_values(void* base, int64_t h, const float (&v)[8]) {
  if constexpr (!STREAM) {
    store8<DT>(base, h, v);
  } else if constexpr (DT == kF32) {
    f32x4* p = reinterpret_cast<f32x4*>(base) + 2 * h;
    __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, p);
    __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, p + 1);
  } else {
    __builtin_nontemporal_store(u32x4{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]),
                                      pack2<DT>(v[6], v[7])},
                                reinterpret_cast<u32x4*>(base) + h);
  }
}

template <int DT, bool STREAM>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(KvCache c, const int64_t* __restrict__ slots, void* __restrict__ k,
               void* __restrict__ v, int halves, KvDiv per_token) {
  const int at = blockIdx.x % (2u * c.heads);  // keys' heads, then values'
  const bool values = at >= c.heads;
  const int head = values ? at - c.heads : at;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(values ? c.v_codes : c.k_codes);
  const uint8_t* scales = values ? c.v_scales : c.k_scales;
  const float dec = global_decode(values ? c.global_v : c.global_k);
  const int64_t slots_held = (int64_t)c.pages * c.page_size;
  const int h0 = blockIdx.x / (2u * c.heads) * (kThreads * kReadEach) + threadIdx.x;
  int64_t slot[kReadEach];
  int t[kReadEach], u[kReadEach];
#pragma unroll
  for (int e = 0; e < kReadEach; ++e) {
    const int h = min(h0 + e * kThreads, halves - 1);
    t[e] = kv_div(h, per_token);
    u[e] = h - t[e] * per_token.d;
    slot[e] = slots[t[e]];
  }
  uint32_t word[kReadEach], byte[kReadEach];
#pragma unroll
  for (int e = 0; e < kReadEach; ++e) {
    word[e] = byte[e] = 0u;  // no slot: zeros
    if (slot[e] >= 0 && slot[e] < slots_held) {
      const int page = kv_div((uint32_t)slot[e], c.page_div);
      const int64_t row = kv_row(c, page, head, (int)slot[e] - page * c.page_size);
      word[e] = codes[row * (c.dim / 8) + u[e]];
      byte[e] = scales[row * (c.dim / 16) + (u[e] >> 1)];
    }
  }
#pragma unroll
  for (int e = 0; e < kReadEach; ++e) {
    if (h0 + e * kThreads >= halves) break;
    float q[8], sc;
    e2m1_decode8_f32(word[e], q);
    {
#pragma clang fp contract(off)
      sc = e4m3_decode(byte[e]) * dec;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)
      q[i] = q[i] * sc;
    }
    store_values<DT, STREAM>(values ? v : k, ((int64_t)t[e] * c.heads + head) * (c.dim / 8) + u[e], q);
  }
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
  const int each = kThreads * kWriteEach;
  const unsigned grid = (unsigned)((halves + each - 1) / each) * 2 * c.heads;
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
  const int each = kThreads * kReadEach;
  const unsigned grid = (unsigned)((halves + each - 1) / each) * 2 * c.heads;
  const KvDiv per = kv_make_div(c.dim / 8);
  const bool stream = 2 * tokens * c.heads * c.dim * (dt == kF32 ? 4 : 2) > kStream;
#define KV_READ(DT, STREAM) kv_read_kernel<DT, STREAM><<<grid, kThreads, 0, s>>>(c, slots, k, v, halves, per)
  if (dt == kF32) {
    if (stream) KV_READ(kF32, true); else KV_READ(kF32, false);
  } else if (dt == kF16) {
    if (stream) KV_READ(kF16, true); else KV_READ(kF16, false);
  } else {
    if (stream) KV_READ(kBF16, true); else KV_READ(kBF16, false);
  }
#undef KV_READ
  return hipGetLastError();
}

}  // namespace nvfp4
