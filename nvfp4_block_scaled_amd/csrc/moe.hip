// moe.hip -- a whole mixture-of-experts layer for a few tokens on NVFP4 expert
// weights (gfx950).
//
//     l = x R^T                               float64 sums: the choice hangs on them
//     chosen: the top_k largest l of a token (ties: the lowest index)
//     p = softmax of the chosen l (or of all of the token's)
//     g, u = x W_gate^T, x W_up^T             of each chosen expert, float32
//     h = g / (1 + exp(-g)) u
//     out = T( sum_j p_j W_down h_j )         in float32, rounded once
//
// Numbers.  A weight without its global scale, e2m1 * e4m3, has 6 significant
// bits and a magnitude of 0 or 2^-10 .. 2688: exact in bfloat16, whose matrix
// products then round nothing but their float32 sums.  What a weight meets is
// cut into bfloat16 pieces of 8 bits: x of 16 bits exactly (bfloat16 1,
// float16 2 pieces), of float32 exactly (3), h to 16 bits for 16-bit types
// (2^-16, far below the output's rounding) and to 24 for float32.  The global
// scales multiply the sums.
//
// Tokens are the columns of the products and weights their rows, 16 rows by 16
// tokens a product.  Weights are the traffic: each workgroup streams rows of
// one expert and meets all tokens of that expert at once.
#include "kv_device.h"
#include "layer_internal.h"

namespace nvfp4 {

namespace {

typedef uint32_t u32x4_8 __attribute__((ext_vector_type(4), aligned(8)));

constexpr int kUnit = 256;  // inner values of a row that a wave takes at a time: 64 a lane

// ----------------------------------------------------------------- pieces

// v as N bfloat16 whose sum it is (up to 2^-8N of it): the leading bits of what
// is left, the last one rounded.  An infinity stays in the first alone.
template <int N>
__device__ __forceinline__ void moe_pieces(float v, uint16_t (&p)[N]) {
  if (v != v) v = __builtin_nanf("");
  const bool finite = __builtin_fabsf(v) < __builtin_huge_valf();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t bits = __float_as_uint(v);
    p[i] = i + 1 < N ? (uint16_t)(bits >> 16) : __builtin_bit_cast(uint16_t, (__bf16)v);
    v = finite ? v - __uint_as_float(bits & 0xFFFF0000u) : 0.0f;
  }
}

// ----------------------------------------------------------------- router

__device__ __forceinline__ double moe_wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

constexpr int kRouterTokens = 4;  // of a wave: the expert's row is loaded once for them

// Workgroups 0 .. routers - 1: logits, a wave an expert and up to four tokens.  The
// others cut x into pieces (PX > 1).
template <int DT, int PX>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeLayer a, int routers) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if ((int)blockIdx.x >= routers) {
    if constexpr (PX > 1) {
      const int64_t all = (int64_t)a.tokens * a.k;
      const int64_t h = ((int64_t)(blockIdx.x - routers) * 256 + threadIdx.x);
      if (h >= all / 8) return;
      float v[8];
      load8x<DT>(a.x, h, v);
      uint16_t p[8][PX];
#pragma unroll
      for (int i = 0; i < 8; ++i) moe_pieces<PX>(v[i], p[i]);
#pragma unroll
      for (int j = 0; j < PX; ++j) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = p[2 * i][j] | (uint32_t)p[2 * i + 1][j] << 16;
        *reinterpret_cast<u32x4*>(a.x_pieces + j * all + 8 * h) = w;
      }
    }
    return;
  }
  const int chunks = (a.tokens + kRouterTokens - 1) / kRouterTokens;
  const int job = blockIdx.x * 4 + wave;
  const int expert = job / chunks, t0 = job % chunks * kRouterTokens;
  if (expert >= a.experts) return;
  double sum[kRouterTokens] = {};
  const int64_t row = (int64_t)expert * (a.k / 8);
  for (int i = lane; i < a.k / 8; i += 64) {
    float w[8];
    load8x<DT>(a.router, row + i, w);
#pragma unroll
    for (int j = 0; j < kRouterTokens; ++j) {
      float v[8];
      load8x<DT>(a.x, (int64_t)min(t0 + j, a.tokens - 1) * (a.k / 8) + i, v);
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[j] = __builtin_fma((double)w[c], (double)v[c], sum[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < kRouterTokens; ++j) {
    const double s = moe_wave_sum(sum[j]);
    if (lane == 0 && t0 + j < a.tokens) a.logits[(int64_t)(t0 + j) * a.experts + expert] = s;
  }
}

// An order of the logits as whole numbers; a NaN is below all.
__device__ __forceinline__ uint64_t moe_order(double l) {
  if (l != l) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(l + 0.0);  // -0 and 0 are equal
  return b >> 63 ? ~b : b | 1ull << 63;
}

// One workgroup a token.  An expert's rank is the number of those ahead of it.
__global__ void __launch_bounds__(256) moe_choose_kernel(MoeLayer a) {
  __shared__ uint64_t order[kMoeMaxExperts];
  __shared__ int chosen[kMoeMaxTopK];
  __shared__ double part[4];
  const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const double* l = a.logits + (int64_t)t * a.experts;
  for (int i = threadIdx.x; i < a.experts; i += 256) order[i] = moe_order(l[i]);
  __syncthreads();
  for (int i = threadIdx.x; i < a.experts; i += 256) {
    const uint64_t mine = order[i];
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < a.experts; ++j) rank += (order[j] > mine) | ((order[j] == mine) & (j < i));
    if (rank < a.top_k) chosen[rank] = i;
  }
  __syncthreads();
  const double top = l[chosen[0]];
  double sum = 0.0;
  if (a.normalize) {
    for (int j = 0; j < a.top_k; ++j) sum += exp(l[chosen[j]] - top);
  } else {
    for (int i = threadIdx.x; i < a.experts; i += 256) sum += exp(l[i] - top);
    sum = moe_wave_sum(sum);
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    sum = part[0] + part[1] + part[2] + part[3];
  }
  for (int j = threadIdx.x; j < a.top_k; j += 256) {
    a.expert_idx[t * a.top_k + j] = chosen[j];
    a.expert_weights[t * a.top_k + j] = (float)(exp(l[chosen[j]] - top) / sum);
  }
}

// ----------------------------------------------------------------- which experts

// The chosen experts of all tokens in LDS: each pair's (-1: none), and the list
// of the different ones in the order of their first pairs.
struct MoeLists {
  int idx[kMoeMaxPairs];
  int first[kMoeMaxExperts];
  int list[kMoeMaxExperts];
  int count;
};
__device__ __forceinline__ void moe_lists(const MoeLayer& a, MoeLists& s) {
  const int pairs = a.tokens * a.top_k;
  for (int i = threadIdx.x; i < a.experts; i += blockDim.x) s.first[i] = INT32_MAX;
  __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    int id = a.expert_idx[p];
    if (id < 0 || id >= a.experts) id = -1;
    s.idx[p] = id;
    if (id >= 0) atomicMin(&s.first[id], p);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    int count = 0;
    for (int base = 0; base < pairs; base += 64) {
      const int p = base + threadIdx.x, id = p < pairs ? s.idx[p] : -1;
      const bool leads = id >= 0 && s.first[id] == p;
      const uint64_t lanes = __ballot(leads);
      if (leads) s.list[count + __popcll(lanes & ((1ull << threadIdx.x) - 1))] = id;
      count += __popcll(lanes);
    }
    if (threadIdx.x == 0) s.count = count;
  }
  __syncthreads();
}
// The first pair of token `t` with `expert`, or -1.
__device__ __forceinline__ int moe_pair(const MoeLayer& a, const MoeLists& s, int t, int expert) {
  if (t >= a.tokens) return -1;
  for (int j = 0; j < a.top_k; ++j)
    if (s.idx[t * a.top_k + j] == expert) return t * a.top_k + j;
  return -1;
}

// ----------------------------------------------------------------- products

// 64 consecutive inner values of one row, as loaded: 4 groups of 16.
struct MoeWeights {
  uint32_t w[8], s;
};
__device__ __forceinline__ MoeWeights moe_load(const uint8_t* codes, const uint8_t* scales, int64_t row, int inner, int at) {
  MoeWeights r;
  const uint8_t* c = codes + row * (inner / 2) + at / 2;
  const uint8_t* s = scales + row * (inner / 16) + at / 16;
  if (at + 64 <= inner) {
    const u32x4_8 x = *reinterpret_cast<const u32x4_8*>(c), y = *reinterpret_cast<const u32x4_8*>(c + 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.w[i] = x[i];
      r.w[4 + i] = y[i];
    }
    __builtin_memcpy(&r.s, s, 4);
  } else {
    r.s = 0u;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      r.w[2 * g] = r.w[2 * g + 1] = 0u;
      if (at + 16 * g < inner) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(c + 8 * g);
        r.w[2 * g] = x.x;
        r.w[2 * g + 1] = x.y;
        r.s |= (uint32_t)s[g] << (8 * g);
      }
    }
  }
  return r;
}
// 8 weights (a dword of codes) times their block scale, exact in bfloat16.
__device__ __forceinline__ bf16x8 moe_decode8(uint32_t w, float s) {
  float v[8];
  e2m1_decode8_f32(w, v);
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1] * s), __float_as_uint(v[2 * i] * s), 0x07060302u);
  return __builtin_bit_cast(bf16x8, r);
}
template <int I>
__device__ __forceinline__ bf16x8 moe_values(const MoeWeights& r) {
  return moe_decode8(r.w[I], e4m3_decode_byte<I / 2>(r.s));
}

// 8 values of a column from element `at` on, zeros past `inner` and of columns that are not there.
__device__ __forceinline__ bf16x8 moe_column(const uint16_t* p, int at, int inner, bool live) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (live && at < inner) v = *reinterpret_cast<const u32x4*>(p + at);
  return __builtin_bit_cast(bf16x8, v);
}

// One unit: NR tiles of 16 rows by MT tiles of 16 tokens.  Lane l has row l % 16
// and inner values 64 (l / 16) .. of the unit on both sides.
template <int NR, int MT, int P>
__device__ __forceinline__ void moe_unit(const MoeWeights (&w)[NR], const uint16_t* const (&col)[MT], const bool (&live)[MT],
                                         int64_t plane, int at, int inner, f32x4 (&acc)[NR][MT]) {
  auto step = [&](auto index) {
    constexpr int I = decltype(index)::value;
    bf16x8 a[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) a[r] = moe_values<I>(w[r]);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int p = P - 1; p >= 0; --p) {  // the small pieces first
        const bf16x8 b = moe_column(col[m] + p * plane, at + 8 * I, inner, live[m]);
#pragma unroll
        for (int r = 0; r < NR; ++r) acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[r], b, acc[r][m], 0, 0, 0);
      }
  };
  step(std::integral_constant<int, 0>{});
  step(std::integral_constant<int, 1>{});
  step(std::integral_constant<int, 2>{});
  step(std::integral_constant<int, 3>{});
  step(std::integral_constant<int, 4>{});
  step(std::integral_constant<int, 5>{});
  step(std::integral_constant<int, 6>{});
  step(std::integral_constant<int, 7>{});
}

constexpr int kUpWaves = 4;

// 16 gate rows and the 16 up rows that go with them, of one expert: a workgroup, its waves
// each a share of the inner values.
template <int MT, int PX, int PH>
__global__ void __launch_bounds__(64 * kUpWaves) moe_up_kernel(MoeLayer a, const uint16_t* x, int64_t x_plane) {
  __shared__ MoeLists lists;
  __shared__ f32x4 part[kUpWaves][2][MT][64];
  moe_lists(a, lists);
  const int tiles = a.f / 16;
  const int which = blockIdx.x / tiles, f0 = (blockIdx.x - which * tiles) * 16;
  if (which >= lists.count) return;
  const int expert = __builtin_amdgcn_readfirstlane(lists.list[which]);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, quarter = lane >> 4;
  int pair[MT];
  const uint16_t* at_x[MT];
  bool live[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    pair[m] = moe_pair(a, lists, 16 * m + col, expert);
    live[m] = pair[m] >= 0;
    at_x[m] = x + (int64_t)min(16 * m + col, a.tokens - 1) * a.k;
  }
  f32x4 acc[2][MT] = {};
  const int units = (a.k + kUnit - 1) / kUnit;
  const int64_t row = (int64_t)expert * 2 * a.f + f0 + col;
  for (int u = wave; u < units; u += kUpWaves) {
    const int at = u * kUnit + 64 * quarter;
    const MoeWeights w[2] = {moe_load(a.up_codes, a.up_scales, row, a.k, at), moe_load(a.up_codes, a.up_scales, row + a.f, a.k, at)};
    moe_unit<2, MT, PX>(w, at_x, live, x_plane, at, a.k, acc);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][r][m][lane] = acc[r][m];
  __syncthreads();
  const float factor = global_decode(a.up_global ? a.up_global + expert : nullptr);
  const int64_t h_plane = (int64_t)a.tokens * a.top_k * a.f;
  for (int m = wave; m < MT; m += kUpWaves) {
    const int p = moe_pair(a, lists, 16 * m + col, expert);
    f32x4 g = part[0][0][m][lane], v = part[0][1][m][lane];
#pragma unroll
    for (int w = 1; w < kUpWaves; ++w) {
      g += part[w][0][m][lane];
      v += part[w][1][m][lane];
    }
    if (p < 0) continue;
    uint16_t piece[4][PH];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x1 = g[i] * factor, x2 = v[i] * factor;
      moe_pieces<PH>(x1 / (1.0f + expf(-x1)) * x2, piece[i]);
    }
#pragma unroll
    for (int j = 0; j < PH; ++j)
      *reinterpret_cast<u32x2*>(a.h_pieces + j * h_plane + (int64_t)p * a.f + f0 + 4 * quarter) =
          u32x2{piece[0][j] | (uint32_t)piece[1][j] << 16, piece[2][j] | (uint32_t)piece[3][j] << 16};
  }
}

constexpr int kDownWaves = 8;

// 16 columns of the output for all tokens: a workgroup, its waves equal runs of
// the units of all chosen experts' rows.
template <int DT, int MT, int PH>
__global__ void __launch_bounds__(64 * kDownWaves) moe_down_kernel(MoeLayer a) {
  __shared__ MoeLists lists;
  __shared__ f32x4 part[kDownWaves][MT][64];
  moe_lists(a, lists);
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, quarter = lane >> 4;
  const int units = (a.f + kUnit - 1) / kUnit, all = lists.count * units;
  const int64_t h_plane = (int64_t)a.tokens * a.top_k * a.f;
  f32x4 total[MT] = {};
  int unit = (int)((int64_t)all * wave / kDownWaves);
  const int last = (int)((int64_t)all * (wave + 1) / kDownWaves);
  while (unit < last) {
    const int which = unit / units;
    const int expert = __builtin_amdgcn_readfirstlane(lists.list[which]);
    const int end = min(last, (which + 1) * units);
    const uint16_t* at_h[MT];
    bool live[MT];
    float weight[MT];
    const float factor = global_decode(a.down_global ? a.down_global + expert : nullptr);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int t = 16 * m + col, p = moe_pair(a, lists, t, expert);
      live[m] = p >= 0;
      at_h[m] = a.h_pieces + (int64_t)max(p, 0) * a.f;
      weight[m] = 0.0f;
      if (p >= 0)  // an expert may stand twice among a token's
        for (int q = p; q < (t + 1) * a.top_k; ++q)
          if (lists.idx[q] == expert) weight[m] += a.expert_weights[q];
      weight[m] *= factor;
    }
    f32x4 acc[1][MT] = {};
    const int64_t row = (int64_t)expert * a.k + n0 + col;
    for (; unit < end; ++unit) {
      const int at = (unit - which * units) * kUnit + 64 * quarter;
      const MoeWeights w[1] = {moe_load(a.down_codes, a.down_scales, row, a.f, at)};
      moe_unit<1, MT, PH>(w, at_h, live, h_plane, at, a.f, acc);
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[m][i] = live[m] ? total[m][i] + weight[m] * acc[0][m][i] : total[m][i];
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) part[wave][m][lane] = total[m];
  __syncthreads();
  for (int m = wave; m < MT; m += kDownWaves) {
    const int t = 16 * m + col;
    f32x4 v = part[0][m][lane];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) v += part[w][m][lane];
    if (t >= a.tokens) continue;
    const int64_t at = (int64_t)t * a.k + n0 + 4 * quarter;
    if constexpr (DT == kF32)
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at) = v;
    else
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
  }
}

// ----------------------------------------------------------------- launches

constexpr int moe_x_pieces(int dt) { return dt == kF32 ? 3 : dt == kF16 ? 2 : 1; }
constexpr int moe_h_pieces(int dt) { return dt == kF32 ? 3 : 2; }

struct MoePlan {
  size_t logits, x, h, bytes;  // offsets in the workspace
};
MoePlan moe_plan(int64_t tokens, int64_t top_k, int64_t experts, int64_t k, int64_t f, int dt) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  MoePlan p;
  p.logits = 0;
  p.x = up((size_t)tokens * experts * 8);
  p.h = p.x + (moe_x_pieces(dt) > 1 ? up((size_t)moe_x_pieces(dt) * tokens * k * 2) : 0);
  p.bytes = p.h + up((size_t)moe_h_pieces(dt) * tokens * top_k * f * 2);
  return p;
}

template <int DT, int MT>
hipError_t launch_products(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT), PH = moe_h_pieces(DT);
  const int pairs = a.tokens * a.top_k, most = pairs < a.experts ? pairs : a.experts;
  const uint16_t* x = PX > 1 ? a.x_pieces : reinterpret_cast<const uint16_t*>(a.x);
  moe_up_kernel<MT, PX, PH><<<(unsigned)(most * (a.f / 16)), 64 * kUpWaves, 0, s>>>(a, x, (int64_t)a.tokens * a.k);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  moe_down_kernel<DT, MT, PH><<<(unsigned)(a.k / 16), 64 * kDownWaves, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT);
  const int chunks = (a.tokens + kRouterTokens - 1) / kRouterTokens;
  const int routers = a.router ? (a.experts * chunks + 3) / 4 : 0;
  const int64_t cuts = PX > 1 ? ((int64_t)a.tokens * a.k / 8 + 255) / 256 : 0;
  if (routers + cuts > 0) {
    moe_logits_kernel<DT, PX><<<(unsigned)(routers + cuts), 256, 0, s>>>(a, routers);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (a.router) {
    moe_choose_kernel<<<(unsigned)a.tokens, 256, 0, s>>>(a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (a.tokens <= 16) return launch_products<DT, 1>(a, s);
  if (a.tokens <= 32) return launch_products<DT, 2>(a, s);
  return launch_products<DT, 4>(a, s);
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t top_k, int64_t experts, int64_t k, int64_t f, int dt) {
  return moe_plan(tokens, top_k, experts, k, f, dt).bytes;
}

hipError_t launch_moe(MoeLayer a, int dt, void* workspace, hipStream_t s) {
  const MoePlan p = moe_plan(a.tokens, a.top_k, a.experts, a.k, a.f, dt);
  uint8_t* w = reinterpret_cast<uint8_t*>(workspace);
  a.logits = reinterpret_cast<double*>(w + p.logits);
  a.x_pieces = reinterpret_cast<uint16_t*>(w + p.x);
  a.h_pieces = reinterpret_cast<uint16_t*>(w + p.h);
  return dt == kF32 ? launch<kF32>(a, s) : dt == kF16 ? launch<kF16>(a, s) : launch<kBF16>(a, s);
}

}  // namespace nvfp4
