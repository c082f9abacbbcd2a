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
// bits and a magnitude of 0 or 2^-10 .. 2688: exact in float16, whose matrix
// products then round nothing but their float32 sums.  What a weight meets is
// brought into float16's range by a power of two of its row (a token's x, a
// pair's h) and cut into pieces: bfloat16 x one, exact down to 2^-27 of the row's
// largest and smaller ones to within 2^-38 of it; float16 x as it is; float32 x
// and, for float16 and float32 layers, h two, 22 bits; h of bfloat16 layers one,
// 2^-11 of each, an eighth of the output's own rounding.  (In bfloat16 no power of
// two is needed, but decoding a weight takes two instructions, not one, and they
// bounded the kernels: 74 % of the vector units' time up, 64 % down.)  The global
// scales and the powers of two multiply the sums.
//
// Tokens are the columns of the products and weights their rows, 16 rows by 16
// tokens a product.  Weights are the traffic: each workgroup streams rows of
// one expert and meets all tokens of that expert at once.
//
// Measured, 16 tokens, 2 of 8 experts of 4096 x 14336, bfloat16: logits 5 us, up 122 -
// 126 (528 MB, 4.2 TB/s), down 81 - 87 (264 MB, 3.1 TB/s); a large copy reaches 5.1.  Waves
// wait 40 % of their time, the vector units are busy 33 and 37 %, LDS 28 %, the
// matrix cores 10 and 7 %: latency of the columns out of L2 and of the weights,
// which neither more loads ahead nor more waves shortened.
// 1 token, 8 of 64 of 2048 x 1024, 19 + 9 MB: 2.7, 15.9 and 9.2 us, a chain of
// logits, choice, weights and sums with little to overlap.
#include <atomic>

#include "layer_internal.h"
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {

namespace {

typedef uint32_t u32x4_8 __attribute__((ext_vector_type(4), aligned(8)));
typedef uint32_t u32_1 __attribute__((aligned(1)));

constexpr int kUnit = 256;  // inner values of a row that a wave takes at a time: 64 a lane

// ----------------------------------------------------------------- pieces

// Pieces of x (0: it is used as it lies) and of h.  Two of h for bfloat16 as well cost
// 1 to 4 % up to 16 tokens and 12 to 25 % from 32 on (32 tokens, 2 of 8 of 4096 x
// 14336: 351 us for 280).  With one the whole output's error against 64 bits is 1.667e-3 (16
// tokens, 2 of 8 of 4096 x 14336), of which the output's own rounding alone is 1.654e-3.
constexpr int moe_x_pieces(int dt) { return dt == kF32 ? 2 : dt == kF16 ? 0 : 1; }
constexpr int moe_h_pieces(int dt) { return dt == kBF16 ? 1 : 2; }

// e such that 2^-e brings a row of largest magnitude `top` (its bits) to 2^13 ..
// 2^14.  Rows of zeros, infinities and NaN stay as they are, and 2^126 is as far as
// it goes: float16's smallest step is then below float32's, and nothing is lost.
__device__ __forceinline__ int moe_exponent(uint32_t top) {
  const int field = (int)(top >> 23);
  return top == 0u || field == 255 ? 0 : max(field - 140, -126);
}
// Four values times 2^-e as P float16 pieces, two to a dword: each piece is one
// rounding of what those before it leave, and one instruction.
template <int P>
__device__ __forceinline__ void moe_pieces(const float (&v)[4], int e, u32x2 (&p)[P]) {
  const float by = __uint_as_float((uint32_t)(127 - e) << 23);
  _Float16 y[4];
#pragma unroll
  for (int j = 0; j < P; ++j) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = j == 0 ? (_Float16)(v[i] * by) : (_Float16)__builtin_fmaf(v[i], by, -(float)y[i]);
    p[j] = u32x2{__builtin_bit_cast(uint32_t, f16x2{y[0], y[1]}), __builtin_bit_cast(uint32_t, f16x2{y[2], y[3]})};
  }
}

// A global scale's decode factor as a number of 0.5 .. 1 and a power of two, which
// goes with the row's: a sum times the factor alone, or times the row's power alone,
// can pass float32's range where the layer does not.
struct MoeFactor {
  float by;
  int exponent;
};
__device__ __forceinline__ MoeFactor moe_factor(const float* global, int expert) {
  const float factor = global_decode(global ? global + expert : nullptr);
  return MoeFactor{__builtin_amdgcn_frexp_mantf(factor), __builtin_amdgcn_frexp_expf(factor)};
}

// ----------------------------------------------------------------- router

__device__ __forceinline__ double moe_wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Workgroups 0 .. routers - 1: logits, a workgroup an expert and TOKENS tokens, for
// which its row is loaded once.  The others, one a token, cut x into pieces (PX >
// 0) and clear the largest |h| of the token's pairs.
template <int DT, int PX, int TOKENS>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeLayer a, int routers) {
  if ((int)blockIdx.x >= routers) {
    const int t = blockIdx.x - routers, eights = a.k / 8;
    for (int j = threadIdx.x; j < a.top_k; j += 256) a.h_top[t * a.top_k + j] = 0u;
    if constexpr (PX > 0) {
      __shared__ uint32_t tops[4];
      const int64_t first = (int64_t)t * eights;
      uint32_t top = 0u;
      for (int h = threadIdx.x; h < eights; h += 256) {
        float v[8];
        load8x<DT>(a.x, first + h, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
      }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
      if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
      __syncthreads();
      top = max(max(tops[0], tops[1]), max(tops[2], tops[3]));
      const int e = moe_exponent(top);
      if (threadIdx.x == 0) a.x_exponent[t] = e;
      for (int h = threadIdx.x; h < eights; h += 256) {
        float v[8];
        load8x<DT>(a.x, first + h, v);
        u32x2 lo[PX], hi[PX];
        moe_pieces<PX>({v[0], v[1], v[2], v[3]}, e, lo);
        moe_pieces<PX>({v[4], v[5], v[6], v[7]}, e, hi);
#pragma unroll
        for (int j = 0; j < PX; ++j)
          *reinterpret_cast<u32x4*>(a.x_pieces + ((int64_t)j * a.tokens + t) * a.k + 8 * h) =
              u32x4{lo[j].x, lo[j].y, hi[j].x, hi[j].y};
      }
    }
    return;
  }
  __shared__ double part[4][TOKENS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chunks = (a.tokens + TOKENS - 1) / TOKENS;
  const int expert = blockIdx.x / chunks, t0 = (blockIdx.x - expert * chunks) * TOKENS;
  double sum[TOKENS] = {};
  const int pieces = a.k / 8;
  const int64_t row = (int64_t)expert * pieces;
#pragma unroll 2
  for (int i = threadIdx.x; i < pieces; i += 256) {
    float w[8];
    load8x<DT>(a.router, row + i, w);
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      float v[8];
      load8x<DT>(a.x, (int64_t)min(t0 + j, a.tokens - 1) * pieces + i, v);
#pragma unroll
      for (int c = 0; c < 8; ++c) sum[j] = __builtin_fma((double)w[c], (double)v[c], sum[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < TOKENS; ++j) {
    const double x = moe_wave_sum(sum[j]);
    if (lane == 0) part[wave][j] = x;
  }
  __syncthreads();
  if (threadIdx.x < TOKENS && t0 + threadIdx.x < a.tokens)
    a.logits[(int64_t)(t0 + threadIdx.x) * a.experts + expert] =
        (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}

// An order of the logits as whole numbers; a NaN is below all.
__device__ __forceinline__ uint64_t moe_order(double l) {
  if (l != l) return 0;
  const uint64_t b = (uint64_t)__double_as_longlong(l + 0.0);  // -0 and 0 are equal
  return b >> 63 ? ~b : b | 1ull << 63;
}
// The chosen experts of tokens t0 .. t0 + count - 1 by the whole workgroup: an
// expert's rank is the number of those ahead of it.  order: count * experts words.
__device__ __forceinline__ void moe_choose(const MoeLayer& a, int t0, int count, uint64_t* order, int* chosen) {
  const int all = count * a.experts;
  for (int i = threadIdx.x; i < all; i += blockDim.x) order[i] = moe_order(a.logits[(int64_t)t0 * a.experts + i]);
  __syncthreads();
  for (int i = threadIdx.x; i < all; i += blockDim.x) {
    const int t = count == 1 ? 0 : i / a.experts, e = i - t * a.experts;
    const uint64_t mine = order[i];
    const uint64_t* of = order + t * a.experts;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < a.experts; ++j) rank += (of[j] > mine) | ((of[j] == mine) & (j < e));
    if (rank < a.top_k) chosen[t * a.top_k + rank] = e;
  }
  __syncthreads();
}
// Their weights, a wave a token.
__device__ __forceinline__ void moe_weigh(const MoeLayer& a, int t0, int count, const int* chosen) {
  const int lane = threadIdx.x & 63;
  for (int t = threadIdx.x >> 6; t < count; t += blockDim.x >> 6) {
    const double* l = a.logits + (int64_t)(t0 + t) * a.experts;
    const int mine = lane < a.top_k ? chosen[t * a.top_k + lane] : 0;
    const double top = l[chosen[t * a.top_k]];
    const double p = lane < a.top_k ? exp(l[mine] - top) : 0.0;
    double sum = p;
    if (!a.normalize) {
      sum = 0.0;
      for (int i = lane; i < a.experts; i += 64) sum += exp(l[i] - top);
    }
    sum = moe_wave_sum(sum);
    if (lane < a.top_k) {
      a.expert_idx[(t0 + t) * a.top_k + lane] = mine;
      a.expert_weights[(t0 + t) * a.top_k + lane] = (float)(p / sum);
    }
  }
}

// One workgroup a token.
__global__ void __launch_bounds__(256) moe_choose_kernel(MoeLayer a) {
  __shared__ uint64_t order[kMoeMaxExperts];
  __shared__ int chosen[kMoeMaxTopK];
  moe_choose(a, blockIdx.x, 1, order, chosen);
  moe_weigh(a, blockIdx.x, 1, chosen);
}

// Whether every workgroup of the up products finds out the choice for itself, and
// one more writes it down: less than a launch of its own takes while that is a few
// hundred steps a thread.  Of 64 experts, kernels without the gaps between them:
// 1 token 27.9 us inside, 31.3 apart; 4 tokens 55.8 and 57.8; 8 tokens 77.0 and 76.8
// (and a gap more); 16 tokens 99.4 and 94.5, past the rule.
constexpr int kChooseMost = 512;
constexpr bool moe_choose_inside(int tokens, int experts) {
  const int all = tokens * experts;
  return all <= kChooseMost && (all + 255) / 256 * experts <= 320;
}

// ----------------------------------------------------------------- which experts

// The chosen experts of all tokens in LDS: each pair's (-1: none), and the list
// of the different ones in the order of their first pairs.
struct MoeLists {
  int *idx, *first, *list;
  int* count;
  int* exponent;  // of each token's x (kMoeMaxTokens, up products) or each pair's h (down products)
  float* weight;  // of each pair (down products)
};
constexpr int moe_list_words(int pairs, int experts) {
  return (pairs + 2 * experts + 1 + (pairs > kMoeMaxTokens ? pairs : kMoeMaxTokens) + pairs + 3) / 4 * 4;
}
__device__ __forceinline__ MoeLists moe_lists_at(const MoeLayer& a, void* lds) {
  int* w = reinterpret_cast<int*>(lds);
  const int pairs = a.tokens * a.top_k;
  int* const exponent = w + pairs + 2 * a.experts + 1;
  return MoeLists{w,        w + pairs, w + pairs + a.experts, w + pairs + 2 * a.experts,
                  exponent, reinterpret_cast<float*>(exponent + (pairs > kMoeMaxTokens ? pairs : kMoeMaxTokens))};
}
// CHOOSE: from the logits (scratch: tokens * experts words of 64 bits in LDS).
template <bool CHOOSE>
__device__ __forceinline__ void moe_lists(const MoeLayer& a, const MoeLists& s, uint64_t* scratch) {
  const int pairs = a.tokens * a.top_k;
  for (int i = threadIdx.x; i < a.experts; i += blockDim.x) s.first[i] = INT32_MAX;
  if constexpr (CHOOSE) moe_choose(a, 0, a.tokens, scratch, s.idx);
  else __syncthreads();
  for (int p = threadIdx.x; p < pairs; p += blockDim.x) {
    int id = CHOOSE ? s.idx[p] : a.expert_idx[p];
    if (id < 0 || id >= a.experts) id = -1;
    if constexpr (!CHOOSE) s.idx[p] = id;
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
    if (threadIdx.x == 0) *s.count = count;
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
//
// A wave's unit: 256 inner values of NR tiles of 16 weight rows, and of the
// columns (x or h of a token) that meet them.  A product's operand is 8 values of
// lane l's row l % 16 from value 8 (l / 16) on, so that neighbouring lanes read
// different rows; loaded that way, every 16 bytes are a cache access of their
// own, and accesses bound the kernels (0.82 a clock and CU, 16 tokens, 2 of 8
// experts of 4096 x 14336: 141 us up, 140 us down).  So a wave loads whole lines,
// 8 lanes a row's 128 bytes, and turns them round in LDS of its own, where no
// other wave waits for it; rows are padded by 16 bytes, which spreads the reads of
// 8 rows over the banks.  The next units' loads are under way meanwhile.

// In LDS, of one wave.  NS: columns in LDS at a time; a last one holds zeros, for
// the lanes whose token has no column among them.
template <int NR, int NS, int P>
struct MoeStage {
  u32x4 codes[NR][16][8 + 1];       // row, chunk of 32 values
  uint32_t scales[NR][16][4];       // row, 4 groups of 16
  u32x4 columns[P][NS + 1][32 + 1]; // column, chunk of 8 values
  __device__ __forceinline__ void clear() {
    if ((threadIdx.x & 63) < 32)
#pragma unroll
      for (int p = 0; p < P; ++p) columns[p][NS][threadIdx.x & 63] = u32x4{0u, 0u, 0u, 0u};
  }
};

// Rows of weights: whole 64s with their scales at whole dwords; any from 64 values
// on; and shorter ones, whose every piece is tested.
enum { kWhole, kAny, kShort };

// One unit's weights on their way: lane l has chunk l % 8 of rows l / 8 and l / 8
// + 8, and the scales of row l / 4, groups 4 (l % 4) ..
//
// No branch stands between a wave's loads, here and below: behind one the compiler
// cannot count what is on its way, and waits for all of it.  So a lane past a
// row's end loads the row's beginning; its weights become 0 by their scales when
// they are staged (MoeStage's columns may hold anything there that is in their row
// anyway), and columns that are too many are the last one again.  Addresses are
// one of the wave and 32 bits of the lane.
template <int NR>
struct MoeWeights {
  u32x4 c[NR][2];
  uint32_t s[NR];
};
template <int NR, int ROWS>
__device__ __forceinline__ void moe_load(MoeWeights<NR>& w, const uint8_t* codes, const uint8_t* scales, const int64_t (&row0)[NR],
                                         int inner, int unit) {
  const int lane = threadIdx.x & 63;
  const uint32_t row_bytes = inner / 2, groups = inner / 16;
  const int from = unit * kUnit + 32 * (lane & 7), group = unit * (kUnit / 16) + 4 * (lane & 3);
  if constexpr (ROWS == kWhole) {
    const uint32_t code_at = (lane >> 3) * row_bytes + (from < inner ? 16 * (lane & 7) : 0);
    const uint32_t code_at2 = code_at + 8 * row_bytes;
    const uint32_t scale_at = (lane >> 2) * groups + (group < (int)groups ? 4 * (lane & 3) : 0);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint8_t* c = codes + row0[r] * row_bytes + unit * (kUnit / 2);
      const uint8_t* s = scales + row0[r] * groups + unit * (kUnit / 16);
      w.c[r][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_8*>(c + code_at));
      w.c[r][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_8*>(c + code_at2));
      w.s[r] = *reinterpret_cast<const uint32_t*>(s + scale_at);  // 8 units share a line: kept
    }
  } else if constexpr (ROWS == kAny) {
    // A chunk or a dword of scales that would pass its row's end ends there with it
    // (moe_stage moves it to its place).  Scales lie anywhere, and so do the loads.
    const uint32_t code_at = (lane >> 3) * row_bytes + min(from, inner - 32) / 2;
    const uint32_t scale_at = (lane >> 2) * groups + min(group, (int)groups - 4);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint8_t* c = codes + row0[r] * row_bytes;
      const uint8_t* s = scales + row0[r] * groups;
      w.c[r][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_8*>(c + code_at));
      w.c[r][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_8*>(c + code_at + 8 * row_bytes));
      w.s[r] = *reinterpret_cast<const u32_1*>(s + scale_at);
    }
  } else {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint8_t* s = scales + (row0[r] + (lane >> 2)) * groups + group;
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const uint8_t* p = codes + (row0[r] + (lane >> 3) + 8 * d) * row_bytes + from / 2;
        u32x4 v = {0u, 0u, 0u, 0u};
        if (from + 32 <= inner) {
          v = *reinterpret_cast<const u32x4_8*>(p);
        } else if (from < inner) {
          const u32x2 half = *reinterpret_cast<const u32x2*>(p);
          v.x = half.x;
          v.y = half.y;
        }
        w.c[r][d] = v;
      }
      w.s[r] = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (group + i < (int)groups) w.s[r] |= (uint32_t)s[i] << (8 * i);
    }
  }
}
template <int ROWS, int NR, int NS, int P>
__device__ __forceinline__ void moe_stage(MoeStage<NR, NS, P>& l, const MoeWeights<NR>& w, int inner, int unit) {
  const int lane = threadIdx.x & 63;
  const bool there = unit * kUnit + 64 * (lane & 3) < inner;
  const bool half = unit * kUnit + 32 * (lane & 7) == inner - 16;
  const int over = max(unit * (kUnit / 16) + 4 * (lane & 3) - (inner / 16 - 4), 0);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      u32x4 c = w.c[r][d];
      if (ROWS == kAny && half) c = u32x4{c.z, c.w, 0u, 0u};
      l.codes[r][(lane >> 3) + 8 * d][lane & 7] = c;
    }
    uint32_t scales = w.s[r];
    if constexpr (ROWS == kWhole) scales = there ? scales : 0u;
    if constexpr (ROWS == kAny) scales = over < 4 ? scales >> (8 * over) : 0u;
    l.scales[r][lane >> 2][lane & 3] = scales;
  }
}

// NS columns of x pieces of a unit on their way: lane l has chunk l % 32 of
// columns l / 32, l / 32 + 2 ..
template <int NS, int P>
struct MoeColumns {
  u32x4 v[P][NS / 2];
};
// `at`: where this lane's columns begin, of `inner` values; a piece is `plane` behind the other.
template <int NS, int P>
__device__ __forceinline__ void moe_load(MoeColumns<NS, P>& x, const uint16_t* base, int64_t plane, const int (&at)[NS / 2], int inner,
                                         int unit) {
  const uint32_t chunk = threadIdx.x & 31;
  const uint32_t from = unit * kUnit + 8 * (int)chunk < inner ? 8 * chunk : 0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const uint16_t* b = base + p * plane + unit * kUnit;
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) x.v[p][i] = *reinterpret_cast<const u32x4*>(b + (uint32_t)(at[i] + from));
  }
}
template <int NR, int NS, int P>
__device__ __forceinline__ void moe_stage(MoeStage<NR, NS, P>& l, const MoeColumns<NS, P>& x) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
#pragma unroll
  for (int i = 0; i < NS / 2; ++i)
#pragma unroll
    for (int p = 0; p < P; ++p) l.columns[p][2 * i + half][lane & 31] = x.v[p][i];
}

// NS columns of h on their way, float32: lane l has values 4 l .. 4 l + 3 of each.
// They become pieces when they are staged.  row, exponent: of slot i, in lane i.
template <int NS>
struct MoeHidden {
  f32x4 v[NS];
};
template <int NS>
__device__ __forceinline__ void moe_load(MoeHidden<NS>& x, const float* base, int row, int inner, int unit) {
  const int from = 4 * (threadIdx.x & 63);
  const uint32_t at = unit * kUnit + from < inner ? from : 0;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    x.v[i] = *reinterpret_cast<const f32x4*>(base + (int64_t)__builtin_amdgcn_readlane(row, i) * inner + unit * kUnit + at);
}
template <int NS, int P>
__device__ __forceinline__ void moe_stage(MoeStage<1, NS, P>& l, const MoeHidden<NS>& x, int exponent, int count) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (i < count) {
      u32x2 piece[P];
      moe_pieces<P>({x.v[i][0], x.v[i][1], x.v[i][2], x.v[i][3]}, __builtin_amdgcn_readlane(exponent, i), piece);
#pragma unroll
      for (int p = 0; p < P; ++p) reinterpret_cast<u32x2*>(l.columns[p][i])[lane] = piece[p];
    }
}

// What a wave's lanes have written to its LDS, its other lanes may read.
__device__ __forceinline__ void moe_settle() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 8 weights (a dword of codes) times their block scale, exact in float16.
__device__ __forceinline__ f16x8 moe_decode8(uint32_t w, _Float16 s) {
  const f16x2 sc = {s, s};
  const f16x2 a = e2m1_decode2_f16<0>(w) * sc, b = e2m1_decode2_f16<1>(w) * sc;
  const f16x2 c = e2m1_decode2_f16<2>(w) * sc, d = e2m1_decode2_f16<3>(w) * sc;
  return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The products of what is staged.  Lane l has row l % 16 and values 64 (l / 16) ..
// + 63 of the unit on both sides.  slot[m]: this lane's column of tile m among
// those staged, or NS.  tiles: which tiles have any.
template <int NR, int MT, int NS, int P>
__device__ __forceinline__ void moe_products(const MoeStage<NR, NS, P>& l, const int (&slot)[MT], uint32_t tiles,
                                             f32x4 (&acc)[NR][MT]) {
  const int lane = threadIdx.x & 63, row = lane & 15, quarter = lane >> 4;
  f16x2 scale[NR][2];
  u32x4 codes[NR][2];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const uint32_t s = l.scales[r][row][quarter];
    scale[r][0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)s, 1.0f, false);
    scale[r][1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)s, 1.0f, true);
#pragma unroll
    for (int j = 0; j < 2; ++j) codes[r][j] = l.codes[r][row][2 * quarter + j];
  }
  // The columns of the next step are read while this one's are multiplied; the
  // order is fixed, as all eight steps' would be read at once otherwise, for a
  // third of the registers.
  u32x4 b[2][MT][P];
  auto read = [&](int i) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        b[i & 1][m][p] = l.columns[p][slot[m]][8 * quarter + i];
      }
  };
  read(0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i < 7) read(i + 1);
    __builtin_amdgcn_sched_barrier(0);
    f16x8 a[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) a[r] = moe_decode8(codes[r][i >> 2][i & 3], (i & 2) ? scale[r][i >> 2].y : scale[r][i >> 2].x);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (MT > 1 && !(tiles >> m & 1u)) continue;
#pragma unroll
      for (int p = P - 1; p >= 0; --p) {  // the small pieces first
#pragma unroll
        for (int r = 0; r < NR; ++r)
          acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[r], __builtin_bit_cast(f16x8, b[i & 1][m][p]), acc[r][m], 0, 0, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The tokens of one expert.  Lane t < 64 has token t's first pair with it.
struct MoeTokens {
  uint64_t live;  // which tokens
  int count;
};
__device__ __forceinline__ MoeTokens moe_tokens(int pair) {
  MoeTokens r;
  r.live = __ballot(pair >= 0);
  r.count = __builtin_popcountll(r.live);
  return r;
}
// Which of them token t is.
__device__ __forceinline__ int moe_rank(const MoeTokens& k, int t) {
  return __builtin_popcountll(k.live & ((1ull << t) - 1));
}
// This lane's column of each tile among those from `from` on, and the tiles that have any.
template <int NS, int MT>
__device__ __forceinline__ uint32_t moe_slots(const MoeTokens& k, int from, int (&slot)[MT]) {
  uint32_t tiles = 0u;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = 16 * m + (threadIdx.x & 15), at = moe_rank(k, t) - from;
    slot[m] = (k.live >> t & 1u) && at >= 0 && at < NS ? at : NS;
    tiles |= __any(slot[m] < NS) ? 1u << m : 0u;
  }
  return tiles;
}

constexpr int kUpWaves = 4, kUpAhead = 2;  // (3 ahead: 126 us for 124, 16 tokens, 2 of 8 of 4096 x 14336)

// 16 gate rows and the 16 up rows that go with them, of one expert, are a job; KW
// waves (all four of a workgroup, or one) take a job, each a share of the inner
// values, and go on to every so many-th.  Weights are on their way two units ahead,
// columns one, over the jobs' ends; at a job's end one wave in turn joins the four
// sums while the others go on.  CHOOSE: moe_choose_inside, and the last workgroup writes the
// choice.  PX: pieces of x here (1 or 2).
constexpr size_t kUpRows = kUpWaves * 2 * kMoeMaxTokens * sizeof(int);
// LDS without the lists: the waves' stages and, for the join, their sums.
template <int MT, int NS, int PX, int KW>
constexpr size_t up_bytes() {
  return kUpWaves * (sizeof(MoeStage<2, NS, PX>) + (KW > 1 ? 2 * MT * 1024 : 0));
}
// Workgroups of a CU: what has room in registers, and in LDS beside lists of `lists`
// bytes (32 tokens, 8 of 64 of 2048 x 1024, bfloat16, two a CU for a launch of three: 120
// us for 133; float32 with 16 columns at a time, one for two: 42 for 45, 16 tokens, 2 of 2 of 2048 x 4096).
template <int MT, int NS, int PX, int KW>
constexpr int up_groups_a_cu(size_t lists) {
  constexpr int registers = MT * PX <= 2 && NS <= 8 ? 3 : 2;
  const int room = (int)(160 * 1024 / (up_bytes<MT, NS, PX, KW>() + kUpRows + lists));
  return room < 1 ? 1 : room < registers ? room : registers;
}

template <int MT, int NS, int PX, int KW, int ROWS, bool CHOOSE>
__global__ void __launch_bounds__(64 * kUpWaves, (up_groups_a_cu<MT, NS, PX, KW>(0))) moe_up_kernel(MoeLayer a, const uint16_t* x) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int rows_of[kUpWaves][2][kMoeMaxTokens];  // of this job's expert and the next one's: its tokens
  static_assert(sizeof(rows_of) == kUpRows, "LDS");
  const MoeLists lists = moe_lists_at(a, lds);
  uint8_t* const mine = lds + 4 * moe_list_words(a.tokens * a.top_k, a.experts);
  if (threadIdx.x < a.tokens) lists.exponent[threadIdx.x] = a.x_exponent ? a.x_exponent[threadIdx.x] : 0;
  moe_lists<CHOOSE>(a, lists, reinterpret_cast<uint64_t*>(mine));
  const int groups = (int)gridDim.x - (CHOOSE ? 1 : 0);
  if (CHOOSE && (int)blockIdx.x == groups) {
    moe_weigh(a, 0, a.tokens, lists.idx);
    return;
  }
  constexpr int kJobs = kUpWaves / KW;  // of a workgroup at a time
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int share = wave % KW, stride = groups * kJobs;
  const int tiles = a.f / 16, jobs = __builtin_amdgcn_readfirstlane(*lists.count) * tiles;
  const int units = (a.k + kUnit - 1) / kUnit;
  const int64_t plane = (int64_t)a.tokens * a.k;
  using Stage = MoeStage<2, NS, PX>;
  Stage& stage = reinterpret_cast<Stage*>(mine)[wave];
  stage.clear();
  f32x4* const parts = reinterpret_cast<f32x4*>(mine + kUpWaves * sizeof(Stage));  // [wave][2][MT][64]
  // A job: tile `tile` of the which-th expert.  (All of it in scalar registers.)
  struct Job {
    int at, which, tile;
  };
  const int step_which = __builtin_amdgcn_readfirstlane(stride / tiles), step_tile = stride - step_which * tiles;
  auto advance = [&](Job& j) {
    j.at += stride;
    j.which += step_which;
    j.tile += step_tile;
    if (j.tile >= tiles) {
      j.tile -= tiles;
      ++j.which;
    }
  };
  auto expert_of = [&](const Job& j) { return __builtin_amdgcn_readfirstlane(lists.list[j.which]); };

  // h of tile m of a job's tokens from its gate and up sums.
  auto hidden = [&](const Job& job, int m, const f32x4& g, const f32x4& v) {
    const int expert = expert_of(job), f0 = job.tile * 16;
    const int t = 16 * m + (lane & 15), p = moe_pair(a, lists, t, expert);
    const MoeFactor factor = moe_factor(a.up_global, expert);
    const int e = lists.exponent[min(t, a.tokens - 1)] + factor.exponent;
    f32x4 h;
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x1 = __builtin_ldexpf(g[i] * factor.by, e), x2 = __builtin_ldexpf(v[i] * factor.by, e);
      h[i] = x1 / (1.0f + expf(-x1)) * x2;
      top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    if (p < 0) return;
    *reinterpret_cast<f32x4*>(a.hidden + (int64_t)p * a.f + f0 + 4 * (lane >> 4)) = h;
    if (lane < 16) atomicMax(a.h_top + p, top);  // (in any order the same)
  };
  // The sums of a job, number `n` of this workgroup's.
  auto finish = [&](const Job& job, int n, const f32x4(&acc)[2][MT]) {
    if constexpr (KW == 1) {
#pragma unroll
      for (int m = 0; m < MT; ++m) hidden(job, m, acc[0][m], acc[1][m]);
    } else {
      f32x4* const part = parts;
      if (n > 0) lds_barrier();  // the last job's are read
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int m = 0; m < MT; ++m) part[((wave * 2 + r) * MT + m) * 64 + lane] = acc[r][m];
      lds_barrier();
      for (int m = (wave + n) % kUpWaves; m < MT; m += kUpWaves) {
        f32x4 g = part[m * 64 + lane], v = part[(MT + m) * 64 + lane];
#pragma unroll
        for (int i = 1; i < kUpWaves; ++i) {
          g += part[((i * 2) * MT + m) * 64 + lane];
          v += part[((i * 2 + 1) * MT + m) * 64 + lane];
        }
        hidden(job, m, g, v);
      }
    }
  };

  Job job;
  job.at = (int)blockIdx.x * kJobs + wave / KW;
  if (job.at >= jobs) return;
  job.which = __builtin_amdgcn_readfirstlane(job.at / tiles);
  job.tile = job.at - job.which * tiles;
  if (KW > 1 && share >= units) {  // fewer units than waves
    const f32x4 none[2][MT] = {};
    for (int n = 0; job.at < jobs; advance(job), ++n) finish(job, n, none);
    return;
  }

  // The unit whose weights are loaded next; the last one again when all are.
  Job w_job = job;
  int w_unit = share;
  int64_t w_row = (int64_t)expert_of(job) * 2 * a.f + job.tile * 16;
  auto load_weights = [&](MoeWeights<2>& to) {
    moe_load<2, ROWS>(to, a.up_codes, a.up_scales, {w_row, w_row + a.f}, a.k, w_unit);
    if (w_unit + KW < units) {
      w_unit += KW;
    } else if (w_job.at + stride < jobs) {
      w_unit = share;
      advance(w_job);
      w_row = (int64_t)expert_of(w_job) * 2 * a.f + w_job.tile * 16;
    }
  };

  // The tokens of a job's expert, and where this lane's columns of x begin.
  MoeTokens tokens, next_tokens;
  int at[NS / 2];
  auto place = [&](const MoeTokens& k, const int* row_of, int from, int(&to)[NS / 2]) {
#pragma unroll
    for (int i = 0; i < NS / 2; ++i) to[i] = row_of[min(from + 2 * i + (lane >> 5), k.count - 1)] * a.k;
  };
  auto open = [&](const Job& j, MoeTokens& k, int* row_of) {
    const int pair = moe_pair(a, lists, lane, expert_of(j));
    k = moe_tokens(pair);
    moe_settle();
    if (pair >= 0) row_of[moe_rank(k, lane)] = lane;
    moe_settle();
    place(k, row_of, 0, at);
  };
  MoeWeights<2> w[kUpAhead];
  MoeColumns<NS, PX> columns;
  int u = share, n = 0;
  load_weights(w[0]);
  open(job, tokens, rows_of[wave][0]);
  moe_load<NS, PX>(columns, x, plane, at, a.k, u);
  load_weights(w[1]);
  int slot[MT];
  uint32_t first = moe_slots<NS, MT>(tokens, 0, slot);
  f32x4 acc[2][MT] = {};
  for (;;) {
#pragma unroll
    for (int j = 0; j < kUpAhead; ++j) {
      moe_stage<ROWS>(stage, w[j], a.k, u);
      moe_stage(stage, columns);
      moe_settle();
      const bool last = u + KW >= units, more_jobs = job.at + stride < jobs;
      if (last && more_jobs) {
        Job next = job;
        advance(next);
        open(next, next_tokens, rows_of[wave][(n + 1) & 1]);
      }
      moe_load<NS, PX>(columns, x, plane, at, a.k, last ? share : u + KW);
      load_weights(w[j]);
      moe_products<2, MT>(stage, slot, first, acc);
      for (int from = NS; from < tokens.count; from += NS) {  // more tokens than have room
        MoeColumns<NS, PX> more;
        int at2[NS / 2], slot2[MT];
        place(tokens, rows_of[wave][n & 1], from, at2);
        moe_load<NS, PX>(more, x, plane, at2, a.k, u);
        moe_settle();
        moe_stage(stage, more);
        moe_settle();
        const uint32_t some = moe_slots<NS, MT>(tokens, from, slot2);
        moe_products<2, MT>(stage, slot2, some, acc);
      }
      moe_settle();
      u += KW;
      if (last) {
        finish(job, n, acc);
        if (!more_jobs) return;
        advance(job);
        ++n;
        u = share;
        tokens = next_tokens;
        first = moe_slots<NS, MT>(tokens, 0, slot);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[r][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    }
  }
}

template <int DT>
__device__ __forceinline__ void moe_store(void* out, int64_t to, const f32x4& v) {
  if constexpr (DT == kF32)
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + to) = v;
  else
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(out) + to) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
}

// Waves of a workgroup of the down products: what has room in LDS, and in registers.
constexpr int down_waves(int MT, int NS, int PH) {
  return NS > 8 && PH == 2 ? 6 : MT > 2 || NS > 8 || (MT == 2 && PH == 2) ? 8 : 12;
}
constexpr int kDownAhead = 3;  // (4: the same within 1 %)

// 16 columns of the output for all tokens: a workgroup, its waves the units of all
// chosen experts' rows, in turn, so that what they read at a time lies together;
// or, where an expert's units are few, a run of them each, so that they do not
// change experts with every unit (16 tokens bfloat16, runs against turns: 8 of 64
// experts of 2048 x 1024, 4 units each, 103 against 121 us of the whole layer; 4 of
// 16 of 2048 x 4096, 16 units, 120 against 125; 4 of 32 of 2048 x 5760, 23 units,
// 232 against 229, and there the rule ends).  Weights are on their way three units
// ahead, columns one, over the experts' ends.
template <int DT, int MT, int NS, int PH, int ROWS>
__global__ void __launch_bounds__(64 * down_waves(MT, NS, PH)) moe_down_kernel(MoeLayer a) {
  constexpr int WAVES = down_waves(MT, NS, PH);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ uint16_t rows_of[WAVES][2][kMoeMaxTokens];  // of this expert and the next one: its pairs
  const MoeLists lists = moe_lists_at(a, lds);
  uint8_t* const mine = lds + 4 * moe_list_words(a.tokens * a.top_k, a.experts);
  for (int p = threadIdx.x; p < a.tokens * a.top_k; p += 64 * WAVES) {
    lists.exponent[p] = moe_exponent(a.h_top[p]);
    lists.weight[p] = a.expert_weights[p];
  }
  moe_lists<false>(a, lists, nullptr);
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int units = (a.f + kUnit - 1) / kUnit, all = __builtin_amdgcn_readfirstlane(*lists.count) * units;
  // this wave's units: begin, begin + stride ..
  const bool runs = units < 2 * WAVES;
  const int each = __builtin_amdgcn_readfirstlane((all + WAVES - 1) / WAVES);
  const int stride = runs ? 1 : WAVES, begin_at = runs ? wave * each : wave, end_at = runs ? min(all, begin_at + each) : all;
  f32x4 total[MT] = {};
  if (begin_at < end_at) {
    auto expert_of = [&](int which) { return __builtin_amdgcn_readfirstlane(lists.list[which]); };
    int which = __builtin_amdgcn_readfirstlane(begin_at / units), u = begin_at - which * units;
    // the unit whose weights are loaded next, of all and of its expert; the last one again when all are
    int w_next = begin_at, w_which = which, w_unit = u;
    int64_t w_row = (int64_t)expert_of(which) * a.k + n0;
    auto load_weights = [&](MoeWeights<1>& to) {
      moe_load<1, ROWS>(to, a.down_codes, a.down_scales, {w_row}, a.f, w_unit);
      if (w_next + stride < end_at) {
        w_next += stride;
        w_unit += stride;
        if (w_unit >= units) {
          do {
            w_unit -= units;
            ++w_which;
          } while (w_unit >= units);
          w_row = (int64_t)expert_of(w_which) * a.k + n0;
        }
      }
    };
    MoeWeights<1> w[kDownAhead];
    load_weights(w[0]);

    using Stage = MoeStage<1, NS, PH>;
    Stage& stage = reinterpret_cast<Stage*>(mine)[wave];
    stage.clear();
    MoeHidden<NS> hidden;
    MoeTokens tokens, next_tokens;
    int slot[MT], row = 0, exponent = 0, next_exponent = 0, n = 0;  // lane i: slot i's pair and its power of two
    uint32_t first = 0u;
    f32x4 acc[1][MT];
    int left = __builtin_amdgcn_readfirstlane((end_at - begin_at + stride - 1) / stride);
    auto place = [&](const MoeTokens& k, const uint16_t* row_of, int from, int& to, int& e) {
      to = row_of[min(from + (lane & 15), k.count - 1)];
      e = lists.exponent[to];
    };
    auto open = [&](int expert, MoeTokens& k, uint16_t* row_of, int& e) {
      const int pair = moe_pair(a, lists, lane, expert);
      k = moe_tokens(pair);
      moe_settle();
      if (pair >= 0) row_of[moe_rank(k, lane)] = (uint16_t)pair;
      moe_settle();
      place(k, row_of, 0, row, e);
    };
    auto begin = [&]() {
      first = moe_slots<NS, MT>(tokens, 0, slot);
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[0][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    };
    auto end = [&]() {  // adds the sums of expert `which`
      const int expert = expert_of(which);
      const MoeFactor factor = moe_factor(a.down_global, expert);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int t = 16 * m + (lane & 15);
        if (!(tokens.live >> t & 1u)) continue;
        const int p = rows_of[wave][n & 1][moe_rank(tokens, t)];
        float weight = 0.0f;
        for (int q = p; q < (t + 1) * a.top_k; ++q)  // an expert may stand twice among a token's
          if (lists.idx[q] == expert) weight += lists.weight[q];
        weight *= factor.by;
        const int e = lists.exponent[p] + factor.exponent;
#pragma unroll
        for (int i = 0; i < 4; ++i) total[m][i] += weight * __builtin_ldexpf(acc[0][m][i], e);
      }
    };
    open(expert_of(which), tokens, rows_of[wave][0], exponent);
    moe_load(hidden, a.hidden, row, a.f, u);
#pragma unroll
    for (int j = 1; j < kDownAhead; ++j) load_weights(w[j]);
    begin();
    for (;;) {
#pragma unroll
      for (int j = 0; j < kDownAhead; ++j) {
        moe_stage<ROWS>(stage, w[j], a.f, u);
        moe_stage(stage, hidden, exponent, tokens.count);
        moe_settle();
        const int now = u;
        const bool more = --left > 0;
        int next = which;
        if (more) {
          u += stride;
          while (u >= units) {
            u -= units;
            ++next;
          }
          if (next != which) open(expert_of(next), next_tokens, rows_of[wave][(n + 1) & 1], next_exponent);
        }
        moe_load(hidden, a.hidden, row, a.f, u);
        load_weights(w[j]);
        moe_products<1, MT>(stage, slot, first, acc);
        for (int from = NS; from < tokens.count; from += NS) {  // more tokens than have room
          MoeHidden<NS> some;
          int row2, e2, slot2[MT];
          place(tokens, rows_of[wave][n & 1], from, row2, e2);
          moe_load(some, a.hidden, row2, a.f, now);
          moe_settle();
          moe_stage(stage, some, e2, tokens.count - from);
          moe_settle();
          const uint32_t tiles = moe_slots<NS, MT>(tokens, from, slot2);
          moe_products<1, MT>(stage, slot2, tiles, acc);
        }
        moe_settle();
        if (!more || next != which) end();
        if (!more) goto done;
        if (next != which) {
          which = next;
          ++n;
          tokens = next_tokens;
          exponent = next_exponent;
          begin();
        }
      }
    }
  done:;
  }
  __syncthreads();
  f32x4* part = reinterpret_cast<f32x4*>(mine);  // [wave][MT][64]
#pragma unroll
  for (int m = 0; m < MT; ++m) part[(wave * MT + m) * 64 + lane] = total[m];
  __syncthreads();
  for (int m = wave; m < MT; m += WAVES) {
    const int t = 16 * m + (lane & 15);
    f32x4 v = part[m * 64 + lane];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v += part[(i * MT + m) * 64 + lane];
    if (t >= a.tokens) continue;
    moe_store<DT>(a.out, (int64_t)t * a.k + n0 + 4 * (lane >> 4), v);
  }
}

// ----------------------------------------------------------------- launches

struct MoePlan {
  size_t logits, x_exponent, h_top, x, h, bytes;  // offsets in the workspace
};
MoePlan moe_plan(int64_t tokens, int64_t top_k, int64_t experts, int64_t k, int64_t f, int dt) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  MoePlan p;
  p.logits = 0;
  p.x_exponent = up((size_t)tokens * experts * 8);
  p.h_top = p.x_exponent + up((size_t)tokens * 4);
  p.x = p.h_top + up((size_t)tokens * top_k * 4);
  p.h = p.x + up((size_t)moe_x_pieces(dt) * tokens * k * 2);
  p.bytes = p.h + up((size_t)tokens * top_k * f * 4);
  return p;
}

// Lets `kernel` have more than 64 KB of dynamic LDS; once per device (or twice,
// by two threads at once).
template <typename K>
hipError_t moe_allow_lds(K* kernel, size_t bytes, std::atomic<bool> (&set)[64]) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  if (dev < 0 || dev >= 64 || set[dev]) return hipSuccess;
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == hipSuccess) set[dev] = true;
  return e;
}

size_t moe_lists_bytes(const MoeLayer& a) { return 4 * (size_t)moe_list_words(a.tokens * a.top_k, a.experts); }
constexpr size_t moe_most_list_bytes(int MT) { return 4 * (size_t)moe_list_words(16 * MT * kMoeMaxTopK, kMoeMaxExperts); }

template <int DT, int MT, int NS, int KW, int ROWS, bool CHOOSE>
hipError_t launch_up(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT) > 0 ? moe_x_pieces(DT) : 1;
  constexpr size_t bytes = up_bytes<MT, NS, PX, KW>();
  static_assert(bytes >= kChooseMost * 8, "the order of the logits fits");
  static std::atomic<bool> set[64];
  if (const hipError_t e = moe_allow_lds(&moe_up_kernel<MT, NS, PX, KW, ROWS, CHOOSE>, bytes + moe_most_list_bytes(MT), set);
      e != hipSuccess)
    return e;
  const int pairs = a.tokens * a.top_k, most = pairs < a.experts ? pairs : a.experts;
  const uint16_t* x = moe_x_pieces(DT) > 0 ? a.x_pieces : reinterpret_cast<const uint16_t*>(a.x);
  // as many workgroups as run at once
  const int jobs = (most * (a.f / 16) + kUpWaves / KW - 1) / (kUpWaves / KW);
  const int resident = device_cu_count() * up_groups_a_cu<MT, NS, PX, KW>(moe_lists_bytes(a));
  const int groups = (jobs < resident ? jobs : resident) + (CHOOSE ? 1 : 0);
  moe_up_kernel<MT, NS, PX, KW, ROWS, CHOOSE><<<groups, 64 * kUpWaves, bytes + moe_lists_bytes(a), s>>>(a, x);
  return hipGetLastError();
}

template <int DT, int MT, int NS, int ROWS>
hipError_t launch_down(const MoeLayer& a, hipStream_t s) {
  constexpr int PH = moe_h_pieces(DT), WAVES = down_waves(MT, NS, PH);
  constexpr size_t staged = WAVES * sizeof(MoeStage<1, NS, PH>), joined = WAVES * MT * 1024;
  constexpr size_t bytes = staged > joined ? staged : joined;
  static_assert(bytes + moe_most_list_bytes(MT) + WAVES * kMoeMaxTokens * 4 + 16 <= 160 * 1024, "LDS");
  static std::atomic<bool> set[64];
  if (const hipError_t e = moe_allow_lds(&moe_down_kernel<DT, MT, NS, PH, ROWS>, bytes + moe_most_list_bytes(MT), set);
      e != hipSuccess)
    return e;
  moe_down_kernel<DT, MT, NS, PH, ROWS><<<(unsigned)(a.k / 16), 64 * WAVES, bytes + moe_lists_bytes(a), s>>>(a);
  return hipGetLastError();
}

template <int DT, int MT, int NS>
hipError_t launch_products(const MoeLayer& a, hipStream_t s) {
  auto rows = [](int inner, const uint8_t* scales) {
    return inner < 64 ? kShort : inner % 64 == 0 && (reinterpret_cast<uintptr_t>(scales) & 3) == 0 ? kWhole : kAny;
  };
  const int up = rows(a.k, a.up_scales), down = rows(a.f, a.down_scales);
  const bool inside = MT <= 2 && a.router && moe_choose_inside(a.tokens, a.experts);  // (most tokens of MT 4 pass it)
  // Up to three units are one wave's, without a join: 20 tokens float16, 3 of 9
  // experts of 128 x 1376 58 us against 65, of 768 x 1376 60 against 65.
  const bool alone = a.k <= 3 * kUnit;
  hipError_t e;
#define MOE_UP(CHOOSE)                                                                                     \
  do {                                                                                                     \
    if (up == kShort) e = launch_up<DT, MT, 8, 1, kShort, CHOOSE>(a, s);                                   \
    else if (alone) e = up == kWhole ? launch_up<DT, MT, NS, 1, kWhole, CHOOSE>(a, s)                      \
                                     : launch_up<DT, MT, NS, 1, kAny, CHOOSE>(a, s);                       \
    else e = up == kWhole ? launch_up<DT, MT, NS, kUpWaves, kWhole, CHOOSE>(a, s)                          \
                          : launch_up<DT, MT, NS, kUpWaves, kAny, CHOOSE>(a, s);                           \
  } while (0)
  if constexpr (MT <= 2) {
    if (inside) MOE_UP(true);
  }
  if (!inside) MOE_UP(false);
#undef MOE_UP
  if (e != hipSuccess) return e;
  if (down == kShort) return launch_down<DT, MT, 8, kShort>(a, s);
  if constexpr (MT == 1) {
    // Fewer columns to load and convert: 1 token, 2 of 8 of 4096 x 14336 17.0 us for
    // 21.1 with 8, 2 tokens, 8 of 64 of 2048 x 1024 12.6 for 13.9.
    if (a.tokens <= 2) return down == kWhole ? launch_down<DT, 1, 2, kWhole>(a, s) : launch_down<DT, 1, 2, kAny>(a, s);
  }
  return down == kWhole ? launch_down<DT, MT, NS, kWhole>(a, s) : launch_down<DT, MT, NS, kAny>(a, s);
}

template <int DT>
hipError_t launch(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT);
  const unsigned cuts = (unsigned)a.tokens;
  // Few logits: a workgroup each, for the latency (2 tokens of 64 experts: 2.7 us, of
  // four tokens 4.0; from 4 tokens on the same); many: four tokens each, so that an
  // expert's row is read less often.
  if (!a.router) {
    moe_logits_kernel<DT, PX, 1><<<cuts, 256, 0, s>>>(a, 0);
  } else if (a.tokens * a.experts <= 1024) {
    const int routers = a.tokens * a.experts;
    moe_logits_kernel<DT, PX, 1><<<routers + cuts, 256, 0, s>>>(a, routers);
  } else {
    const int routers = (a.tokens + 3) / 4 * a.experts;
    moe_logits_kernel<DT, PX, 4><<<routers + cuts, 256, 0, s>>>(a, routers);
  }
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (a.router && !(a.tokens <= 32 && moe_choose_inside(a.tokens, a.experts))) {
    moe_choose_kernel<<<(unsigned)a.tokens, 256, 0, s>>>(a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  // Columns at a time, about as many as an expert has tokens (an expert's weights
  // are staged again for those that are left): 16 where there are more than 5 an
  // expert.  32 tokens, 2 of 8 of 4096 x 14336 bfloat16: 300 us, with 8 at a time
  // 345.  They cost registers, and with them a workgroup a CU: 16 tokens there, 4 an
  // expert, 210 us with 8.  (Two pieces and more than 32 tokens would spill with 16.)
  const bool wide = a.tokens > 8 && 5 * a.experts < a.tokens * a.top_k;
  if (a.tokens <= 16) return wide ? launch_products<DT, 1, 16>(a, s) : launch_products<DT, 1, 8>(a, s);
  if (a.tokens <= 32) return wide ? launch_products<DT, 2, 16>(a, s) : launch_products<DT, 2, 8>(a, s);
  return wide && DT == kBF16 ? launch_products<DT, 4, DT == kBF16 ? 16 : 8>(a, s) : launch_products<DT, 4, 8>(a, s);
}

}  // namespace

size_t moe_workspace(int64_t tokens, int64_t top_k, int64_t experts, int64_t k, int64_t f, int dt) {
  return moe_plan(tokens, top_k, experts, k, f, dt).bytes;
}

hipError_t launch_moe(MoeLayer a, int dt, void* workspace, hipStream_t s) {
  const MoePlan p = moe_plan(a.tokens, a.top_k, a.experts, a.k, a.f, dt);
  uint8_t* w = reinterpret_cast<uint8_t*>(workspace);
  a.logits = reinterpret_cast<double*>(w + p.logits);
  a.x_exponent = moe_x_pieces(dt) > 0 ? reinterpret_cast<int*>(w + p.x_exponent) : nullptr;
  a.h_top = reinterpret_cast<uint32_t*>(w + p.h_top);
  a.x_pieces = reinterpret_cast<uint16_t*>(w + p.x);
  a.hidden = reinterpret_cast<float*>(w + p.h);
  return dt == kF32 ? launch<kF32>(a, s) : dt == kF16 ? launch<kF16>(a, s) : launch<kBF16>(a, s);
}

}  // namespace nvfp4
