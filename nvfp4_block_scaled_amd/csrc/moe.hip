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
#include <atomic>

#include "layer_internal.h"
#include "nvfp4_device.h"

namespace nvfp4 {

namespace {

typedef uint32_t u32x4_8 __attribute__((ext_vector_type(4), aligned(8)));

constexpr int kUnit = 256;  // inner values of a row that a wave takes at a time: 64 a lane

// ----------------------------------------------------------------- pieces

// Pieces of x (0: it is used as it lies) and of h.
constexpr int moe_x_pieces(int dt) { return dt == kF32 ? 2 : dt == kF16 ? 0 : 1; }
constexpr int moe_h_pieces(int dt) { return dt == kBF16 ? 1 : 2; }

// e such that 2^-e brings a row of largest magnitude `top` (its bits) to 2^13 ..
// 2^14.  Rows of zeros, infinities and NaN stay as they are.
__device__ __forceinline__ int moe_exponent(uint32_t top) {
  const int field = (int)(top >> 23);
  return top == 0u || field == 255 ? 0 : field - 140;
}
// Four values times 2^-e as P float16 pieces, two to a dword.
template <int P>
__device__ __forceinline__ void moe_pieces(const float (&v)[4], int e, u32x2 (&p)[P]) {
  float y[4];
  f16x2 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = __builtin_ldexpf(v[i], -e);
#pragma unroll
  for (int j = 0; j < P; ++j) {
    a = f16x2{(_Float16)y[0], (_Float16)y[1]};
    b = f16x2{(_Float16)y[2], (_Float16)y[3]};
    p[j] = u32x2{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b)};
    y[0] -= (float)a.x;
    y[1] -= (float)a.y;
    y[2] -= (float)b.x;
    y[3] -= (float)b.y;
  }
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
// hundred steps a thread.
constexpr bool moe_choose_inside(int tokens, int experts) {
  const int all = tokens * experts;
  return all <= 1024 && (all + 255) / 256 * experts <= 320;
}

// ----------------------------------------------------------------- which experts

// The chosen experts of all tokens in LDS: each pair's (-1: none), and the list
// of the different ones in the order of their first pairs.
struct MoeLists {
  int *idx, *first, *list;
  int* count;
};
constexpr int moe_list_words(int pairs, int experts) { return (pairs + 2 * experts + 1 + 3) / 4 * 4; }
__device__ __forceinline__ MoeLists moe_lists_at(const MoeLayer& a, void* lds) {
  int* w = reinterpret_cast<int*>(lds);
  const int pairs = a.tokens * a.top_k;
  return MoeLists{w, w + pairs, w + pairs + a.experts, w + pairs + 2 * a.experts};
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
// other wave waits for it; chunks of 16 bytes lie at their number xor the row's,
// which spreads both the writes and the reads over the banks.  The next unit's
// loads are under way meanwhile.

constexpr int kSlots = 8;  // columns in LDS at a time

// In LDS, of one wave.
template <int NR, int P>
struct MoeStage {
  u32x4 codes[NR][16][8];       // row, chunk of 32 values
  uint32_t scales[NR][16][4];   // row, 4 groups of 16
  u32x4 columns[P][kSlots][32]; // column, chunk of 8 values
};

// One unit's weights on their way: lane l has chunk l % 8 of rows l / 8 and l / 8
// + 8, and the scales of row l / 4, groups 4 (l % 4) ...  WHOLE: rows are whole
// 64s and scales whole dwords.  Past the end of a row scales are 0, and so are its weights.
template <int NR>
struct MoeWeights {
  u32x4 c[NR][2];
  uint32_t s[NR];
};
template <int NR, bool WHOLE>
__device__ __forceinline__ void moe_load(MoeWeights<NR>& w, const uint8_t* codes, const uint8_t* scales, const int64_t (&row0)[NR],
                                         int inner, int unit) {
  const int lane = threadIdx.x & 63;
  const int from = unit * kUnit + 32 * (lane & 7), group = unit * (kUnit / 16) + 4 * (lane & 3), groups = inner / 16;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint8_t* p = codes + (row0[r] + (lane >> 3) + 8 * d) * (inner / 2) + from / 2;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (WHOLE ? from < inner : from + 32 <= inner) {
        v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_8*>(p));
      } else if (!WHOLE && from < inner) {
        const u32x2 half = *reinterpret_cast<const u32x2*>(p);
        v.x = half.x;
        v.y = half.y;
      }
      w.c[r][d] = v;
    }
    const uint8_t* p = scales + (row0[r] + (lane >> 2)) * groups + group;
    w.s[r] = 0u;
    if constexpr (WHOLE) {
      if (group < groups) w.s[r] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (group + i < groups) w.s[r] |= (uint32_t)p[i] << (8 * i);
    }
  }
}
template <int NR, int P>
__device__ __forceinline__ void moe_stage(MoeStage<NR, P>& l, const MoeWeights<NR>& w) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
#pragma unroll
    for (int d = 0; d < 2; ++d) l.codes[r][(lane >> 3) + 8 * d][(lane & 7) ^ (lane >> 3)] = w.c[r][d];
    l.scales[r][lane >> 2][lane & 3] = w.s[r];
  }
}

// kSlots columns of x pieces of a unit on their way: lane l has chunk l % 32 of
// columns l / 32, l / 32 + 2 ..
template <int P>
struct MoeColumns {
  u32x4 v[P][kSlots / 2];
};
// `at`: where this lane's columns begin; `count` of them are there, of `inner`
// values, a piece `plane` behind the other.
template <int P>
__device__ __forceinline__ void moe_load(MoeColumns<P>& x, const uint16_t* base, int64_t plane, const int (&at)[kSlots / 2], int count,
                                         int inner, int unit) {
  const int from = unit * kUnit + 8 * (threadIdx.x & 31);
  const bool there = from < inner;
#pragma unroll
  for (int i = 0; i < kSlots / 2; ++i)
    if (2 * i < count) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        x.v[p][i] = u32x4{0u, 0u, 0u, 0u};
        if (there) x.v[p][i] = *reinterpret_cast<const u32x4*>(base + p * plane + at[i] + from);
      }
    }
}
template <int NR, int P>
__device__ __forceinline__ void moe_stage(MoeStage<NR, P>& l, const MoeColumns<P>& x, int count) {
  const int lane = threadIdx.x & 63, half = lane >> 5;
#pragma unroll
  for (int i = 0; i < kSlots / 2; ++i)
    if (2 * i < count) {
#pragma unroll
      for (int p = 0; p < P; ++p) l.columns[p][2 * i + half][(lane & 31) ^ (2 * i + half)] = x.v[p][i];
    }
}

// kSlots columns of h on their way, float32: lane l has values 4 l .. 4 l + 3 of
// each.  They become pieces when they are staged.  row: slot i's pair, in lane i.
struct MoeHidden {
  f32x4 v[kSlots];
};
__device__ __forceinline__ void moe_load(MoeHidden& x, const float* base, int row, int count, int inner, int unit) {
  const int from = unit * kUnit + 4 * (threadIdx.x & 63);
  const bool there = from < inner;
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (i < count) {
      x.v[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      const float* p = base + (int64_t)__builtin_amdgcn_readlane(row, i) * inner;
      if (there) x.v[i] = *reinterpret_cast<const f32x4*>(p + from);
    }
}
template <int P>
__device__ __forceinline__ void moe_stage(MoeStage<1, P>& l, const MoeHidden& x, int exponent, int count) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if (i < count) {
      u32x2 piece[P];
      moe_pieces<P>({x.v[i][0], x.v[i][1], x.v[i][2], x.v[i][3]}, __builtin_amdgcn_readlane(exponent, i), piece);
#pragma unroll
      for (int p = 0; p < P; ++p) reinterpret_cast<u32x2*>(&l.columns[p][i][(lane >> 1) ^ i])[lane & 1] = piece[p];
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
// those staged, or -1: it meets zeros.  tiles: which tiles have any.
template <int NR, int MT, int P>
__device__ __forceinline__ void moe_products(const MoeStage<NR, P>& l, const int (&slot)[MT], uint32_t tiles,
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
    for (int j = 0; j < 2; ++j) codes[r][j] = l.codes[r][row][(2 * quarter + j) ^ (row & 7)];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f16x8 a[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) a[r] = moe_decode8(codes[r][i >> 2][i & 3], (i & 2) ? scale[r][i >> 2].y : scale[r][i >> 2].x);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (MT > 1 && !(tiles >> m & 1u)) continue;
#pragma unroll
      for (int p = P - 1; p >= 0; --p) {  // the small pieces first
        const int at = max(slot[m], 0);
        u32x4 v = l.columns[p][at][(8 * quarter + i) ^ at];
        if (slot[m] < 0) v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < NR; ++r)
          acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a[r], __builtin_bit_cast(f16x8, v), acc[r][m], 0, 0, 0);
      }
    }
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
template <int MT>
__device__ __forceinline__ uint32_t moe_slots(const MoeTokens& k, int from, int (&slot)[MT]) {
  uint32_t tiles = 0u;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = 16 * m + (threadIdx.x & 15), at = moe_rank(k, t) - from;
    slot[m] = (k.live >> t & 1u) && at >= 0 && at < kSlots ? at : -1;
    tiles |= __any(slot[m] >= 0) ? 1u << m : 0u;
  }
  return tiles;
}

constexpr int kUpWaves = 4;

// 16 gate rows and the 16 up rows that go with them, of one expert: a workgroup,
// its waves each a share of the inner values.  CHOOSE: moe_choose_inside, and the
// last workgroup writes the choice.  PX: pieces of x here (1 or 2).
template <int MT, int PX, bool WHOLE, bool CHOOSE>
__global__ void __launch_bounds__(64 * kUpWaves, MT * PX == 1 ? 4 : MT * PX == 2 ? 3 : 2) moe_up_kernel(MoeLayer a, const uint16_t* x) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int row_of[kMoeMaxTokens];  // of the expert's tokens
  const MoeLists lists = moe_lists_at(a, lds);
  uint8_t* const mine = lds + 4 * moe_list_words(a.tokens * a.top_k, a.experts);
  moe_lists<CHOOSE>(a, lists, reinterpret_cast<uint64_t*>(mine));
  if (CHOOSE && blockIdx.x == gridDim.x - 1) {
    moe_weigh(a, 0, a.tokens, lists.idx);
    return;
  }
  const int tiles = a.f / 16;
  const int which = blockIdx.x / tiles, f0 = (blockIdx.x - which * tiles) * 16;
  if (which >= *lists.count) return;
  const int expert = __builtin_amdgcn_readfirstlane(lists.list[which]);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int units = (a.k + kUnit - 1) / kUnit;
  const int64_t row0[2] = {(int64_t)expert * 2 * a.f + f0, (int64_t)expert * 2 * a.f + a.f + f0};
  MoeWeights<2> w;
  if (wave < units) moe_load<2, WHOLE>(w, a.up_codes, a.up_scales, row0, a.k, wave);
  const int my_pair = moe_pair(a, lists, lane, expert);
  const MoeTokens tokens = moe_tokens(my_pair);
  if (wave == 0 && my_pair >= 0) row_of[moe_rank(tokens, lane)] = lane;
  __syncthreads();
  MoeStage<2, PX>& stage = reinterpret_cast<MoeStage<2, PX>*>(mine)[wave];
  f32x4 acc[2][MT] = {};
  MoeColumns<PX> columns;
  const int64_t plane = (int64_t)a.tokens * a.k;
  auto place = [&](int from, int(&at)[kSlots / 2]) {
#pragma unroll
    for (int i = 0; i < kSlots / 2; ++i) at[i] = row_of[min(from + 2 * i + (lane >> 5), tokens.count - 1)] * a.k;
  };
  int at[kSlots / 2], slot[MT];
  place(0, at);
  const uint32_t first = moe_slots<MT>(tokens, 0, slot);
  if (wave < units) moe_load<PX>(columns, x, plane, at, tokens.count, a.k, wave);
  for (int u = wave; u < units; u += kUpWaves) {
    moe_stage<2, PX>(stage, w);
    moe_stage<2, PX>(stage, columns, tokens.count);
    moe_settle();
    if (u + kUpWaves < units) {
      moe_load<PX>(columns, x, plane, at, tokens.count, a.k, u + kUpWaves);
      moe_load<2, WHOLE>(w, a.up_codes, a.up_scales, row0, a.k, u + kUpWaves);
    }
    moe_products<2, MT, PX>(stage, slot, first, acc);
    for (int from = kSlots; from < tokens.count; from += kSlots) {  // more tokens than have room
      MoeColumns<PX> more;
      int at2[kSlots / 2], slot2[MT];
      place(from, at2);
      moe_load<PX>(more, x, plane, at2, tokens.count - from, a.k, u);
      moe_settle();
      moe_stage<2, PX>(stage, more, tokens.count - from);
      moe_settle();
      const uint32_t some = moe_slots<MT>(tokens, from, slot2);
      moe_products<2, MT, PX>(stage, slot2, some, acc);
    }
    moe_settle();
  }
  __syncthreads();
  f32x4* part = reinterpret_cast<f32x4*>(mine);  // [wave][2][MT][64]
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[((wave * 2 + r) * MT + m) * 64 + lane] = acc[r][m];
  __syncthreads();
  const float factor = global_decode(a.up_global ? a.up_global + expert : nullptr);
  for (int m = wave; m < MT; m += kUpWaves) {
    const int t = 16 * m + (lane & 15), p = moe_pair(a, lists, t, expert);
    const int e = a.x_exponent && t < a.tokens ? a.x_exponent[t] : 0;
    f32x4 g = part[m * 64 + lane], v = part[(MT + m) * 64 + lane];
#pragma unroll
    for (int i = 1; i < kUpWaves; ++i) {
      g += part[((i * 2) * MT + m) * 64 + lane];
      v += part[((i * 2 + 1) * MT + m) * 64 + lane];
    }
    f32x4 h;
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x1 = __builtin_ldexpf(g[i] * factor, e), x2 = __builtin_ldexpf(v[i] * factor, e);
      h[i] = x1 / (1.0f + expf(-x1)) * x2;
      top = max(top, __float_as_uint(h[i]) & 0x7FFFFFFFu);
    }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    if (p < 0) continue;
    *reinterpret_cast<f32x4*>(a.hidden + (int64_t)p * a.f + f0 + 4 * (lane >> 4)) = h;
    if (lane < 16) atomicMax(a.h_top + p, top);  // (in any order the same)
  }
}

// Waves of a workgroup of the down products: what has room in LDS, and in registers.
constexpr int down_waves(int MT, int PH) { return MT > 2 || (MT == 2 && PH == 2) ? 8 : 12; }

// 16 columns of the output for all tokens: a workgroup, its waves in turn the
// units of all chosen experts' rows: what they read at a time lies together.
template <int DT, int MT, int PH, bool WHOLE>
__global__ void __launch_bounds__(64 * down_waves(MT, PH)) moe_down_kernel(MoeLayer a) {
  constexpr int WAVES = down_waves(MT, PH);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int rows_of[WAVES][kMoeMaxTokens];
  const MoeLists lists = moe_lists_at(a, lds);
  uint8_t* const mine = lds + 4 * moe_list_words(a.tokens * a.top_k, a.experts);
  moe_lists<false>(a, lists, nullptr);
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int units = (a.f + kUnit - 1) / kUnit, all = *lists.count * units;
  int* const row_of = rows_of[wave];
  f32x4 total[MT] = {};
  if (wave < all) {
    MoeWeights<1> w[2];
    // the unit whose weights are loaded next: of all, and of its expert
    int next = wave, next_which = wave / units, next_u = wave - next_which * units;
    int64_t next_row[1];
    auto seek = [&]() { next_row[0] = (int64_t)__builtin_amdgcn_readfirstlane(lists.list[next_which]) * a.k + n0; };
    auto load = [&](MoeWeights<1>& x) {
      if (next >= all) return;
      moe_load<1, WHOLE>(x, a.down_codes, a.down_scales, next_row, a.f, next_u);
      next += WAVES;
      next_u += WAVES;
      if (next_u >= units && next < all) {
        do {
          next_u -= units;
          ++next_which;
        } while (next_u >= units);
        seek();
      }
    };
    seek();
    load(w[0]);

    MoeStage<1, PH>& stage = reinterpret_cast<MoeStage<1, PH>*>(mine)[wave];
    MoeHidden hidden;
    MoeTokens tokens;
    int slot[MT], row = 0, exponent = 0;  // lane i: slot i's pair and its power of two
    uint32_t first = 0u;
    float weight[MT];
    f32x4 acc[1][MT];
    int which = wave / units, u = wave - which * units, left = (all - wave + WAVES - 1) / WAVES;
    auto place = [&](int from, int& to, int& e) {
      to = row_of[min(from + (lane & (kSlots - 1)), tokens.count - 1)];
      e = moe_exponent(a.h_top[to]);
    };
    auto begin = [&]() {  // the columns of expert `which`
      const int expert = __builtin_amdgcn_readfirstlane(lists.list[which]);
      const int pair = moe_pair(a, lists, lane, expert);
      tokens = moe_tokens(pair);
      moe_settle();
      if (pair >= 0) row_of[moe_rank(tokens, lane)] = pair;
      moe_settle();
      place(0, row, exponent);
      moe_load(hidden, a.hidden, row, tokens.count, a.f, u);
      first = moe_slots<MT>(tokens, 0, slot);
      const float factor = global_decode(a.down_global ? a.down_global + expert : nullptr);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int t = 16 * m + (lane & 15), p = moe_pair(a, lists, t, expert);
        weight[m] = 0.0f;
        if (p >= 0)  // an expert may stand twice among a token's
          for (int q = p; q < (t + 1) * a.top_k; ++q)
            if (lists.idx[q] == expert) weight[m] += a.expert_weights[q];
        weight[m] *= factor;
        acc[0][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    };
    auto end = [&]() {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int t = 16 * m + (lane & 15);
        const bool live = tokens.live >> t & 1u;
        const int e = live ? moe_exponent(a.h_top[row_of[moe_rank(tokens, t)]]) : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          total[m][i] = live ? total[m][i] + weight[m] * __builtin_ldexpf(acc[0][m][i], e) : total[m][i];
      }
    };
    begin();
    load(w[1]);
    while (left > 0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (left <= 0) break;
        moe_stage<1, PH>(stage, w[j]);
        moe_stage<PH>(stage, hidden, exponent, tokens.count);
        moe_settle();
        const int now = u;
        --left;
        u += WAVES;
        const bool over = u >= units;
        if (!over && left > 0) moe_load(hidden, a.hidden, row, tokens.count, a.f, u);
        load(w[j]);
        moe_products<1, MT, PH>(stage, slot, first, acc);
        for (int from = kSlots; from < tokens.count; from += kSlots) {  // more tokens than have room
          MoeHidden more;
          int row2, e2, slot2[MT];
          place(from, row2, e2);
          moe_load(more, a.hidden, row2, tokens.count - from, a.f, now);
          moe_settle();
          moe_stage<PH>(stage, more, e2, tokens.count - from);
          moe_settle();
          const uint32_t some = moe_slots<MT>(tokens, from, slot2);
          moe_products<1, MT, PH>(stage, slot2, some, acc);
        }
        moe_settle();
        if (over && left > 0) {
          end();
          do {
            u -= units;
            ++which;
          } while (u >= units);
          begin();
        }
      }
    }
    end();
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
    const int64_t to = (int64_t)t * a.k + n0 + 4 * (lane >> 4);
    if constexpr (DT == kF32)
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + to) = v;
    else
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + to) = u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
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
constexpr size_t kMoeMaxListBytes = 4 * moe_list_words(kMoeMaxPairs, kMoeMaxExperts);

template <int DT, int MT, bool WHOLE, bool CHOOSE>
hipError_t launch_up(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT) > 0 ? moe_x_pieces(DT) : 1;
  constexpr size_t staged = kUpWaves * sizeof(MoeStage<2, PX>), joined = kUpWaves * 2 * MT * 1024;
  constexpr size_t bytes = staged > joined ? staged : joined;
  static_assert(bytes >= 1024 * 8, "the order of the logits fits");
  static std::atomic<bool> set[64];
  if (const hipError_t e = moe_allow_lds(&moe_up_kernel<MT, PX, WHOLE, CHOOSE>, bytes + kMoeMaxListBytes, set); e != hipSuccess)
    return e;
  const int pairs = a.tokens * a.top_k, most = pairs < a.experts ? pairs : a.experts;
  const uint16_t* x = moe_x_pieces(DT) > 0 ? a.x_pieces : reinterpret_cast<const uint16_t*>(a.x);
  moe_up_kernel<MT, PX, WHOLE, CHOOSE>
      <<<(unsigned)(most * (a.f / 16) + (CHOOSE ? 1 : 0)), 64 * kUpWaves, bytes + moe_lists_bytes(a), s>>>(a, x);
  return hipGetLastError();
}

template <int DT, int MT, bool WHOLE>
hipError_t launch_down(const MoeLayer& a, hipStream_t s) {
  constexpr int PH = moe_h_pieces(DT), WAVES = down_waves(MT, PH);
  constexpr size_t staged = WAVES * sizeof(MoeStage<1, PH>), joined = WAVES * MT * 1024;
  constexpr size_t bytes = staged > joined ? staged : joined;
  static_assert(bytes + kMoeMaxListBytes + WAVES * kMoeMaxTokens * 4 <= 160 * 1024, "LDS");
  static std::atomic<bool> set[64];
  if (const hipError_t e = moe_allow_lds(&moe_down_kernel<DT, MT, PH, WHOLE>, bytes + kMoeMaxListBytes, set); e != hipSuccess)
    return e;
  moe_down_kernel<DT, MT, PH, WHOLE><<<(unsigned)(a.k / 16), 64 * WAVES, bytes + moe_lists_bytes(a), s>>>(a);
  return hipGetLastError();
}

template <int DT, int MT>
hipError_t launch_products(const MoeLayer& a, hipStream_t s) {
  auto whole = [](int inner, const uint8_t* scales) { return inner % 64 == 0 && (reinterpret_cast<uintptr_t>(scales) & 3) == 0; };
  const bool inside = MT <= 2 && a.router && moe_choose_inside(a.tokens, a.experts);  // (most tokens of MT 4 pass it)
  hipError_t e;
  if constexpr (MT <= 2) {
    if (inside) e = whole(a.k, a.up_scales) ? launch_up<DT, MT, true, true>(a, s) : launch_up<DT, MT, false, true>(a, s);
  }
  if (!inside) e = whole(a.k, a.up_scales) ? launch_up<DT, MT, true, false>(a, s) : launch_up<DT, MT, false, false>(a, s);
  if (e != hipSuccess) return e;
  return whole(a.f, a.down_scales) ? launch_down<DT, MT, true>(a, s) : launch_down<DT, MT, false>(a, s);
}

template <int DT>
hipError_t launch(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT);
  const unsigned cuts = (unsigned)a.tokens;
  // Few logits: a workgroup each, for the latency; many: four tokens each, for the traffic.
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
  a.x_exponent = moe_x_pieces(dt) > 0 ? reinterpret_cast<int*>(w + p.x_exponent) : nullptr;
  a.h_top = reinterpret_cast<uint32_t*>(w + p.h_top);
  a.x_pieces = reinterpret_cast<uint16_t*>(w + p.x);
  a.hidden = reinterpret_cast<float*>(w + p.h);
  return dt == kF32 ? launch<kF32>(a, s) : dt == kF16 ? launch<kF16>(a, s) : launch<kBF16>(a, s);
}

}  // namespace nvfp4
