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

constexpr int moe_x_pieces(int dt) { return dt == kF32 ? 3 : dt == kF16 ? 2 : 1; }
constexpr int moe_h_pieces(int dt) { return dt == kF32 ? 3 : 2; }

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

// Where x and h lie in the workspace: per row the units of 256 values, of each
// the 8 steps of a product in turn, of a step the pieces, and of a piece the 8
// values of each quarter of a wave (values 64 quarter + 8 step .. of the unit).
// So the four quarters' loads of a column are one line's 64 bytes; as the values
// themselves lie they were four lines, and these loads took as long as the
// weights' (16 tokens, 2 of 8 experts of 4096 x 14336: down products 262 us).
__host__ __device__ constexpr int64_t moe_row(int inner, int pieces) {
  return (int64_t)((inner + kUnit - 1) / kUnit) * kUnit * pieces;
}
__device__ __forceinline__ int moe_place(int at, int pieces) {  // of the first piece of the 8 values from `at` on
  return ((at / kUnit * 8 + (at & 63) / 8) * pieces) * 32 + (at & (kUnit - 1)) / 64 * 8;
}

// ----------------------------------------------------------------- router

__device__ __forceinline__ double moe_wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Workgroups 0 .. routers - 1: logits, a workgroup an expert and TOKENS tokens, for
// which its row is loaded once.  The others lay x out in pieces.
template <int DT, int PX, int TOKENS>
__global__ void __launch_bounds__(256) moe_logits_kernel(MoeLayer a, int routers) {
  if ((int)blockIdx.x >= routers) {
    // with zeros behind the end of a row, as weights behind it are 0 and 0 times anything else might be NaN
    constexpr int PH = moe_h_pieces(DT);
    const int per_row = (int)moe_row(a.k, 1) / 8, more = (int)moe_row(a.f, 1) - a.f;
    int h = (int)(blockIdx.x - routers) * 256 + threadIdx.x;
    if (h >= a.tokens * per_row) {
      h -= a.tokens * per_row;
      if (more == 0 || h >= a.tokens * a.top_k * (more / 8)) return;
      const int p = h / (more / 8), at = a.f + 8 * (h - p * (more / 8));
#pragma unroll
      for (int j = 0; j < PH; ++j)
        *reinterpret_cast<u32x4*>(a.h_pieces + p * moe_row(a.f, PH) + moe_place(at, PH) + 32 * j) = u32x4{0u, 0u, 0u, 0u};
      return;
    }
    const int t = h / per_row, at = 8 * (h - t * per_row);
    float v[8] = {};
    if (at < a.k) load8x<DT>(a.x, (int64_t)t * (a.k / 8) + at / 8, v);
    uint16_t p[8][PX];
#pragma unroll
    for (int i = 0; i < 8; ++i) moe_pieces<PX>(v[i], p[i]);
#pragma unroll
    for (int j = 0; j < PX; ++j) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = p[2 * i][j] | (uint32_t)p[2 * i + 1][j] << 16;
      *reinterpret_cast<u32x4*>(a.x_pieces + t * moe_row(a.k, PX) + moe_place(at, PX) + 32 * j) = w;
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
  const double mine = threadIdx.x < a.top_k ? exp(l[chosen[threadIdx.x]] - top) : 0.0;
  double sum = mine;
  if (!a.normalize) {
    sum = 0.0;
    for (int i = threadIdx.x; i < a.experts; i += 256) sum += exp(l[i] - top);
  }
  sum = moe_wave_sum(sum);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  sum = (part[0] + part[1]) + (part[2] + part[3]);
  if (threadIdx.x < a.top_k) {
    a.expert_idx[t * a.top_k + threadIdx.x] = chosen[threadIdx.x];
    a.expert_weights[t * a.top_k + threadIdx.x] = (float)(mine / sum);
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

// 64 consecutive inner values of one row, as loaded: 4 groups of 16.  WHOLE: rows
// are whole 64s; then a lane past a row's end loads the row's beginning, and no
// branch stands between the loads.  Scales past the end are 0, and so are weights.
struct MoeWeights {
  uint32_t w[8], s;
};
template <bool WHOLE>
__device__ __forceinline__ MoeWeights moe_load(const uint8_t* codes, const uint8_t* scales, int64_t row, int inner, int at) {
  MoeWeights r;
  const int from = WHOLE && at >= inner ? 0 : at;
  const uint8_t* c = codes + row * (inner / 2) + from / 2;
  const uint8_t* s = scales + row * (inner / 16) + from / 16;
  if (WHOLE || at + 64 <= inner) {
    const u32x4_8 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4_8*>(c));
    const u32x4_8 y = __builtin_nontemporal_load(reinterpret_cast<const u32x4_8*>(c + 16));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.w[i] = x[i];
      r.w[4 + i] = y[i];
    }
    if constexpr (WHOLE) {
      r.s = *reinterpret_cast<const uint32_t*>(s);
      if (at >= inner) r.s = 0u;
    } else {
      __builtin_memcpy(&r.s, s, 4);
    }
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
__device__ __forceinline__ bf16x8 moe_values(const MoeWeights& r, int i) {
  return moe_decode8(r.w[i], e4m3_decode(r.s >> (8 * (i >> 1))));
}

// One unit: NR tiles of 16 rows by MT tiles of 16 tokens.  Lane l has row l % 16
// and inner values 64 (l / 16) .. of the unit on both sides.  `col`: this lane's
// column of each tile, at its quarter's values of the unit's first step.
//
// `ahead` loads the weights of a later unit.  Loads come back in the order of
// their issue, so it is called behind the unit's last loads of columns: ahead of
// them, waiting for those (in a cache) would wait for weights from memory too.
template <int NR, int MT, int P, typename F>
__device__ __forceinline__ void moe_unit(const MoeWeights (&w)[NR], const uint16_t* const (&col)[MT], int unit,
                                         f32x4 (&acc)[NR][MT], F ahead) {
  constexpr int H = MT * P <= 2 ? 8 : MT * P <= 4 ? 4 : 2;  // steps whose columns are loaded at a time
#pragma unroll
  for (int c = 0; c < 8 / H; ++c) {
    bf16x8 b[H][MT][P];
#pragma unroll
    for (int i = 0; i < H; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int p = 0; p < P; ++p)
          b[i][m][p] = *reinterpret_cast<const bf16x8*>(col[m] + (unit * 8 + c * H + i) * P * 32 + p * 32);
    __builtin_amdgcn_sched_barrier(0);
    if (c + 1 == 8 / H) {
      ahead();
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
      bf16x8 a[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) a[r] = moe_values(w[r], c * H + i);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int p = P - 1; p >= 0; --p)  // the small pieces first
#pragma unroll
          for (int r = 0; r < NR; ++r) acc[r][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[r], b[i][m][p], acc[r][m], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}
// The row that a column without a token reads instead: the first one that has
// (no line more); its sums are not looked at.  0 if none has.
__device__ __forceinline__ int moe_instead(int row, bool live) {
  const uint64_t lanes = __ballot(live);
  const int other = lanes ? __builtin_amdgcn_readlane(row, __builtin_ctzll(lanes)) : 0;
  return live ? row : other;
}

constexpr int kUpWaves = 4;

// 16 gate rows and the 16 up rows that go with them, of one expert: a workgroup,
// its waves each a share of the inner values.
template <int MT, int PX, int PH, bool WHOLE>
__global__ void __launch_bounds__(64 * kUpWaves) moe_up_kernel(MoeLayer a) {
  __shared__ MoeLists lists;
  __shared__ f32x4 part[kUpWaves][2][MT][64];
  moe_lists(a, lists);
  const int tiles = a.f / 16;
  const int which = blockIdx.x / tiles, f0 = (blockIdx.x - which * tiles) * 16;
  if (which >= lists.count) return;
  const int expert = __builtin_amdgcn_readfirstlane(lists.list[which]);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, quarter = lane >> 4;
  const int units = (a.k + kUnit - 1) / kUnit;
  const int64_t row = (int64_t)expert * 2 * a.f + f0 + col;
  MoeWeights w[2][2];
  auto load = [&](int u, MoeWeights(&x)[2]) {
    const int at = u * kUnit + 64 * quarter;
    x[0] = moe_load<WHOLE>(a.up_codes, a.up_scales, row, a.k, at);
    x[1] = moe_load<WHOLE>(a.up_codes, a.up_scales, row + a.f, a.k, at);
  };
  if (wave < units) load(wave, w[0]);
  const uint16_t* at_x[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int t = 16 * m + col;
    at_x[m] = a.x_pieces + moe_instead(t, moe_pair(a, lists, t, expert) >= 0) * moe_row(a.k, PX) + 8 * quarter;
  }
  f32x4 acc[2][MT] = {};
  for (int u = wave; u < units;) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (u >= units) break;
      moe_unit<2, MT, PX>(w[j], at_x, u, acc, [&]() {
        if (u + kUpWaves < units) load(u + kUpWaves, w[1 - j]);
      });
      u += kUpWaves;
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) part[wave][r][m][lane] = acc[r][m];
  __syncthreads();
  const float factor = global_decode(a.up_global ? a.up_global + expert : nullptr);
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
      *reinterpret_cast<u32x2*>(a.h_pieces + p * moe_row(a.f, PH) + moe_place(f0 + 4 * quarter, PH) + 32 * j + 4 * (quarter & 1)) =
          u32x2{piece[0][j] | (uint32_t)piece[1][j] << 16, piece[2][j] | (uint32_t)piece[3][j] << 16};
  }
}

constexpr int kDownWaves = 16, kDownAhead = 2;

// 16 columns of the output for all tokens: a workgroup, its waves in turn the
// units of all chosen experts' rows: what they read at a time lies together.
template <int DT, int MT, int PH, bool WHOLE>
__global__ void __launch_bounds__(64 * kDownWaves) moe_down_kernel(MoeLayer a) {
  __shared__ MoeLists lists;
  __shared__ f32x4 part[kDownWaves][MT][64];
  moe_lists(a, lists);
  const int n0 = blockIdx.x * 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 15, quarter = lane >> 4;
  const int units = (a.f + kUnit - 1) / kUnit, all = lists.count * units;
  f32x4 total[MT] = {};
  if (wave < all) {
    MoeWeights w[kDownAhead + 1][1];
    // the unit that is loaded next, all of them, and of its expert
    int next = wave, next_which = wave / units, next_u = wave - next_which * units;
    int64_t next_row = 0;
    auto seek = [&]() {
      next_row = (int64_t)__builtin_amdgcn_readfirstlane(lists.list[next_which]) * a.k + n0 + col;
    };
    auto load = [&](MoeWeights& x) {
      if (next >= all) return;
      x = moe_load<WHOLE>(a.down_codes, a.down_scales, next_row, a.f, next_u * kUnit + 64 * quarter);
      next += kDownWaves;
      next_u += kDownWaves;
      if (next_u >= units && next < all) {
        do {
          next_u -= units;
          ++next_which;
        } while (next_u >= units);
        seek();
      }
    };
    seek();
#pragma unroll
    for (int j = 0; j < kDownAhead; ++j) load(w[j][0]);

    const uint16_t* at_h[MT];
    bool live[MT];
    float weight[MT];
    f32x4 acc[1][MT] = {};
    int which = wave / units, u = wave - which * units, left = (all - wave + kDownWaves - 1) / kDownWaves;
    auto begin = [&]() {  // the columns of expert `which`
      const int expert = __builtin_amdgcn_readfirstlane(lists.list[which]);
      const float factor = global_decode(a.down_global ? a.down_global + expert : nullptr);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int t = 16 * m + col, p = moe_pair(a, lists, t, expert);
        live[m] = p >= 0;
        at_h[m] = a.h_pieces + moe_instead(p, live[m]) * moe_row(a.f, PH) + 8 * quarter;
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
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) total[m][i] = live[m] ? total[m][i] + weight[m] * acc[0][m][i] : total[m][i];
    };
    begin();
    while (left > 0) {
#pragma unroll
      for (int j = 0; j <= kDownAhead; ++j) {
        if (left <= 0) break;
        moe_unit<1, MT, PH>(w[j], at_h, u, acc, [&]() { load(w[(j + kDownAhead) % (kDownAhead + 1)][0]); });
        --left;
        u += kDownWaves;
        if (u >= units && left > 0) {
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

struct MoePlan {
  size_t logits, x, h, bytes;  // offsets in the workspace
};
MoePlan moe_plan(int64_t tokens, int64_t top_k, int64_t experts, int64_t k, int64_t f, int dt) {
  auto up = [](size_t n) { return (n + 255) / 256 * 256; };
  MoePlan p;
  p.logits = 0;
  p.x = up((size_t)tokens * experts * 8);
  p.h = p.x + up((size_t)tokens * moe_row((int)k, moe_x_pieces(dt)) * 2);
  p.bytes = p.h + up((size_t)tokens * top_k * moe_row((int)f, moe_h_pieces(dt)) * 2);
  return p;
}

template <int DT, int MT>
hipError_t launch_products(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT), PH = moe_h_pieces(DT);
  const int pairs = a.tokens * a.top_k, most = pairs < a.experts ? pairs : a.experts;
  const unsigned up = (unsigned)(most * (a.f / 16)), down = (unsigned)(a.k / 16);
  if (a.k % 64 == 0) moe_up_kernel<MT, PX, PH, true><<<up, 64 * kUpWaves, 0, s>>>(a);
  else moe_up_kernel<MT, PX, PH, false><<<up, 64 * kUpWaves, 0, s>>>(a);
  if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  if (a.f % 64 == 0) moe_down_kernel<DT, MT, PH, true><<<down, 64 * kDownWaves, 0, s>>>(a);
  else moe_down_kernel<DT, MT, PH, false><<<down, 64 * kDownWaves, 0, s>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t launch(const MoeLayer& a, hipStream_t s) {
  constexpr int PX = moe_x_pieces(DT);
  const int64_t eights = a.tokens * (moe_row(a.k, 1) + a.top_k * (moe_row(a.f, 1) - a.f)) / 8;
  const unsigned cuts = (unsigned)((eights + 255) / 256);
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
