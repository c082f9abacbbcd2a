// kv_attention.hip -- attention of 16-bit or float32 queries over keys and
// values held in NVFP4 (kv_device.h), for gfx950.
//
// Query i of a sequence with n queries and a context of L tokens (its own
// among them) stands at position p = L - n + i.  It sees key j when j < L,
// with `causal` j <= p, and with a window w > 0 also j > p - w:
//     s_j = scale * q . k_j,   lse = log sum_j exp(s_j),
//     out = sum_j exp(s_j - lse) v_j;   no visible key: out = 0, lse = -inf.
//
// Numbers.  A held value e2m1 * e4m3 has at most 6 significant bits and a
// magnitude of 0 or 2^-10 .. 2688, so float16 holds it exactly and the
// matrix cores multiply it without any rounding; the global scales go into
// the factor of the scores and into the output.  A query row is brought into
// float16's range by a power of two, which keeps every bit of a float16 or
// bfloat16 element (down to 2^-38 of the row's largest); a float32 element
// becomes the sum of two float16, 22 bits.  Probabilities are rounded to
// float16 for their product with the values (2^-12 relative, below the
// rounding of a 16-bit output; float32: two float16 again).  Scores, the
// running maximum, sums and outputs are float32.
//
// Rows.  The `groups` query heads of a kv head and the queries of a sequence
// share its keys, so they form the rows r = query * groups + head of one
// product, and keys and values are read once for all of them.
#include "kv_device.h"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kNone = -__builtin_huge_valf();

// A tile's scores move its running maximum only when one exceeds it by more
// than 2^kLag, so most tiles skip the rescaling of the output.  Probabilities
// are kept times 2^kBias (2^(kLag + kBias) < 65504).
//
// Small weights.  Below 2^-14 a float16 loses bits, and in a 4-bit cache an
// output may consist of small weights alone (the keys with large weights
// hold an exact 0 there).  So weights below KvSmall::kLimit, 2^-26 of the
// largest (float32 queries, whose second float16 is 2^-11 smaller: 2^-15),
// enter the product in a further pass, times 2^kShift with the output scaled
// along, and so keep their bits.  Tiles without such weights, nearly all
// unless a row's scores spread over more than 18 nats, take one pass.
constexpr float kLag = 3.0f, kBias = 12.0f;
template <int SPLIT> struct KvSmall {
  static constexpr float kLimitLog2 = SPLIT == 2 ? -3.0f : -14.0f;
  static constexpr float kLimit = SPLIT == 2 ? 0x1p-3f : 0x1p-14f;
  static constexpr float kUp = SPLIT == 2 ? 0x1p18f : 0x1p29f, kDown = SPLIT == 2 ? 0x1p-18f : 0x1p-29f;
  static constexpr int kPasses = SPLIT == 2 ? 4 : 3;  // outputs stay below 2^44 2^58
};

// ----------------------------------------------------------------- ranges

// The rows [row0, row0 + rows) of a sequence and the keys [lo, hi) that any of them may see.
struct KvRange {
  int first, n, context;  // first token and number of queries, context length
  int lo, hi;
};
__device__ __forceinline__ KvRange kv_range(const KvAttention& a, int b, int row0, int rows) {
  KvRange r;
  r.first = a.query_starts ? a.query_starts[b] : b;
  r.n = a.query_starts ? a.query_starts[b + 1] - r.first : 1;
  // what lies outside the sizes that the caller gave is not touched
  r.first = max(0, min(r.first, (int)a.tokens));
  r.n = max(0, min(min(r.n, a.max_queries), (int)a.tokens - r.first));
  r.context = a.context_lens[b];
  r.lo = 0;
  r.hi = min(r.context, a.max_keys);
  if (a.causal) {
    const int q0 = row0 / a.groups, q1 = min((row0 + rows - 1) / a.groups, r.n - 1);
    r.hi = min(r.hi, r.context - r.n + q1 + 1);
    if (a.window > 0) r.lo = max(0, r.context - r.n + q0 - a.window + 1);
  }
  return r;
}

// ----------------------------------------------------------------- decode

// 8 codes (a dword) times a block scale, exact in float16.
__device__ __forceinline__ f16x8 kv_decode8(uint32_t w, _Float16 s) {
  const f16x2 sc = {s, s};
  const f16x2 a = e2m1_decode2_f16<0>(w) * sc, b = e2m1_decode2_f16<1>(w) * sc;
  const f16x2 c = e2m1_decode2_f16<2>(w) * sc, d = e2m1_decode2_f16<3>(w) * sc;
  return f16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// Two scale bytes (bytes 0 and 1 of w) as float16, exact.
__device__ __forceinline__ f16x2 kv_scale2(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, false);
}

// The codes and scales of NG groups of 16 of one cached row, from group `g0`.
template <int NG>
struct KvGroups {
  uint32_t w[2 * NG];
  uint32_t s;  // scale bytes
};
// EXACT: dim = 64 NG, so a lane's NG groups exist and lie on an 8 NG byte
// boundary; otherwise groups from `groups` on are zeros.  live: the row exists.
template <int NG, bool EXACT>
__device__ __forceinline__ KvGroups<NG> kv_load(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                int64_t row, int dim, int g0, bool live) {
  KvGroups<NG> r;
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i) r.w[i] = 0u;
  r.s = 0u;
  const uint8_t* c = codes + row * (dim / 2) + 8 * g0;
  const uint8_t* s = scales + row * (dim / 16) + g0;
  if constexpr (EXACT) {
    if (live) {
      if constexpr (NG == 1) {
        const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(c));
        r.w[0] = x.x; r.w[1] = x.y;
        r.s = *s;
      } else {
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) {
          const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c) + i);
          r.w[4 * i] = x.x; r.w[4 * i + 1] = x.y; r.w[4 * i + 2] = x.z; r.w[4 * i + 3] = x.w;
        }
        if constexpr (NG == 2) r.s = *reinterpret_cast<const uint16_t*>(s);
        else r.s = *reinterpret_cast<const uint32_t*>(s);
      }
    }
  } else {
    const int have = dim / 16 - g0;
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (live && i < have) {
        const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(c) + i);
        r.w[2 * i] = x.x; r.w[2 * i + 1] = x.y;
        r.s |= (uint32_t)s[i] << (8 * i);
      }
  }
  return r;
}
// Dwords 2g, 2g + 1 (group g) as 16 float16.
template <int NG>
__device__ __forceinline__ void kv_values(const KvGroups<NG>& r, f16x8 (&v)[2 * NG]) {
  const f16x2 s01 = kv_scale2(r.s);
  f16x2 s23 = s01;
  if constexpr (NG > 2) s23 = kv_scale2(r.s >> 16);
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const _Float16 s = g == 0 ? s01.x : g == 1 ? s01.y : g == 2 ? s23.x : s23.y;
    v[2 * g] = kv_decode8(r.w[2 * g], s);
    v[2 * g + 1] = kv_decode8(r.w[2 * g + 1], s);
  }
}

// Two transposing LDS reads: the 16 lanes of a quarter point at four rows of
// 16 float16 (8 bytes a lane); each gets one column's four values.
__device__ __forceinline__ f16x8 kv_read_transposed(const uint8_t* lo, const uint8_t* hi) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lo);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)hi);
  return __builtin_bit_cast(f16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ----------------------------------------------------------------- queries

// `count` (a multiple of 8) elements of a query row from element d on, as
// floats; elements from dim on are zeros.
template <int COUNT>
__device__ __forceinline__ void kv_load_query(const KvAttention& a, int dt, bool vec, int64_t at, int d, int dim,
                                              bool live, float (&x)[COUNT]) {
#pragma unroll
  for (int i = 0; i < COUNT / 8; ++i) {
    float f[8] = {};
    if (live && d + 8 * i < dim) {
      const int64_t e = at + d + 8 * i;
      if (vec) {
        if (dt == kF32) load8x<kF32>(a.q, e >> 3, f);
        else if (dt == kF16) load8x<kF16>(a.q, e >> 3, f);
        else load8x<kBF16>(a.q, e >> 3, f);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          f[j] = dt == kF32 ? reinterpret_cast<const float*>(a.q)[e + j]
                 : dt == kF16 ? (float)reinterpret_cast<const _Float16*>(a.q)[e + j]
                              : (float)reinterpret_cast<const __bf16*>(a.q)[e + j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) x[8 * i + j] = f[j];
  }
}

// The power of two 2^-e that brings a row of largest magnitude `top` to
// 2^13 .. 2^14, and 2^e.  Rows of zeros, infinities and NaN stay as they are.
__device__ __forceinline__ float kv_row_power(float top, float& back) {
  const int field = (int)((__float_as_uint(top) >> 23) & 0xFFu);
  if (!(top > 0.0f) || field == 255) {
    back = 1.0f;
    return 1.0f;
  }
  const int e = max(-112, field - 140);
  back = __builtin_ldexpf(1.0f, e);
  return __builtin_ldexpf(1.0f, -e);
}

template <int DT>
__device__ __forceinline__ void kv_store4(void* out, int64_t e, const float (&v)[4]) {
  if constexpr (DT == kF32) {
    *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(out) + e) = f32x4{v[0], v[1], v[2], v[3]};
  } else {
    *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(out) + e) =
        u32x2{pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
  }
}
__device__ __forceinline__ void kv_store4(int dt, void* out, int64_t e, const float (&v)[4]) {
  if (dt == kF32) kv_store4<kF32>(out, e, v);
  else if (dt == kF16) kv_store4<kF16>(out, e, v);
  else kv_store4<kBF16>(out, e, v);
}

// ----------------------------------------------------------------- few rows
//
// Up to 16 MT rows share a chunk of keys.  A workgroup of four waves takes one
// (chunk, kv head, sequence); each wave walks its own tiles of 32 keys with
// its own running maximum, and the four meet at the end.
//
// Per tile a lane holds 64 NG / 4 values of key l % 16 (+ 16): it loads their
// codes with one wide load and uses them in place as rows of the matrix
// product S^T = K Q^T (16 x 16 x 32), whose k order is free as long as the
// query fragments follow it.  Lane l then holds the scores of row l % 16 for
// keys 4 (l / 16) + i, which is the operand layout of the second product
// O^T = V^T P^T, so probabilities never leave their lane.  Values are decoded
// the same way, written to the wave's own LDS as float16 and read back
// transposed (ds_read_b64_tr_b16); nothing in the loop waits for another wave.
// The next tile's codes are loaded before this tile's work.
constexpr int kFewWaves = 4;
constexpr int kFewTile = 32;
constexpr int kFewStep = kFewWaves * kFewTile;

struct KvSplit {
  int chunk, splits;  // keys per chunk, chunks per row tile (1: the output is written directly)
  float* sums;        // [rows of q * heads][splits][dim], times 2^kBias
  float* stats;       // [rows of q * heads][splits][2]: maximum (log2), sum
};

constexpr int few_row_bytes(int NG) { return 128 * NG + 32; }  // a key's values in LDS: +32 spreads the banks

template <int NG, int MT, int SPLIT, bool EXACT>
__global__ void __launch_bounds__(256, (NG * MT * SPLIT > 4 ? 1 : NG * MT * SPLIT > 2 ? 2 : 4))
kv_few_kernel(KvCache c, KvAttention a, KvSplit sp, int dt, bool q_vec) {
  constexpr int DP = 64 * NG, STEPS = 2 * NG, DB = DP / 16, RB = few_row_bytes(NG);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ float stat_m[kFewWaves][16 * MT], stat_l[kFewWaves][16 * MT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, quarter = lane >> 4;
  const int b = blockIdx.y;
  const int split = blockIdx.x % sp.splits, tile_head = blockIdx.x / sp.splits;
  const int head = tile_head % c.heads;
  const int row0 = tile_head / c.heads * 16 * MT;

  const KvRange rg = kv_range(a, b, row0, 16 * MT);
  const int rows = rg.n * a.groups;
  if (row0 >= rows) return;
  const int begin = rg.lo + split * sp.chunk, end = min(rg.hi, begin + sp.chunk);
  if (begin >= end && split > 0) return;  // the first chunk's workgroup answers for rows that see nothing

  // page numbers of the chunk, -1 where there is no such page
  int* page_of = reinterpret_cast<int*>(lds + kFewWaves * kFewTile * RB);
  const int p0 = kv_div(begin, c.page_div);
  if (begin < end) {
    const int count = (int)kv_div(end - 1, c.page_div) - p0 + 1;
    for (int i = threadIdx.x; i < count; i += 256) {
      const int p = a.page_table[b * a.table_stride + p0 + i];
      page_of[i] = p >= 0 && p < c.pages ? p : -1;
    }
  }

  // queries: row `col` of each row tile, values 16 NG quarter ..
  f16x8 q[MT][SPLIT][STEPS];
  float factor[MT];
  int see_lo[MT], see_hi[MT];  // keys that row `col` sees
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = row0 + 16 * m + col;
    const bool live = r < rows;
    const int qi = r / a.groups;
    const int64_t at = (int64_t)(rg.first + qi) * a.q_token + (head * a.groups + (r - qi * a.groups)) * a.q_head;
    float x[16 * NG];
    kv_load_query<16 * NG>(a, dt, q_vec, at, 16 * NG * quarter, c.dim, live, x);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 16 * NG; ++i) top = fmaxf(top, __builtin_fabsf(x[i]));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    float back;
    const float power = kv_row_power(top, back);
    factor[m] = a.scale * kLog2e * global_decode(c.global_k) * back;
#pragma unroll
    for (int t = 0; t < STEPS; ++t)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float y = x[8 * t + j] * power;
        q[m][0][t][j] = (_Float16)y;
        if constexpr (SPLIT == 2) q[m][SPLIT - 1][t][j] = (_Float16)(y - (float)(_Float16)y);
      }
    const int pos = rg.context - rg.n + qi;
    see_hi[m] = !live ? 0 : a.causal ? min(rg.hi, pos + 1) : rg.hi;
    see_lo[m] = a.causal && a.window > 0 ? max(0, pos - a.window + 1) : 0;
  }
  // keys that every row sees: [all_lo, all_hi)
  int all_hi = rg.hi, all_lo = 0;
  if (a.causal) {
    all_hi = min(rg.hi, rg.context - rg.n + row0 / a.groups + 1);
    if (a.window > 0)
      all_lo = max(0, rg.context - rg.n + min(rg.n - 1, (row0 + 16 * MT - 1) / a.groups) - a.window + 1);
  }
  __syncthreads();

  f32x4 acc[MT][DB];
  float m_run[MT], sub[MT], l_run[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    m_run[m] = kNone;
    sub[m] = -kBias;
    l_run[m] = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  uint8_t* mine = lds + wave * kFewTile * RB;
  const int g0 = NG * quarter;
  KvGroups<NG> kn[2], vn[2];  // the next tile
  uint32_t live_n = 0;        // which of its 32 keys exist
  auto fetch = [&](int tile) {
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int j = tile + 16 * u + col;
      bool live = j < end;
      int64_t row = 0;
      if (live) {
        const int pi = kv_div(j, c.page_div);
        const int page = page_of[pi - p0];
        live = page >= 0;
        row = kv_row(c, max(page, 0), head, j - pi * c.page_size);
      }
      bits |= (uint32_t)(__ballot(live) & 0xFFFFu) << (16 * u);
      kn[u] = kv_load<NG, EXACT>(c.k_codes, c.k_scales, row, c.dim, g0, live);
      vn[u] = kv_load<NG, EXACT>(c.v_codes, c.v_scales, row, c.dim, g0, live);
    }
    live_n = bits;
  };
  int tile = begin + wave * kFewTile;
  if (tile < end) fetch(tile);
  for (; tile < end; tile += kFewStep) {
    const KvGroups<NG> k0 = kn[0], k1 = kn[1], v0 = vn[0], v1 = vn[1];
    const uint32_t live = live_n;
    if (tile + kFewStep < end) fetch(tile + kFewStep);

    // scores
    f32x4 s[MT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f16x8 kf[STEPS];
      kv_values<NG>(u == 0 ? k0 : k1, kf);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int t = 0; t < STEPS; ++t)
#pragma unroll
          for (int e = SPLIT - 1; e >= 0; --e)
            x = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf[t], q[m][e][t], x, 0, 0, 0);
        s[m][u] = x;
      }
    }
    // values into LDS
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f16x8 vf[STEPS];
      kv_values<NG>(u == 0 ? v0 : v1, vf);
#pragma unroll
      for (int t = 0; t < STEPS; ++t)
        *reinterpret_cast<f16x8*>(mine + (16 * u + col) * RB + 32 * NG * quarter + 16 * t) = vf[t];
    }
    // probabilities
    const bool masked = live != 0xFFFFFFFFu || tile < all_lo || tile + kFewTile > all_hi;
    float w[MT][8];
    bool small = false;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = s[m][i >> 2][i & 3] * factor[m];
      if (masked) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = 16 * (i >> 2) + 4 * quarter + (i & 3);
          const bool see = ((live >> key) & 1u) && tile + key >= see_lo[m] && tile + key < see_hi[m];
          x[i] = see ? x[i] : kNone;
        }
      }
      float top = x[0], low = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        top = fmaxf(top, x[i]);
        low = fminf(low, x[i]);
      }
      if (__any(top > m_run[m] + kLag)) {  // rare once a row has met its large scores
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m_run[m], top);
        const float keep = m_run[m] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m_run[m] - next);
        m_run[m] = next;
        sub[m] = next == kNone ? -kBias : next - kBias;
        l_run[m] *= keep;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][d][i] *= keep;
      }
      small |= low - sub[m] < KvSmall<SPLIT>::kLimitLog2;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w[m][i] = __builtin_amdgcn_exp2f(x[i] - sub[m]);
        l_run[m] += w[m][i];
      }
    }
    // output: 16 values (rows) of V^T at a time, keys 4 quarter + 16 u + (0 .. 3) a lane
    bool again = __any(small);
    for (int pass = 1;; ++pass) {
      float rest[MT][8];
      if (again) {
        bool any = false;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const bool tiny = w[m][i] < KvSmall<SPLIT>::kLimit;
            rest[m][i] = tiny ? w[m][i] * KvSmall<SPLIT>::kUp : 0.0f;
            any |= rest[m][i] > 0.0f;
            if (tiny) w[m][i] = 0.0f;
          }
        again = __any(any) && pass < KvSmall<SPLIT>::kPasses;
      }
      f16x8 p[MT][SPLIT];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[m][0][i] = (_Float16)w[m][i];
          if constexpr (SPLIT == 2) p[m][SPLIT - 1][i] = (_Float16)(w[m][i] - (float)(_Float16)w[m][i]);
        }
#pragma unroll
      for (int d = 0; d < DB; ++d) {
        const uint8_t* at = mine + (4 * quarter + (col >> 2)) * RB + 32 * d + 8 * (col & 3);
        const f16x8 vt = kv_read_transposed(at, at + 16 * RB);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = SPLIT - 1; e >= 0; --e)
            acc[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt, p[m][e], acc[m][d], 0, 0, 0);
      }
      if (!again) {
        if (pass > 1) {
          float down = KvSmall<SPLIT>::kDown;
          for (int i = 2; i < pass; ++i) down *= KvSmall<SPLIT>::kDown;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[m][d][i] *= down;
        }
        break;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][d][i] *= KvSmall<SPLIT>::kUp;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[m][i] = rest[m][i];
      }
    }
  }

  // the four waves meet
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float l = l_run[m];
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (quarter == 0) {
      stat_m[wave][16 * m + col] = m_run[m];
      stat_l[wave][16 * m + col] = l;
    }
  }
  const float value_factor = global_decode(c.global_v);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (m > 0) __syncthreads();
    float* own = reinterpret_cast<float*>(mine) + col * (DP + 4);
#pragma unroll
    for (int d = 0; d < DB; ++d) *reinterpret_cast<f32x4*>(own + 16 * d + 4 * quarter) = acc[m][d];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * (DP / 4); i += 256) {
      const int rr = i / (DP / 4), d = 4 * (i - rr * (DP / 4));
      const int r = row0 + 16 * m + rr;
      if (r >= rows || d >= c.dim) continue;
      float mt = stat_m[0][16 * m + rr];
#pragma unroll
      for (int w = 1; w < kFewWaves; ++w) mt = fmaxf(mt, stat_m[w][16 * m + rr]);
      float l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) {
        const float mw = stat_m[w][16 * m + rr];
        const float by = mw == kNone ? 0.0f : __builtin_amdgcn_exp2f(mw - mt);
        l += by * stat_l[w][16 * m + rr];
        const f32x4 o = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds + w * kFewTile * RB) +
                                                        rr * (DP + 4) + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += by * o[j];
      }
      const int qi = r / a.groups;
      const int64_t row = (int64_t)(rg.first + qi) * a.query_heads + head * a.groups + (r - qi * a.groups);
      if (sp.splits == 1) {
        const float by = l == 0.0f ? 0.0f : value_factor / l;  // a NaN stays one
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= by;
        kv_store4(dt, a.out, row * c.dim + d, v);
        if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? kNone : (mt - kBias + __builtin_log2f(l)) * kLn2;
      } else {
        const int64_t at = row * sp.splits + split;
        kv_store4<kF32>(sp.sums, at * c.dim + d, v);
        if (d == 0) *reinterpret_cast<f32x2*>(sp.stats + 2 * at) = f32x2{mt, l};
      }
    }
  }
}

// ----------------------------------------------------------------- joining the chunks

// One wave per query and query head: the maximum over its chunks, then their
// sums in chunk order (the same bits on every run).
__global__ void __launch_bounds__(256) kv_join_kernel(KvCache c, KvAttention a, KvSplit sp, int tile_rows, int dt) {
  const int lane = threadIdx.x & 63, b = blockIdx.y;
  const int r0 = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int qi = r0 / a.query_heads, qh = r0 - qi * a.query_heads;
  const int r = qi * a.groups + qh % a.groups;  // its row among those of its kv head
  const KvRange rg = kv_range(a, b, r / tile_rows * tile_rows, tile_rows);
  if (qi >= rg.n) return;
  const int used = rg.hi > rg.lo ? (rg.hi - rg.lo + sp.chunk - 1) / sp.chunk : 1;
  const int64_t row = (int64_t)(rg.first + qi) * a.query_heads + qh;
  const float* stats = sp.stats + 2 * row * sp.splits;
  float top = kNone;
  for (int i = lane; i < used; i += 64) top = fmaxf(top, stats[2 * i]);
  top = wave_max(top);
  const float* sums = sp.sums + row * sp.splits * c.dim;
  float l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool on = 4 * lane < c.dim;
#pragma unroll 4
  for (int i = 0; i < used; ++i) {
    const f32x2 st = *reinterpret_cast<const f32x2*>(stats + 2 * i);
    const float by = st.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(st.x - top);
    l += by * st.y;
    if (on) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(sums + (int64_t)i * c.dim + 4 * lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += by * o[j];
    }
  }
  const float by = l == 0.0f ? 0.0f : global_decode(c.global_v) / l;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= by;
  if (on) kv_store4(dt, a.out, row * c.dim + 4 * lane, v);
  if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? kNone : (top - kBias + __builtin_log2f(l)) * kLn2;
}

// ----------------------------------------------------------------- launches

struct KvPlan {
  int row_tiles, tile_rows;  // rows a workgroup takes, and how many such tiles a sequence and kv head has
  int chunk, splits;
  size_t sums_bytes, bytes;
};

KvPlan kv_plan(const KvCache& c, const KvAttention& a) {
  KvPlan p;
  const int64_t rows = (int64_t)a.max_queries * a.groups;
  p.tile_rows = rows <= 16 ? 16 : 32;
  p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  int64_t keys = a.max_keys;
  if (a.window > 0) keys = keys < (int64_t)a.window + a.max_queries ? keys : (int64_t)a.window + a.max_queries;
  const int64_t items = (int64_t)a.seqs * c.heads * p.row_tiles;
  const int64_t want = 8 * device_cu_count();
  int64_t splits = (want + items - 1) / items;
  const int64_t most = (keys + kFewStep - 1) / kFewStep;
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  int64_t chunk = (keys + splits - 1) / splits;
  chunk = (chunk + kFewStep - 1) / kFewStep * kFewStep;
  if (chunk > 2048) chunk = 2048;
  if (chunk < kFewStep) chunk = kFewStep;
  splits = keys > 0 ? (keys + chunk - 1) / chunk : 1;
  p.chunk = (int)chunk;
  p.splits = (int)splits;
  const int64_t parts = a.tokens * a.query_heads * splits;
  p.sums_bytes = splits > 1 ? ((size_t)parts * c.dim * 4 + 255) / 256 * 256 : 0;
  p.bytes = splits > 1 ? p.sums_bytes + ((size_t)parts * 8 + 255) / 256 * 256 : 0;
  return p;
}

constexpr int kMaxLds = 144 * 1024;  // leaves room for the kernels' static LDS

// Lets `kernel` have more than 64 KB of dynamic LDS; once per device.
template <typename K>
hipError_t allow_lds(K* kernel, bool (&set)[64]) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  if (dev < 0 || dev >= 64 || set[dev]) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds);
  if (e == hipSuccess) set[dev] = true;
  return e;
}

template <int NG, bool EXACT>
hipError_t launch_few(const KvCache& c, const KvAttention& a, const KvSplit& sp, const KvPlan& p, int dt, bool q_vec,
                      hipStream_t s) {
  const dim3 grid((unsigned)(p.splits * c.heads * p.row_tiles), a.seqs);
  const size_t lds = (size_t)kFewWaves * kFewTile * few_row_bytes(NG) + 4 * (p.chunk / c.page_size + 2);
#define KV_FEW(MT, SPLIT)                                                                         \
  do {                                                                                            \
    static bool set[64];                                                                          \
    if (hipError_t e = allow_lds(&kv_few_kernel<NG, MT, SPLIT, EXACT>, set)) return e;            \
    kv_few_kernel<NG, MT, SPLIT, EXACT><<<grid, 256, lds, s>>>(c, a, sp, dt, q_vec);              \
  } while (0)
  if (p.tile_rows == 16) {
    if (dt == kF32) KV_FEW(1, 2); else KV_FEW(1, 1);
  } else {
    if (dt == kF32) KV_FEW(2, 2); else KV_FEW(2, 1);
  }
#undef KV_FEW
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(const KvCache& c, const KvAttention& a) { return kv_plan(c, a).bytes; }

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, int dt, void* workspace, hipStream_t s) {
  const KvPlan p = kv_plan(c, a);
  KvSplit sp{p.chunk, p.splits, reinterpret_cast<float*>(workspace),
             reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + p.sums_bytes)};
  const bool q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && (a.q_token | a.q_head) % 8 == 0;
  hipError_t e;
  if (c.dim == 64) e = launch_few<1, true>(c, a, sp, p, dt, q_vec, s);
  else if (c.dim == 128) e = launch_few<2, true>(c, a, sp, p, dt, q_vec, s);
  else if (c.dim == 256) e = launch_few<4, true>(c, a, sp, p, dt, q_vec, s);
  else if (c.dim < 64) e = launch_few<1, false>(c, a, sp, p, dt, q_vec, s);
  else if (c.dim < 128) e = launch_few<2, false>(c, a, sp, p, dt, q_vec, s);
  else if (c.dim <= 192) e = launch_few<3, false>(c, a, sp, p, dt, q_vec, s);
  else e = launch_few<4, false>(c, a, sp, p, dt, q_vec, s);
  if (e != hipSuccess || p.splits == 1) return e;
  const dim3 grid((unsigned)(((int64_t)a.max_queries * a.query_heads + 3) / 4), a.seqs);
  kv_join_kernel<<<grid, 256, 0, s>>>(c, a, sp, p.tile_rows, dt);
  return hipGetLastError();
}

}  // namespace nvfp4
