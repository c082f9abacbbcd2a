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
// bfloat16 element down to 2^-27 of the row's largest, and smaller ones to
// within 2^-38 of it; a float32 element becomes the sum of two float16, 22
// bits.  Probabilities are rounded to float16 for their product with the values
// (2^-11 of each: an eighth of a bfloat16 output's own rounding, as much as a
// float16 output's; float32: two float16 again, 2^-22).  Scores, the running
// maximum, sums and outputs are float32.
//
// What a mask hides reaches no output, not even as NaN (notes in both kernels).
//
// Rows.  The `groups` query heads of a kv head and the queries of a sequence
// share its keys, so they form the rows r = query * groups + head of one
// product, and keys and values are read once for all of them.
#include <atomic>

#include "kv_device.h"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.693147180559945309417f;
constexpr float kNone = -__builtin_huge_valf();
constexpr float kNaN = __builtin_nanf("");

// A tile's scores move its running maximum only when one exceeds it by more
// than 2^kLag, so that tiles whose maximum hardly grows skip the rescaling of
// the output.  Probabilities are kept times 2^kBias (2^(kLag + kBias) < 65504).
//
// The second float16 of a float32 query's probability is kept times 2^11, its
// products taken with the values times 2^-11 (exact too: a value is a multiple
// of 2^-10), which gives it the range of the first.
//
// Small weights.  Below 2^-14 a float16 loses bits, and in a 4-bit cache an
// output may consist of small weights alone (the keys with large weights
// hold an exact 0 there).  So weights below 2^kSmall, 2^-29 of the largest,
// enter products of their own, in bands of 2^kShift, with the output or their
// sums scaled along, and so keep their bits down to 2^-145 of the largest.
// Tiles without such weights, nearly all unless a row's scores spread over more
// than 20 nats, skip this.  Measured with scores of 1.8 nats deviation, 5 x up
// to 1023 queries over up to 9001 keys: 441 us without any such handling, 468
// with it; with kLag 3 and kBias 12, a window of 2^26, 550; with all bands'
// sums apart, which needs no scaled output, 474 against 443.
//
// Large scores.  A weight's exponent is score - sub with sub = maximum - kBias
// rounded.  Beyond kBig that rounding, and that of scores which are products
// never rounded by themselves, could let weights pass 65504; so there exponents
// are kept below kMost apart.  Elsewhere they are at most kLag + kBias + 2^-4.
constexpr float kLag = 0.9f, kBias = 15.0f;
constexpr float kBig = 0x1p18f, kMost = 15.99f;
constexpr float kSmall = -14.0f, kShift = 29.0f;
constexpr float kUp = 0x1p29f, kDown = 0x1p-29f;
constexpr float kRest = 0x1p11f;
constexpr int kBands = 5, kNearBands = 3;  // outputs stay below 2^45, in near bands 2^45 2^58

// ----------------------------------------------------------------- ranges

// The first key that the query at position `pos` (below 0: before the context) may see.
__device__ __forceinline__ int kv_window_begin(const KvAttention& a, int pos) {
  return a.causal && a.window > 0 ? max(0, max(pos, 0) - a.window + 1) : 0;  // (without overflow for any window)
}

// Positions stay below kKvMaxKeys, some thousands below 2^31: a tile or a
// chunk past the end of a context is still an int.
//
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
  r.context = max(0, min(a.context_lens[b], kKvMaxKeys));
  r.lo = 0;
  r.hi = min(r.context, a.max_keys);
  if (a.causal) {
    const int q0 = kv_div(row0, a.group_div), q1 = min((int)kv_div(row0 + rows - 1, a.group_div), r.n - 1);
    r.hi = min(r.hi, r.context - r.n + q1 + 1);
    r.lo = kv_window_begin(a, r.context - r.n + q0);
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
template <int NG, bool EXACT>
struct KvGroups {
  uint32_t w[2 * NG];
  uint32_t s[EXACT ? 1 : NG];  // scale bytes: of all groups in one, or one each (joining them would wait for the loads)
};
// The codes of a row begin at byte page * page_bytes + head_bytes + offset *
// dim/2, its scales at an eighth of that.  (page_bytes < 2^32: one
// multiply-add for the page.)
struct KvPlace {
  uint32_t page_bytes;
  uint64_t head_bytes;
};
__device__ __forceinline__ KvPlace kv_place(const KvCache& c, int head) {
  return KvPlace{(uint32_t)(c.heads * c.page_size) * (uint32_t)(c.dim / 2),
                 (uint64_t)head * c.page_size * (c.dim / 2)};
}
__device__ __forceinline__ uint64_t kv_page_start(const KvPlace& p, int page) {
  return (uint64_t)(uint32_t)page * p.page_bytes + p.head_bytes;
}
template <int NG, bool EXACT>
__device__ __forceinline__ uint32_t kv_row_start(int off, int dim) {
  return (uint32_t)off * (EXACT ? 32u * NG : (uint32_t)dim / 2);
}

// A key's page (counted from the run's first) and its offset there, moved on
// by a fixed number of keys without a division.
struct KvStep {
  int pages, rest;  // keys = pages * page_size + rest
};
__device__ __forceinline__ KvStep kv_step(const KvCache& c, int keys) {
  const int q = __builtin_amdgcn_readfirstlane(kv_div(keys, c.page_div));
  return KvStep{q, keys - q * c.page_size};
}
__device__ __forceinline__ void kv_advance(const KvStep& s, int page_size, int& page, int& off) {
  off += s.rest;
  const bool over = off >= page_size;
  page += s.pages + (over ? 1 : 0);
  off -= over ? page_size : 0;
}

template <bool ONCE, typename T>
__device__ __forceinline__ T kv_fetch(const T* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(p);
  else return *p;
}
// Groups g0 .. g0 + NG - 1 of the row at `at` (kv_offset).  EXACT: dim = 64 NG,
// so they exist and lie on an 8 NG byte boundary; otherwise groups from
// dim / 16 on are zeros, as is a row that is not `live`.  ONCE: the row is
// read by this workgroup only.
template <int NG, bool EXACT, bool ONCE>
__device__ __forceinline__ KvGroups<NG, EXACT> kv_load(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                uint64_t at, int dim, int g0, bool live) {
  KvGroups<NG, EXACT> r;
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i) r.w[i] = 0u;
#pragma unroll
  for (int i = 0; i < (EXACT ? 1 : NG); ++i) r.s[i] = 0u;
  const uint8_t* c = codes + at + 8 * g0;
  const uint8_t* s = scales + (at >> 3) + g0;
  if constexpr (EXACT) {
    if (live) {
      if constexpr (NG == 1) {
        const u32x2 x = kv_fetch<ONCE>(reinterpret_cast<const u32x2*>(c));
        r.w[0] = x.x; r.w[1] = x.y;
        r.s[0] = *s;
      } else {
#pragma unroll
        for (int i = 0; i < NG / 2; ++i) {
          const u32x4 x = kv_fetch<ONCE>(reinterpret_cast<const u32x4*>(c) + i);
          r.w[4 * i] = x.x; r.w[4 * i + 1] = x.y; r.w[4 * i + 2] = x.z; r.w[4 * i + 3] = x.w;
        }
        if constexpr (NG == 2) r.s[0] = *reinterpret_cast<const uint16_t*>(s);
        else r.s[0] = *reinterpret_cast<const uint32_t*>(s);
      }
    }
  } else {
    const int have = dim / 16 - g0;
#pragma unroll
    for (int i = 0; i < NG; ++i)
      if (live && i < have) {
        const u32x2 x = kv_fetch<ONCE>(reinterpret_cast<const u32x2*>(c) + i);
        r.w[2 * i] = x.x; r.w[2 * i + 1] = x.y;
        r.s[i] = s[i];
      }
  }
  return r;
}
// The block scale of group g.
template <int NG, bool EXACT>
__device__ __forceinline__ _Float16 kv_scale_of(const KvGroups<NG, EXACT>& r, int g) {
  if constexpr (!EXACT) return kv_scale2(r.s[g]).x;
  const f16x2 two = kv_scale2(g < 2 ? r.s[0] : r.s[0] >> 16);
  return g & 1 ? two.y : two.x;
}
// Which groups' block scales are no numbers (bit 8 g + 7 of a joint one), and
// the scales without them.
template <int NG, bool EXACT>
__device__ __forceinline__ uint32_t kv_no_numbers(const KvGroups<NG, EXACT>& r) {
  if constexpr (EXACT) return ((r.s[0] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
  uint32_t bad = 0u;
#pragma unroll
  for (int g = 0; g < NG; ++g) bad |= (((r.s[g] & 0x7Fu) + 1u) & 0x80u) << (8 * g);
  return bad;
}
template <int NG, bool EXACT>
__device__ __forceinline__ void kv_drop(KvGroups<NG, EXACT>& r, uint32_t bad) {
  if constexpr (EXACT) {
    r.s[0] &= ~((bad >> 7) * 0xFFu);
  } else {
#pragma unroll
    for (int g = 0; g < NG; ++g) r.s[g] = bad >> (8 * g + 7) & 1u ? 0u : r.s[g];
  }
}
// Dwords 2g, 2g + 1 (group g) as 16 float16.
template <int NG, bool EXACT>
__device__ __forceinline__ void kv_values(const KvGroups<NG, EXACT>& r, f16x8 (&v)[2 * NG]) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const _Float16 s = kv_scale_of(r, g);
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

// Values for the second float16 of a probability.
__device__ __forceinline__ f16x8 kv_rest_values(f16x8 v) {
  return v * (_Float16)(1.0f / kRest);
}

// The same value, computed where it stands: keeps what a rare path derives from
// it out of the registers of the loop around that path.
__device__ __forceinline__ int opaque(int v) {
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ float opaque(float v) {
  asm("" : "+v"(v));
  return v;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// A weight's exponent, at most kMost (a NaN stays one).
__device__ __forceinline__ float kv_most(float t) { return t > kMost ? kMost : t; }

// ----------------------------------------------------------------- queries

// 8 elements of a query row as they lie in memory.
template <int SPLIT>
struct KvRaw {
  uint32_t w[4 * SPLIT];  // float32 for SPLIT 2, else 16-bit pairs
};
template <int SPLIT>
__device__ __forceinline__ KvRaw<SPLIT> kv_load_query(const KvAttention& a, bool vec, int64_t e, bool live) {
  KvRaw<SPLIT> r;
#pragma unroll
  for (int i = 0; i < 4 * SPLIT; ++i) r.w[i] = 0u;
  if (live) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < SPLIT; ++i) {
        const u32x4 x = reinterpret_cast<const u32x4*>(a.q)[SPLIT * (e >> 3) + i];
        r.w[4 * i] = x.x; r.w[4 * i + 1] = x.y; r.w[4 * i + 2] = x.z; r.w[4 * i + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4 * SPLIT; ++i) {
        if constexpr (SPLIT == 2) {
          r.w[i] = reinterpret_cast<const uint32_t*>(a.q)[e + i];
        } else {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(a.q) + e + 2 * i;
          r.w[i] = p[0] | (uint32_t)p[1] << 16;
        }
      }
    }
  }
  return r;
}
template <int SPLIT>
__device__ __forceinline__ void kv_unpack_query(const KvRaw<SPLIT>& r, int dt, float (&x)[8]) {
  if constexpr (SPLIT == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r.w[i]);
  } else {
    const u32x4 w = {r.w[0], r.w[1], r.w[2], r.w[3]};
    if (dt == kF16) unpack8<kF16>(w, x);
    else unpack8<kBF16>(w, x);
  }
}
template <int SPLIT>
__device__ __forceinline__ float kv_query_top(KvRaw<SPLIT>& r, int dt) {
  float x[8], top = 0.0f;
  kv_unpack_query<SPLIT>(r, dt, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, __builtin_fabsf(x[i]));
  // unpacked again when they are converted, rather than kept as floats
#pragma unroll
  for (int i = 0; i < 4 * SPLIT; ++i) r.w[i] = opaque((int)r.w[i]);
  return top;
}
// Times sign 2^-e as one or two float16.
template <int SPLIT>
__device__ __forceinline__ void kv_query_halves(const KvRaw<SPLIT>& r, int dt, int e, float sign, f16x8& hi, f16x8& lo) {
  float x[8];
  kv_unpack_query<SPLIT>(r, dt, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __builtin_ldexpf(x[i], -e) * sign;
    hi[i] = (_Float16)y;
    if constexpr (SPLIT == 2) lo[i] = (_Float16)(y - (float)hi[i]);
  }
}

// e such that 2^-e brings a row of largest magnitude `top` to 2^13 .. 2^14.
// Rows of zeros, infinities and NaN stay as they are.
__device__ __forceinline__ int kv_row_exponent(float top) {
  const int field = (int)((__float_as_uint(top) >> 23) & 0xFFu);
  return !(top > 0.0f) || field == 255 ? 0 : field - 140;
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

// ----------------------------------------------------------------- sharing out the keys
//
// Contexts differ in length and live on the device, so the workgroups share
// the work out themselves.  The keys of every (sequence, kv head) pair are cut
// into units of kFewStep keys, the pairs' units are counted through in order,
// and each of the launch's workgroups takes an equal run of them: a part of one
// pair, or the end of one and the beginning of the next ones.  The part of
// pair p that workgroup g computes has the number g + p, which no other part
// has.  A pair that one workgroup takes whole is written out by it; the parts
// of the others are joined by a second launch, 5 us.  (One workgroup per fixed
// chunk of keys instead cost 3 us of start and end for each chunk, and left
// compute units idle in the last round: 57 - 110 us, by the chunk's length,
// against 50 for 32 contexts of up to 8192, 8 heads.)
constexpr int kFewWaves = 4;
constexpr int kFewTile = 32;
constexpr int kFewStep = kFewWaves * kFewTile;

struct KvShare {
  int groups;    // workgroups of the launch
  int rows;      // rows of a part
  float* sums;   // [parts][rows][dim], times 2^kBias; null: workgroup g takes pair g whole
  float* stats;  // [parts][rows][2]: maximum (log2), sum
};

// Sequences 64 at a time, one per lane: their ranges and the units before them.
struct KvScan {
  KvRange range;  // of sequence base + lane
  int units;      // of one pair of this sequence; 0 past the last one and without queries
  int first;      // units before this sequence
  int after;      // units up to the end of the block
};
__device__ __forceinline__ void kv_scan(const KvCache& c, const KvAttention& a, int rows, int base, int before,
                                        KvScan& s) {
  const int lane = threadIdx.x & 63, b = base + lane;
  s.units = 0;
  s.range = KvRange{0, 0, 0, 0, 0};
  if (b < a.seqs) {
    s.range = kv_range(a, b, 0, rows);
    // a sequence that sees nothing still has a unit: its rows are written as zeros
    if (s.range.n > 0) s.units = max(1, (s.range.hi - s.range.lo + kFewStep - 1) / kFewStep);
  }
  int sum = s.units * c.heads;  // all units together stay below 2^30
  const int own = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(sum, off, 64);
    if (lane >= off) sum += up;
  }
  s.first = before + sum - own;
  s.after = before + __builtin_amdgcn_readlane(sum, 63);
}
// Lane `lane`'s (wave-uniform) range, in scalar registers.
__device__ __forceinline__ KvRange kv_range_of(const KvScan& s, int lane) {
  return KvRange{__builtin_amdgcn_readlane(s.range.first, lane), __builtin_amdgcn_readlane(s.range.n, lane),
                 __builtin_amdgcn_readlane(s.range.context, lane), __builtin_amdgcn_readlane(s.range.lo, lane),
                 __builtin_amdgcn_readlane(s.range.hi, lane)};
}
// Units of one workgroup.  Leaves the scan at the last 64 sequences (with up
// to 64 of them: at all).
__device__ __forceinline__ int kv_units_each(const KvCache& c, const KvAttention& a, const KvShare& sh, KvScan& s) {
  int total = 0;
  for (int base = 0; base < a.seqs; base += 64) {
    kv_scan(c, a, sh.rows, base, total, s);
    total = s.after;
  }
  return (total + sh.groups - 1) / sh.groups;
}

// ----------------------------------------------------------------- few rows
//
// Up to 16 MT rows of a pair share a run of its keys.  Each of a workgroup's
// four waves walks its own tiles of 32 keys with its own running maximum, and
// the four meet at the end of the run.
//
// Per tile a lane holds 64 NG / 4 values of key l % 16 (+ 16): it loads their
// codes with one wide load and uses them in place as rows of the matrix
// product S^T = K Q^T (16 x 16 x 32), whose k order is free as long as the
// query fragments follow it.  Lane l then holds the scores of row l % 16 for
// keys 4 (l / 16) + i, which is the operand layout of the second product
// O^T = V^T P^T, so probabilities never leave their lane.  Values are decoded
// the same way, written to the wave's own LDS as float16 and read back
// transposed (ds_read_b64_tr_b16); nothing in the loop waits for another wave.
//
// Bound by memory while contexts are long: 4 x 131072 keys, 8 heads of 128,
// 604 MB, 112 - 120 us with the join, 5.0 - 5.4 TB/s (vector units busy 58 %
// of the time, LDS 31 %, matrix cores 12 %).  Shorter ones show the start, a
// chain of four dependent loads (lengths, page number, codes; queries beside
// them), about 7 us, and the join: 32 contexts of up to 8192, 166 MB, 49 us,
// 3.4 TB/s.  A whole tile in flight a wave and three workgroups a CU cover the
// latency (1 or 2 a CU: 81 and 58 us).  With 17 to 32 rows one workgroup a CU
// has its registers, and that latency shows: 8 x 30000 keys, 4 heads of 128, 16
// rows 45 us, 24 rows 78, 32 rows 80.

constexpr int few_row_bytes(int NG) { return 128 * NG + 32; }  // a key's values in LDS: +32 spreads the banks
constexpr int kFewPages = 512;  // pages staged at a time
constexpr uint64_t kNoPage = ~0ull;

// Waves per SIMD, and workgroups per CU, that an instance's registers are cut
// to.  What the compiler then spills, vector registers by <dim / 64, row tiles,
// float16 a query element>: <1, 1, 1> 9, <2, 1, 1> 2, <1, 2, 1> 17, <4, 1, 1> 2,
// <4, 2, 1> 37, <4, 2, 2> 175, the others none; for heads that are no whole 64s
// up to 25 more.  All spill 148 to 228 scalar registers into vector lanes.
constexpr int few_occupancy(int NG, int MT, int SPLIT) {
  const int size = NG * MT * SPLIT;
  return size == 1 ? 4 : size == 2 ? 3 : size <= 4 && MT == 1 ? 2 : 1;
}

template <int NG, int MT, int SPLIT, bool EXACT>
__global__ void __launch_bounds__(256, few_occupancy(NG, MT, SPLIT))
kv_few_kernel(KvCache c, KvAttention a, KvShare sh, int dt, bool q_vec) {
  constexpr int DP = 64 * NG, STEPS = 2 * NG, DB = DP / 16, RB = few_row_bytes(NG);
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ float stat_m[kFewWaves][16 * MT], stat_l[kFewWaves][16 * MT];
  __shared__ uint32_t no_numbers[2][16 * MT];  // per row, of this run and the next one: groups that are NaN
  uint64_t* page_of = reinterpret_cast<uint64_t*>(lds + kFewWaves * kFewTile * RB);  // of this run and of the next one
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, quarter = lane >> 4;
  uint8_t* mine = lds + wave * kFewTile * RB;
  const int g0 = NG * quarter;
  const float value_factor = global_decode(c.global_v);
  const float key_factor = a.scale * kLog2e * global_decode(c.global_k);

  // A run: some of the keys of one pair.
  struct Run {
    KvRange rg;
    int b, head, begin, end, pages;  // pages: staged page numbers
    bool whole;
  };
  // Keys whose page numbers are staged at a time.
  const int span = (int)min((int64_t)1 << 30, (int64_t)(kFewPages - 2) * c.page_size / kFewStep * kFewStep);
  auto pages_of = [&](int from, int end) {
    return from < end ? (int)kv_div(from + min(end - from, span) - 1, c.page_div) - (int)kv_div(from, c.page_div) + 1 : 0;
  };
  KvScan scan;
  int unit = 0, last_unit = 0, base = 0, before = 0;
  // The run that begins with `unit`; `scan` holds the 64 sequences from `base`.
  auto next_run = [&](KvScan& scan, Run& r) {
    if (unit >= last_unit) return false;
    while (unit >= scan.after) {
      base += 64;
      before = scan.after;
      if (base >= a.seqs) {  // past the last unit
        last_unit = unit;
        return false;
      }
      kv_scan(c, a, sh.rows, base, before, scan);
    }
    const int at_lane = __builtin_amdgcn_readfirstlane(63 - __builtin_clzll(__ballot(scan.units > 0 && scan.first <= unit)));
    r.b = base + at_lane;
    r.rg = kv_range_of(scan, at_lane);
    const int pair_units = __builtin_amdgcn_readlane(scan.units, at_lane);
    const int inside = unit - __builtin_amdgcn_readlane(scan.first, at_lane);
    r.head = __builtin_amdgcn_readfirstlane(inside / pair_units);
    const int off = inside - r.head * pair_units;
    const int take = min(pair_units - off, last_unit - unit);
    unit += take;
    r.whole = take == pair_units;
    r.begin = r.rg.lo + off * kFewStep;
    r.end = min(r.rg.hi, r.begin + take * kFewStep);
    r.pages = __builtin_amdgcn_readfirstlane(pages_of(r.begin, r.end));
    return true;
  };
  Run now, next;
  next.pages = next.begin = 0;
  bool more_runs = false;
  if (sh.sums == nullptr) {  // one workgroup a pair
    now.b = __builtin_amdgcn_readfirstlane(blockIdx.x / c.heads);
    now.head = blockIdx.x - now.b * c.heads;
    now.rg = kv_range(a, now.b, 0, sh.rows);
    now.whole = true;
    now.begin = now.rg.lo;
    now.end = now.rg.hi;
    now.pages = pages_of(now.begin, now.end);
    if (now.rg.n == 0) return;
  } else {
    const int each = kv_units_each(c, a, sh, scan);
    if (a.seqs > 64) kv_scan(c, a, sh.rows, 0, 0, scan);
    unit = __builtin_amdgcn_readfirstlane((int)blockIdx.x * each);
    last_unit = unit + __builtin_amdgcn_readfirstlane(each);
    if (!next_run(scan, now)) return;
    more_runs = next_run(scan, next);
  }

  KvRaw<SPLIT> raw[MT][STEPS];
  auto load_queries = [&](const Run& r) {
    const int rows = r.rg.n * a.groups;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int i = 16 * m + col;  // this lane's row
      const int qi = kv_div(i, a.group_div);
      const int64_t at = (int64_t)(r.rg.first + qi) * a.q_token + (r.head * a.groups + (i - qi * a.groups)) * a.q_head;
#pragma unroll
      for (int t = 0; t < STEPS; ++t) {
        const int d = 16 * NG * quarter + 8 * t;
        raw[m][t] = kv_load_query<SPLIT>(a, q_vec, at + d, i < rows && d < c.dim);
      }
    }
  };
  // Where this head's codes start in the i-th page from that of key `from` on.
  auto page_at = [&](const Run& r, int from, int i) {
    const int p = a.page_table[r.b * a.table_stride + kv_div(from, c.page_div) + i];
    return p >= 0 && p < c.pages ? kv_page_start(kv_place(c, r.head), p) : kNoPage;
  };

  // A tile's keys are loaded once the last tile's are used up, its values
  // likewise: two thirds of a tile's time ahead, in the same registers.
  KvGroups<NG, EXACT> kt[2], vt[2];
  uint64_t row[2];       // this lane's rows of the tile that is being loaded
  bool there[2];
  uint32_t exists = 0u;  // which of its 32 keys do
  int buf = 0, to = 0, staged = 0;
  int page[2], off[2];   // of this lane's keys, from the span's first page
  const KvStep step = kv_step(c, kFewStep);
  auto locate = [&](int at) {
    exists = 0u;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint64_t start = page_of[buf * kFewPages + min(page[u], staged - 1)];
      there[u] = (start != kNoPage) & (at + 16 * u + col < to);
      row[u] = start + kv_row_start<NG, EXACT>(off[u], c.dim);
      exists |= (uint32_t)(__ballot(there[u]) & 0xFFFFu) << (16 * u);
      kv_advance(step, c.page_size, page[u], off[u]);
    }
  };
  auto load = [&](const uint8_t* codes, const uint8_t* scales, KvGroups<NG, EXACT>(&x)[2]) {
#pragma unroll
    for (int u = 0; u < 2; ++u) x[u] = kv_load<NG, EXACT, true>(codes, scales, row[u], c.dim, g0, there[u]);
  };
  // This wave's first tile of the keys from `from` on, whose page numbers are staged.
  auto begin_span = [&](const Run& r, int from) {
    to = from + min(r.end - from, span);
    staged = pages_of(from, r.end);
    const int first = from + wave * kFewTile;
    if (first < to) {
      const int p0 = kv_div(from, c.page_div);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int j = first + 16 * u + col;
        page[u] = (int)kv_div(j, c.page_div);
        off[u] = j - page[u] * c.page_size;
        page[u] -= p0;
      }
      locate(first);
      load(c.k_codes, c.k_scales, kt);
      load(c.v_codes, c.v_scales, vt);
    }
  };

  // Loads in the order of their use, and all that the next run needs before
  // this one's keys: a run that follows another begins with its first tile on
  // the way while the last one's sums are still being put together.
  load_queries(now);
  for (int i = threadIdx.x; i < now.pages + next.pages; i += 256) {
    const bool second = i >= now.pages;
    page_of[second ? kFewPages + i - now.pages : i] =
        second ? page_at(next, next.begin, i - now.pages) : page_at(now, now.begin, i);
  }
  if (threadIdx.x < 32 * MT) (&no_numbers[0][0])[threadIdx.x] = 0u;
  lds_barrier();
  begin_span(now, now.begin);

  for (;;) {
  const KvRange rg = now.rg;
  const int head = now.head, begin = now.begin, end = now.end;
  const int rows = rg.n * a.groups;

  // row `col` of each row tile, values 16 NG quarter ..
  f16x8 q[MT][SPLIT][STEPS];
  float factor[MT];
  int see_lo[MT], see_hi[MT];  // keys that row `col` sees
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float top = 0.0f;
#pragma unroll
    for (int t = 0; t < STEPS; ++t) top = fmaxf(top, kv_query_top<SPLIT>(raw[m][t], dt));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int e = kv_row_exponent(top);
    factor[m] = __builtin_ldexpf(key_factor, e);
#pragma unroll
    for (int t = 0; t < STEPS; ++t) kv_query_halves<SPLIT>(raw[m][t], dt, e, 1.0f, q[m][0][t], q[m][SPLIT - 1][t]);
    const int r = 16 * m + col;
    const int pos = rg.context - rg.n + (int)kv_div(r, a.group_div);
    see_hi[m] = r >= rows ? 0 : a.causal ? min(rg.hi, pos + 1) : rg.hi;
    see_lo[m] = kv_window_begin(a, pos);
  }
  // keys that every row sees: [all_lo, all_hi)
  int all_hi = rg.hi, all_lo = 0;
  if (a.causal) {
    all_hi = min(rg.hi, rg.context - rg.n + 1);
    all_lo = kv_window_begin(a, rg.context - 1);
  }

  f32x4 acc[MT][DB];
  float m_run[MT], sub[MT], l_run[MT];
  bool large = false;  // some row has had a maximum beyond kBig
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    m_run[m] = kNone;
    sub[m] = -kBias;
    l_run[m] = 0.0f;
#pragma unroll
    for (int d = 0; d < DB; ++d) acc[m][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  for (int from = begin; from < end;) {
  for (int tile = from + wave * kFewTile; tile < to; tile += kFewStep) {
    const uint32_t live = exists;
    const bool more = tile + kFewStep < to;
    if (more) locate(tile + kFewStep);

    // scores
    f32x4 s[MT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f16x8 kf[STEPS];
      kv_values<NG, EXACT>(kt[u], kf);
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
    if (more) load(c.k_codes, c.k_scales, kt);
    // values into LDS
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      f16x8 vf[STEPS];
      kv_values<NG, EXACT>(vt[u], vf);
#pragma unroll
      for (int t = 0; t < STEPS; ++t)
        *reinterpret_cast<f16x8*>(mine + (16 * u + col) * RB + 32 * NG * quarter + 16 * t) = vf[t];
    }
    if (more) load(c.v_codes, c.v_scales, vt);
    // probabilities
    const bool masked = live != 0xFFFFFFFFu || tile < all_lo || tile + kFewTile > all_hi;
    float x[MT][8], low = 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[m][i] = s[m][i >> 2][i & 3] * factor[m];
      if (masked && m == 0 && rg.n > 1) {
        // A value that is no number must not reach the rows that do not see
        // its key (0 times it is NaN).  Those that do are noted for the end of
        // the run, and the tile is left without it.  (The heads of one query see
        // the same keys.)  NaN put into the sums here instead costs heads of 256
        // with 17 to 32 rows their registers: 8 x up to 8000, 86 us against 53.
        uint8_t* const held = mine + opaque(col) * RB + 32 * NG * opaque(quarter);  // this lane's groups
        bool any = false;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const _Float16 v = *reinterpret_cast<const _Float16*>(held + 16 * u * RB + 32 * g);
            any |= v != v;
          }
        if (__any(any)) {
#pragma unroll 1
          for (int i = 0; i < 2 * NG; ++i) {
            const int u = i / NG, g = i - u * NG;
            f16x8* at = reinterpret_cast<f16x8*>(held + 16 * u * RB + 32 * g);
            const bool own = at[0][0] != at[0][0];
            for (uint64_t lanes = __ballot(own); lanes; lanes &= lanes - 1) {
              const int l = __builtin_ctzll(lanes), key = tile + 16 * u + (l & 15), group = NG * (l >> 4) + g;
#pragma unroll
              for (int mm = 0; mm < MT; ++mm)
                if (quarter == 0 && key >= see_lo[mm] && key < see_hi[mm])
                  atomicOr(&no_numbers[buf][16 * mm + col], 1u << group);
            }
            if (own) at[0] = at[1] = f16x8{0, 0, 0, 0, 0, 0, 0, 0};
          }
        }
      }
      if (masked) {
        const int h = 4 * opaque(quarter);
        const int lo = see_lo[m] - tile - h, hi = see_hi[m] - tile - h;
        const uint32_t have = live >> h;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = 16 * (i >> 2) + (i & 3);
          x[m][i] = (((have >> key) & 1u) & (key >= lo) & (key < hi)) ? x[m][i] : kNone;
        }
      }
      float top = fmaxf(x[m][0], x[m][1]);
#pragma unroll
      for (int i = 2; i < 8; i += 2) top = max3(top, x[m][i], x[m][i + 1]);
      if (__any(top > m_run[m] + kLag)) {  // rare once a row has met its large scores
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m_run[m], top);
        const float keep = m_run[m] == kNone ? 0.0f : __builtin_amdgcn_exp2f(m_run[m] - next);
        m_run[m] = next;
        sub[m] = next == kNone ? -kBias : next - kBias;
        large |= __any(__builtin_fabsf(sub[m]) > kBig) != 0;
        l_run[m] *= keep;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[m][d][i] *= keep;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[m][i] -= sub[m];
      if (large) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[m][i] = kv_most(x[m][i]);
      }
#pragma unroll
      for (int i = 0; i < 8; i += 2) low = min3(low, x[m][i], x[m][i + 1]);
    }
    // output: 16 values (rows) of V^T at a time, keys 4 quarter + 16 u + (0 .. 3) a lane
    f16x8 p[MT][SPLIT];
    auto weight = [&](int m, int i, float w) {
      p[m][0][i] = (_Float16)w;
      if constexpr (SPLIT == 2) p[m][SPLIT - 1][i] = (_Float16)((w - (float)(_Float16)w) * kRest);
    };
    auto values_of = [&](int d) {
      const uint8_t* at = mine + (4 * quarter + (col >> 2)) * RB + 32 * d + 8 * (col & 3);
      return kv_read_transposed(at, at + 16 * RB);
    };
    if (__any(low < kSmall)) {  // the bands of small weights, then the rest
      float shift = kShift, down = kDown;
      bool any = false;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) any |= (x[m][i] < kSmall) & (x[m][i] > kNone);
      for (int band = 1; band < kBands && __any(any); ++band) {
        any = false;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float t = x[m][i] + shift;
            const bool lower = (t < kSmall) & (band < kBands - 1);
            const bool in = (t < kSmall + kShift) & !lower;
            const float w = in ? __builtin_amdgcn_exp2f(t) : 0.0f;
            l_run[m] += w * down;
            any |= lower & (t > kNone);
            weight(m, i, w);
          }
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          const f16x8 vf = values_of(d);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int e = SPLIT - 1; e >= 0; --e)
              sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(e ? kv_rest_values(vf) : vf, p[m][e], sum, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][d][i] += sum[i] * down;
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        shift += kShift;
        down *= kDown;
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[m][i] = x[m][i] < kSmall ? kNone : x[m][i];
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float w = __builtin_amdgcn_exp2f(x[m][i]);
        l_run[m] += w;
        weight(m, i, w);
      }
#pragma unroll
    for (int d = 0; d < DB; ++d) {
      const f16x8 vf = values_of(d);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = SPLIT - 1; e >= 0; --e)
          acc[m][d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(e ? kv_rest_values(vf) : vf, p[m][e], acc[m][d], 0, 0, 0);
    }
  }
  from = to;
  if (from < end) {
    lds_barrier();
    for (int i = threadIdx.x; i < pages_of(from, end); i += 256) page_of[buf * kFewPages + i] = page_at(now, from, i);
    lds_barrier();
    begin_span(now, from);
  }
  }
  if (more_runs) {  // the next run's first tile
    buf ^= 1;
    begin_span(next, next.begin);
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
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (m > 0) lds_barrier();
    float* own = reinterpret_cast<float*>(mine) + col * (DP + 4);
#pragma unroll
    for (int d = 0; d < DB; ++d) *reinterpret_cast<f32x4*>(own + 16 * d + 4 * quarter) = acc[m][d];
    lds_barrier();
    for (int i = threadIdx.x; i < 16 * (DP / 4); i += 256) {
      const int rr = i / (DP / 4), d = 4 * (i - rr * (DP / 4));
      const int r = 16 * m + rr;
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
      // (buf is the next run's already, if there is one)
      if (rg.n > 1 && (no_numbers[more_runs ? buf ^ 1 : buf][r] >> (d >> 4) & 1u)) v[0] = v[1] = v[2] = v[3] = kNaN;
      const int qi = kv_div(r, a.group_div);
      const int64_t row = (int64_t)(rg.first + qi) * a.query_heads + head * a.groups + (r - qi * a.groups);
      if (now.whole) {
        const float by = l == 0.0f ? 0.0f : value_factor / l;  // a NaN stays one
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= by;
        kv_store4(dt, a.out, row * c.dim + d, v);
        if (d == 0 && a.lse) a.lse[row] = l == 0.0f ? kNone : (mt - kBias + __builtin_log2f(l)) * kLn2;
      } else {
        const int64_t at = ((int64_t)blockIdx.x + now.b * c.heads + head) * sh.rows + r;
        kv_store4<kF32>(sh.sums, at * c.dim + d, v);
        if (d == 0) *reinterpret_cast<f32x2*>(sh.stats + 2 * at) = f32x2{mt, l};
      }
    }
  }
  if (!more_runs) return;
  now = next;
  load_queries(now);
  // (scanned anew: kept, the scan would cost the loop a dozen registers)
  more_runs = unit < last_unit;
  if (more_runs) {
    KvScan again;
    kv_scan(c, a, sh.rows, base, before, again);
    more_runs = next_run(again, next);
    if (more_runs)
      for (int i = threadIdx.x; i < next.pages; i += 256) page_of[(buf ^ 1) * kFewPages + i] = page_at(next, next.begin, i);
  }
  lds_barrier();  // the sums have been read and the next page numbers are there
  if (threadIdx.x < 16 * MT) no_numbers[buf ^ 1][threadIdx.x] = 0u;  // (for the run after this one)
  }
}

// ----------------------------------------------------------------- many rows
//
// 128 rows of a (sequence, kv head) per workgroup, 32 per wave, against tiles
// of keys and values that the workgroup decodes once into LDS as float16 for
// all of them: S^T = K Q^T and O^T = V^T P^T on 32 x 32 x 16 products, the
// probabilities again staying in the lane that computed their scores.  Two
// buffers: while a tile is multiplied the next one's codes (loaded a tile
// earlier) are decoded into the other, and the loads of the one after it are
// under way; one barrier a tile.  Rows of LDS are padded so that the 16-byte
// reads of K and the transposing reads of V touch every bank once.
//
// No unit bounds it alone.  4096 causal queries over as many keys, 32 heads of
// 128: vector units busy 48 % of the time, LDS 37 % (its bank conflicts 14 %),
// matrix cores 28 %; a wave waits 28 % of its time, and 26 % more for its turn
// to issue.  Two waves a SIMD, in step by a barrier a tile, do not cover one
// another better than that.  By hand: the 16 scores a lane holds of a 32 x 32
// tile take 512 cycles of the matrix cores and about 320 of the vector units
// (each an exponential, 8.6, a multiply-add, 4.9, half a conversion to float16,
// 3.7, maximum and sum), decoding besides, and the four waves' 16 KB each of
// fragments of a tile 512 cycles of the CU's LDS.  187 - 203 us by the machine,
// 680 - 735 TFLOP/s; up to 1023 queries each of 5 sequences over up to 9001
// keys: 421 - 453 us, 675 - 725 TFLOP/s; a large float16 matrix product reaches
// 1324.  256 rows and 8 waves share the decoding further, but not the reads of
// fragments, and leave one workgroup a CU: 192 against 198 us and 470 against
// 440 (kernels of the time).  float32 queries: one workgroup a CU for its
// registers, and four products for one.
//
// Too few workgroups for the GPU split the keys further (KvChunks).
constexpr int kManyRows = 128;
constexpr int many_tile(int NG) { return NG <= 2 ? 64 : 32; }
constexpr int many_k_row(int NG) { return 128 * NG + 16; }
constexpr int many_v_row(int NG) { return 128 * NG + 32; }
constexpr int many_lds(int NG) { return 2 * many_tile(NG) * (many_k_row(NG) + many_v_row(NG)); }

struct KvChunks {
  int chunk, splits;  // keys per chunk (a multiple of 64), chunks per tile of rows
  int row_tiles;      // of a sequence and kv head
  float* sums;        // [tokens][query_heads][splits][dim], times 2^kBias
  float* stats;       // [tokens][query_heads][splits][2]: maximum (log2), sum
};

template <int NG, int SPLIT, bool EXACT>
__global__ void __launch_bounds__(256, (NG * SPLIT <= 2 ? 2 : 1))
kv_many_kernel(KvCache c, KvAttention a, KvChunks sp, int dt, bool q_vec) {
  constexpr int DP = 64 * NG, TILE = many_tile(NG), SUB = TILE / 32, STEPS = DP / 16, DB = DP / 32;
  constexpr int KROW = many_k_row(NG), VROW = many_v_row(NG), BUF = TILE * (KROW + VROW);
  constexpr int NEAR = NG * SPLIT <= 4 ? kNearBands : 1;  // (more registers would be spilled)
  constexpr bool BOTH = TILE == 64;  // every thread decodes keys and values; else half of them each
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  // four lanes a key: which keys of a buffer exist, with values that are
  // numbers; where some do not, also which exist and which have other values
  __shared__ uint64_t fine[2][4], exists[2][4], odd[2][4];
  __shared__ uint32_t odd_groups[2][256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 31, half = lane >> 5;
  const int b = blockIdx.y;
  int x = blockIdx.x;
  const int split = x % sp.splits;
  x /= sp.splits;
  const int head = x % c.heads;
  const int row0 = (sp.row_tiles - 1 - x / c.heads) * kManyRows;  // the longest ranges first
  const KvRange rg = kv_range(a, b, row0, kManyRows);
  const int rows = rg.n * a.groups;
  if (row0 >= rows) return;
  const int keys = max(0, rg.hi - rg.lo), before = min(keys, split * sp.chunk);
  const int begin = rg.lo + before, end = begin + min(keys - before, sp.chunk);
  if (begin >= end && split > 0) return;  // the first chunk's workgroup answers for rows that see nothing

  // what this thread decodes: NG groups of one key (and of its value)
  const int key_of = BOTH ? threadIdx.x >> 2 : (threadIdx.x & 127) >> 2;
  const bool second = !BOTH && threadIdx.x >= 128;
  const int g0 = NG * (threadIdx.x & 3);
  // The page number of this thread's key, as it stands in the table (checked
  // when it is used, a tile later: nothing may wait for it here).  Past the
  // end the last key's.
  const KvStep step = kv_step(c, TILE);
  const int32_t* table = a.page_table + b * a.table_stride;
  const int last_page = begin < end ? (int)kv_div(end - 1, c.page_div) : 0;
  int page_l = kv_div(begin + key_of, c.page_div);  // page and offset of the next tile to look up
  int off_l = begin + key_of - page_l * c.page_size;
  int page_d = page_l, off_d = off_l;               // .. and to load
  auto lookup = [&]() {
    const int p = table[min(page_l, last_page)];
    kv_advance(step, c.page_size, page_l, off_l);
    return p;
  };
  KvGroups<NG, EXACT> kt, vt;
  int live = 0;
  const KvPlace place = kv_place(c, head);
  auto load = [&](int tile, int page) {
    const int j = tile + key_of;
    const bool there = (page >= 0) & (page < c.pages) & (j < end);
    live = there | (j >= end);  // past the end every row's mask holds
    const uint64_t row = kv_page_start(place, page) + kv_row_start<NG, EXACT>(off_d, c.dim);
    kv_advance(step, c.page_size, page_d, off_d);
    if constexpr (BOTH) {
      kt = kv_load<NG, EXACT, false>(c.k_codes, c.k_scales, row, c.dim, g0, there);
      vt = kv_load<NG, EXACT, false>(c.v_codes, c.v_scales, row, c.dim, g0, there);
    } else {
      kt = kv_load<NG, EXACT, false>(second ? c.v_codes : c.k_codes, second ? c.v_scales : c.k_scales, row, c.dim, g0,
                                     there);
    }
  };
  // Decodes piece i (8 values) of what was loaded and writes it to buffer `buf`.
  constexpr int PIECES = (BOTH ? 4 : 2) * NG;
  auto store_piece = [&](int buf, int i) {
    const bool of_v = BOTH ? i >= 2 * NG : second;
    const KvGroups<NG, EXACT>& x = BOTH && i >= 2 * NG ? vt : kt;
    const int w = BOTH && i >= 2 * NG ? i - 2 * NG : i;
    uint8_t* at = lds + buf * BUF + (of_v ? TILE * KROW + key_of * VROW : key_of * KROW) + 32 * g0 + 16 * w;
    *reinterpret_cast<f16x8*>(at) = kv_decode8(x.w[w], kv_scale_of(x, w >> 1));
  };
  // A value that is no number must not reach the rows that do not see its key
  // (0 times it is NaN): it is decoded as 0, and the rows that do get their
  // NaN from these notes.
  auto store_flags = [&](int buf) {
    const uint32_t bad = BOTH ? kv_no_numbers(vt) : second ? kv_no_numbers(kt) : 0u;
    const uint64_t bits = __ballot((live != 0) & (bad == 0u));
    if (lane == 0) fine[buf][wave] = bits;
    if (~bits) {
      const uint64_t there = __ballot(live != 0), others = __ballot(bad != 0u);
      if (lane == 0) {
        exists[buf][wave] = there;
        odd[buf][wave] = others;
      }
      odd_groups[buf][opaque((int)threadIdx.x)] = bad;
      if constexpr (BOTH) kv_drop(vt, bad);
      else kv_drop(kt, bad);
    }
  };
  int page = 0, page2 = 0;
  if (begin < end) {
    page = lookup();
    page2 = lookup();
  }

  // queries: row `col` of this wave's 32
  const int r = row0 + 32 * wave + col;
  const bool row_live = r < rows;
  const int qi = kv_div(r, a.group_div), qh = head * a.groups + r - qi * a.groups;
  f16x8 q[SPLIT][STEPS];
  float factor;
  {
    const int64_t at = (int64_t)(rg.first + qi) * a.q_token + qh * a.q_head;
    KvRaw<SPLIT> raw[STEPS];
    float top = 0.0f;
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      const int d = 16 * t + 8 * half;
      raw[t] = kv_load_query<SPLIT>(a, q_vec, at + d, row_live && d < c.dim);
      top = fmaxf(top, kv_query_top<SPLIT>(raw[t], dt));
    }
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int e = kv_row_exponent(top);
    // The masks and extremes below are those of the bare products, so the
    // factor has to be positive.  Its sign (or NaN) goes into the query.  A
    // factor of 0, of a global scale of 0 or of a row so small that it
    // underflows, becomes the smallest normal number: scores stay below 2^-90,
    // as good as 0, and those that are masked stay -inf.
    factor = __builtin_ldexpf(a.scale * kLog2e * global_decode(c.global_k), e);
    const float sign = factor < 0.0f ? -1.0f : factor != factor ? factor : 1.0f;
    factor = fmaxf(__builtin_fabsf(factor), 0x1p-126f);
#pragma unroll
    for (int t = 0; t < STEPS; ++t) kv_query_halves<SPLIT>(raw[t], dt, e, sign, q[0][t], q[SPLIT - 1][t]);
  }
  const int pos = rg.context - rg.n + qi;
  const int see_hi = !row_live ? 0 : a.causal ? min(end, pos + 1) : end;
  const int see_lo = kv_window_begin(a, pos);
  // keys that every row of this wave sees
  int all_lo = 0, all_hi = end;
  if (a.causal) {
    const int w0 = min(row0 + 32 * wave, rows - 1), base = rg.context - rg.n;
    all_hi = min(end, base + (int)kv_div(w0, a.group_div) + 1);
    all_lo = kv_window_begin(a, base + (int)kv_div(min(w0 + 31, rows - 1), a.group_div));
  }

  f32x16 acc[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
  float m_run = kNone, sub = -kBias, l_run = 0.0f;
  uint64_t large = 0;  // lanes whose rows have had a maximum beyond kBig

  if (begin < end) {
    load(begin, page);
    page = page2;
    page2 = lookup();
    store_flags(0);
#pragma unroll
    for (int i = 0; i < PIECES; ++i) store_piece(0, i);
    load(begin + TILE, page);
    page = page2;
    page2 = lookup();
    lds_barrier();
  }
  int buf = 0;
  for (int tile = begin; tile < end; tile += TILE, buf ^= 1) {
    const uint8_t* kb = lds + buf * BUF;
    const uint8_t* vb = kb + TILE * KROW;
    // Scores.  The order is fixed by hand: K fragments kAhead products ahead,
    // and the decoding of the next tile between the products.
    f32x16 s[SUB];
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[u][i] = 0.0f;
    uint64_t have = ~0ull;
#pragma unroll
    for (int i = 0; i < 4; ++i) have &= fine[buf][i];
    if (!BOTH) store_flags(buf ^ 1);
    // largest and smallest scores, in four chains; those of the first 32 keys
    // while the others' products run
    float top4[4], low4[4];
    auto extremes = [&](int u, int k, bool begin_chain) {
      const float a0 = s[u][4 * k], a1 = s[u][4 * k + 1], a2 = s[u][4 * k + 2], a3 = s[u][4 * k + 3];
      top4[k] = max3(begin_chain ? fmaxf(a0, a1) : max3(top4[k], a0, a1), a2, a3);
      low4[k] = min3(begin_chain ? fminf(a0, a1) : min3(low4[k], a0, a1), a2, a3);
    };
    {
      constexpr int N = SUB * STEPS, kAhead = 3;
      f16x8 kf[kAhead + 1];
      auto fetch = [&](int n) {
        kf[n % (kAhead + 1)] = *reinterpret_cast<const f16x8*>(kb + (32 * (n / STEPS) + col) * KROW +
                                                               32 * (n % STEPS) + 16 * half);
      };
#pragma unroll
      for (int n = 0; n < kAhead; ++n) fetch(n);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n + kAhead < N) fetch(n + kAhead);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = SPLIT - 1; e >= 0; --e)
          s[n / STEPS] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf[n % (kAhead + 1)], q[e][n % STEPS], s[n / STEPS], 0, 0, 0);
        if (BOTH && n * PIECES / N == 2 * NG - 1 && (n + 1) * PIECES / N == 2 * NG) store_flags(buf ^ 1);  // ahead of values
        // (after the last tile: what is decoded then is not read)
        if (n * PIECES / N != (n + 1) * PIECES / N) store_piece(buf ^ 1, n * PIECES / N);
        if (SUB == 2 && n >= STEPS + 2 && n < STEPS + 4) {
          extremes(0, 2 * (n - STEPS - 2), true);
          extremes(0, 2 * (n - STEPS - 2) + 1, true);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    load(tile + 2 * TILE, page);  // (past the end: nothing)
    page = page2;
    page2 = lookup();
    {
      const bool edge = tile < all_lo || tile + TILE > all_hi, holes = have != ~0ull;
      if (edge) {
        const int h = opaque(half);
        const int lo = see_lo - tile - 4 * h, hi = see_hi - tile - 4 * h;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = 32 * u + 8 * (i >> 2) + (i & 3);
            s[u][i] = ((key >= lo) & (key < hi)) ? s[u][i] : kNone;
          }
      }
      if (holes) {  // pages that are not there, values that are no numbers
        const int h = opaque(half);
        const int lo = opaque(see_lo), hi = opaque(see_hi);
        uint64_t there[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const bool noted = fine[buf][w] != ~0ull;
          there[w] = noted ? exists[buf][w] : ~0ull;
          for (uint64_t lanes = noted ? odd[buf][w] : 0ull; lanes; lanes &= lanes - 1) {
            const int thread = 64 * w + __builtin_ctzll(lanes), key = tile + ((BOTH ? thread : thread & 127) >> 2);
            const uint32_t groups = odd_groups[buf][thread];
            if (key >= lo && key < hi)
#pragma unroll
              for (int i = 0; i < 2 * DB; ++i) {
                const int g = i - NG * (thread & 3);
                if (g >= 0 && g < NG && (groups >> (8 * g + 7) & 1u))
#pragma unroll
                  for (int j = 0; j < 8; ++j) acc[i >> 1][8 * (i & 1) + j] = kNaN;
              }
          }
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = 8 * (i >> 2) + 4 * h + (i & 3);  // of this half tile
            if (!(there[2 * u + (i >> 3)] >> (4 * (key & 15)) & 1)) s[u][i] = kNone;
          }
      }
      if (SUB == 1 || edge || holes) {
#pragma unroll
        for (int k = 0; k < 4; ++k) extremes(0, k, true);
      }
      if constexpr (SUB == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) extremes(SUB - 1, k, false);
      }
      // (the factor is positive)
      float top = max3(fmaxf(top4[0], top4[1]), top4[2], top4[3]) * factor;
      const float low = min3(fminf(low4[0], low4[1]), low4[2], low4[3]) * factor;
      if (__any(top > m_run + kLag)) {
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float next = fmaxf(m_run, top);
        const float keep = m_run == kNone ? 0.0f : __builtin_amdgcn_exp2f(m_run - next);
        m_run = next;
        sub = next == kNone ? -kBias : next - kBias;
        large |= __ballot(__builtin_fabsf(sub) > kBig);
        l_run *= keep;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[d][i] *= keep;
      }
      // values 32 d .. of the 16 keys of group g, transposed
      auto values_of = [&](int g, int d) {
        const uint8_t* at = vb + (16 * g + 4 * half + ((lane & 15) >> 2)) * VROW + 64 * d +
                            32 * ((lane >> 4) & 1) + 8 * (lane & 3);
        return kv_read_transposed(at, at + 8 * VROW);
      };
      f16x8 p[SUB][2][SPLIT];
      auto weight = [&](int u, int i, float w) {
        p[u][i >> 3][0][i & 7] = (_Float16)w;
        if constexpr (SPLIT == 2) p[u][i >> 3][SPLIT - 1][i & 7] = (_Float16)((w - (float)(_Float16)w) * kRest);
      };
      float by = factor, below = sub;  // a weight's exponent is s * by - below
      if (__ballot(low - sub < kSmall) | large) {  // the bands of small weights, then the rest
        if (large) {
          const float f = opaque(factor), less = opaque(sub);
          const bool big = __builtin_fabsf(less) > kBig;
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
#pragma clang fp contract(off)
              const float x = s[u][i] * f;
              s[u][i] = big ? kv_most(x - less) : s[u][i];
            }
          by = big ? 1.0f : by;
          below = big ? 0.0f : below;
        }
        const float f = opaque(by), less = opaque(below);
        float shift = kShift, up = kUp, down = kDown;
        bool any = false;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float t = __builtin_fmaf(s[u][i], f, -less);
            any |= (t < kSmall) & (t > kNone);
          }
        int band = 1;
        for (; band < NEAR && __any(any); ++band) {  // the output scaled along: few instructions
          any = false;
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float t = __builtin_fmaf(s[u][i], f, -less) + shift;
              const bool lower = t < kSmall;
              const bool in = (t < kSmall + kShift) & !lower;
              const float w = in ? __builtin_amdgcn_exp2f(t) : 0.0f;
              l_run += w * down;
              any |= lower & (t > kNone);
              weight(u, i, w);
            }
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] *= up;
#pragma unroll
          for (int n = 0; n < 2 * SUB * DB; ++n) {
            const f16x8 vf = values_of(n / DB, n % DB);
#pragma unroll
            for (int e = SPLIT - 1; e >= 0; --e)
              acc[n % DB] = __builtin_amdgcn_mfma_f32_32x32x16_f16(e ? kv_rest_values(vf) : vf, p[n / DB >> 1][n / DB & 1][e],
                                                                   acc[n % DB], 0, 0, 0);
          }
#pragma unroll
          for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[d][i] *= down;
          shift += kShift;
          up *= kUp;
          down *= kDown;
        }
        for (; band < kBands && __any(any); ++band) {  // where that would pass float32: sums apart
          any = false;
#pragma unroll
          for (int g = 0; g < 2 * SUB; ++g) {  // (16 keys at a time: few registers)
            f16x8 w8[SPLIT];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float t = __builtin_fmaf(s[g >> 1][8 * (g & 1) + j], f, -less) + shift;
              const bool lower = (t < kSmall) & (band < kBands - 1);
              const bool in = (t < kSmall + kShift) & !lower;
              const float w = in ? __builtin_amdgcn_exp2f(t) : 0.0f;
              l_run += w * down;
              any |= lower & (t > kNone);
              w8[0][j] = (_Float16)w;
              if constexpr (SPLIT == 2) w8[SPLIT - 1][j] = (_Float16)((w - (float)(_Float16)w) * kRest);
            }
#pragma unroll
            for (int d = 0; d < DB; ++d) {
              const f16x8 vf = values_of(g, d);
              f32x16 sum;
#pragma unroll
              for (int i = 0; i < 16; ++i) sum[i] = 0.0f;
#pragma unroll
              for (int e = SPLIT - 1; e >= 0; --e)
                sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(e ? kv_rest_values(vf) : vf, w8[e], sum, 0, 0, 0);
#pragma unroll
              for (int i = 0; i < 16; ++i) acc[d][i] += sum[i] * down;
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          shift += kShift;
          down *= kDown;
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            s[u][i] = __builtin_fmaf(s[u][i], f, -less) < kSmall ? kNone : s[u][i];
      }
      // Output, in a fixed order too: V fragments kAhead products ahead, and the
      // probabilities of the next 16 keys between the products of these.
      {
        constexpr int G = 2 * SUB, N = G * DB, kAhead = 3;
        f16x8 vf[kAhead + 1];
        auto fetch = [&](int n) { vf[n % (kAhead + 1)] = values_of(n / DB, n % DB); };
        auto probability = [&](int g, int j) {
          const int u = g >> 1, i = 8 * (g & 1) + j;
          const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(s[u][i], by, -below));
          l_run += w;
          weight(u, i, w);
        };
#pragma unroll
        for (int n = 0; n < kAhead; ++n) fetch(n);
#pragma unroll
        for (int j = 0; j < 8; ++j) probability(0, j);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int g = n / DB, d = n % DB;
          if (n + kAhead < N) fetch(n + kAhead);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int e = SPLIT - 1; e >= 0; --e)
            acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(e ? kv_rest_values(vf[n % (kAhead + 1)]) : vf[n % (kAhead + 1)],
                                                            p[g >> 1][g & 1][e], acc[d], 0, 0, 0);
          if (g + 1 < G) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j * DB / 8 == d) probability(g + 1, j);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    lds_barrier();
  }

  l_run += __shfl_xor(l_run, 32, 64);
  if (!row_live) return;
  const int64_t row = (int64_t)(rg.first + qi) * a.query_heads + qh;
  if (sp.splits == 1) {
    const float by = l_run == 0.0f ? 0.0f : global_decode(c.global_v) / l_run;  // a NaN stays one
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 32 * d + 8 * i + 4 * half;
        const float v[4] = {acc[d][4 * i] * by, acc[d][4 * i + 1] * by, acc[d][4 * i + 2] * by, acc[d][4 * i + 3] * by};
        if (at < c.dim) kv_store4(dt, a.out, row * c.dim + at, v);
      }
    if (a.lse && half == 0) a.lse[row] = l_run == 0.0f ? kNone : (m_run - kBias + __builtin_log2f(l_run)) * kLn2;
  } else {
    const int64_t part = row * sp.splits + split;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 32 * d + 8 * i + 4 * half;
        const float v[4] = {acc[d][4 * i], acc[d][4 * i + 1], acc[d][4 * i + 2], acc[d][4 * i + 3]};
        if (at < c.dim) kv_store4<kF32>(sp.sums, part * c.dim + at, v);
      }
    if (half == 0) *reinterpret_cast<f32x2*>(sp.stats + 2 * part) = f32x2{m_run, l_run};
  }
}

// ----------------------------------------------------------------- joining the parts

// Row `row` of the output from its parts at, at + stride, ..: by one workgroup
// (WAVES 4: many parts) or one wave (WAVES 1: many rows of a few parts).  Each
// wave sums some of the parts, several side by side (dim / 4 lanes a part),
// and everything is added in a fixed order, so every run gives the same bits.
template <int WAVES>
__device__ __forceinline__ void kv_join(const KvCache& c, const KvAttention& a, int dt, const float* sums,
                                        const float* stats, int64_t at, int64_t stride, int parts, int64_t row) {
  const int lane = threadIdx.x & 63, wave = WAVES == 1 ? 0 : threadIdx.x >> 6;
  float top = kNone;
  for (int i = lane; i < parts; i += 64) top = fmaxf(top, stats[2 * (at + i * stride)]);
  top = wave_max(top);
  const int wide = c.dim / 4, each_wave = 64 / wide;  // lanes of a part, parts side by side
  const int side = lane / wide, d = 4 * (lane - side * wide);
  float l = 0.0f, v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (side < each_wave) {
#pragma unroll 4
    for (int i = wave * each_wave + side; i < parts; i += WAVES * each_wave) {
      const int64_t e = at + i * stride;
      const f32x2 st = *reinterpret_cast<const f32x2*>(stats + 2 * e);
      const f32x4 o = *reinterpret_cast<const f32x4*>(sums + e * c.dim + d);
      const float by = st.x == kNone ? 0.0f : __builtin_amdgcn_exp2f(st.x - top);
      l += by * st.y;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += by * o[j];
    }
  }
  for (int s = 1; s < each_wave; ++s) {  // the parts side by side, onto the first
    const float l2 = __shfl(l, lane + s * wide, 64);
    float v2[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v2[j] = __shfl(v[j], lane + s * wide, 64);
    if (side == 0) {
      l += l2;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += v2[j];
    }
  }
  if constexpr (WAVES > 1) {
    __shared__ __attribute__((aligned(16))) float part[WAVES][kKvMaxDim];
    __shared__ float part_l[WAVES];
    if (side == 0) *reinterpret_cast<f32x4*>(&part[wave][d]) = f32x4{v[0], v[1], v[2], v[3]};
    if (lane == 0) part_l[wave] = l;
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      l += part_l[w];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += side == 0 ? part[w][d + j] : 0.0f;
    }
  }
  l = __shfl(l, 0, 64);
  if (side > 0) return;
  const float by = l == 0.0f ? 0.0f : global_decode(c.global_v) / l;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= by;
  kv_store4(dt, a.out, row * c.dim + d, v);
  if (a.lse && lane == 0) a.lse[row] = l == 0.0f ? kNone : (top - kBias + __builtin_log2f(l)) * kLn2;
}

__global__ void __launch_bounds__(256) kv_join_few_kernel(KvCache c, KvAttention a, KvShare sh, int dt) {
  const int b = blockIdx.y;
  const int qi = blockIdx.x / a.query_heads, qh = blockIdx.x - qi * a.query_heads;
  const int head = qh / a.groups, r = qi * a.groups + qh - head * a.groups;
  KvScan scan;
  const int each = kv_units_each(c, a, sh, scan);
  int base = 0;
  if (a.seqs > 64) {
    kv_scan(c, a, sh.rows, 0, 0, scan);
    while (b >= base + 64) {
      base += 64;
      kv_scan(c, a, sh.rows, base, scan.after, scan);
    }
  }
  const KvRange rg = kv_range_of(scan, b - base);
  if (qi >= rg.n) return;
  const int units = __builtin_amdgcn_readlane(scan.units, b - base);
  const int u0 = __builtin_amdgcn_readlane(scan.first, b - base) + head * units;
  const int g0 = u0 / each, g1 = (u0 + units - 1) / each;
  if (g0 == g1) return;  // one workgroup had it all
  const int parts = g1 - g0 + 1;
  const int64_t at = ((int64_t)g0 + b * c.heads + head) * sh.rows + r;
  kv_join<kFewWaves>(c, a, dt, sh.sums, sh.stats, at, sh.rows, parts, (int64_t)(rg.first + qi) * a.query_heads + qh);
}

__global__ void __launch_bounds__(256) kv_join_many_kernel(KvCache c, KvAttention a, KvChunks sp, int dt) {
  const int row_of = blockIdx.x * 4 + (threadIdx.x >> 6);
  const int qi = row_of / a.query_heads, qh = row_of - qi * a.query_heads;
  const int r = qi * a.groups + qh % a.groups;  // its row among those of its kv head
  const KvRange rg = kv_range(a, blockIdx.y, r / kManyRows * kManyRows, kManyRows);
  if (qi >= rg.n) return;
  const int parts = rg.hi > rg.lo ? (rg.hi - rg.lo - 1) / sp.chunk + 1 : 1;
  const int64_t row = (int64_t)(rg.first + qi) * a.query_heads + qh;
  kv_join<1>(c, a, dt, sp.sums, sp.stats, row * sp.splits, 1, parts, row);
}

// ----------------------------------------------------------------- launches

// Contexts of up to so many keys are left to one workgroup a pair: no parts, no
// second launch, and with many pairs fewer runs to begin.  8 heads of 128, us,
// alone against shared out with the join:
//   700 keys: 1 sequence 14.1 / 13.4, 16 sequences 15.0 / 18.0; 1024 keys: 16.2 /
//   13.3, 17.2 / 18.5
//   2048 keys: 1 sequence 24.7 / 14.0; 16 26.2 / 27.6 (heads of 256 40 / 32); 64
//   40 / 51; 128, lengths up to that 55 / 82
//   4096 keys: 64 sequences 72 / 83, lengths up to that 58 / 63
// Past 4096 keys one long context among short ones would keep all waiting.  With
// few pairs the rule gives up to 3 us (1 sequence of 1024 keys) for one launch
// and no workspace; the size of a head is not in it.
constexpr int kFewAlone = 1024, kFewAloneMost = 4096;
// (A launch has fewer than 2^24 workgroups.)
constexpr int64_t few_alone(int64_t pairs) {
  return pairs >= 1 << 24 ? -1 : pairs >= (kFewAloneMost - kFewAlone) / 6 ? kFewAloneMost : kFewAlone + 6 * pairs;
}

struct KvPlan {
  bool few;
  int mt, groups;                 // few rows: row tiles of 16, workgroups
  int row_tiles, chunk, splits;   // many rows
  size_t sums_bytes, bytes;
};

constexpr int few_groups(int dim) { return dim <= 64 ? 1 : dim <= 128 ? 2 : dim <= 192 ? 3 : 4; }

// Up to 32 rows a (sequence, kv head) the keys are streamed once past all of
// them; more rows are matrix work.  32 rows, 8 x 30000 keys, 4 heads, few
// against many, us: dim 128 76 / 90, float32 92 / 175; dim 256 128 / 254,
// float32 282 / 317 (48 rows of dim 128 on the many-rows kernel: 92, 96 rows 105).
KvPlan kv_plan(const KvCache& c, const KvAttention& a, int split) {
  KvPlan p{};
  const int64_t rows = (int64_t)a.max_queries * a.groups;
  int64_t keys = a.max_keys;
  if (a.window > 0 && keys > (int64_t)a.window + a.max_queries) keys = (int64_t)a.window + a.max_queries;
  const int64_t pairs = (int64_t)a.seqs * c.heads;
  size_t parts;
  p.few = rows <= 32;
  if (p.few) {
    p.mt = rows <= 16 ? 1 : 2;
    // as many workgroups as run at once, but no more than there can be units
    const int64_t units = pairs * (keys > kFewStep ? (keys + kFewStep - 1) / kFewStep : 1);
    const int64_t most = (int64_t)device_cu_count() * few_occupancy(few_groups(c.dim), p.mt, split);
    const bool alone = keys <= few_alone(pairs);
    p.groups = (int)(alone ? pairs : units < most ? units : most);
    parts = alone ? 0 : (size_t)(p.groups + pairs) * 16 * p.mt;
  } else {
    p.row_tiles = (int)((rows + kManyRows - 1) / kManyRows);
    const int64_t tiles = pairs * p.row_tiles;
    // As many workgroups as run at once (two a CU: heads of up to 128 in 16 bits
    // and of 64 in 32; the other instances run one), rounded to the nearest number of
    // splits; for short contexts rounded down, as a second launch is worth only
    // a whole factor there.  3 x 400 queries, 32 heads of 128, us, nearest
    // against down: 2000 keys 102 / 88, 4200 keys 168 / 168, 9000 keys 315 /
    // 371; 3 x 777 over 777 keys, 16 heads, 57 / 34.
    int64_t splits = (2 * device_cu_count() + (keys >= 4096 ? tiles / 2 : 0)) / tiles;
    const int64_t most = keys / 256;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    p.chunk = (int)((keys / splits + 64) / 64 * 64);
    p.splits = keys > 0 ? (int)((keys + p.chunk - 1) / p.chunk) : 1;
    parts = p.splits > 1 ? (size_t)a.tokens * a.query_heads * p.splits : 0;
  }
  p.sums_bytes = (parts * c.dim * 4 + 255) / 256 * 256;
  p.bytes = p.sums_bytes + (parts * 8 + 255) / 256 * 256;
  return p;
}

constexpr int kMaxLds = 144 * 1024;  // leaves room for the kernels' static LDS

// Lets `kernel` have more than 64 KB of dynamic LDS; once per device (or twice,
// by two threads at once).
template <typename K>
hipError_t allow_lds(K* kernel, std::atomic<bool> (&set)[64]) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) dev = 0;
  if (dev < 0 || dev >= 64 || set[dev]) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLds);
  if (e == hipSuccess) set[dev] = true;
  return e;
}

template <int NG, bool EXACT>
hipError_t launch_few(const KvCache& c, const KvAttention& a, const KvShare& sh, const KvPlan& p, int dt, bool q_vec,
                      hipStream_t s) {
  const size_t lds = (size_t)kFewWaves * kFewTile * few_row_bytes(NG) + 2 * 8 * kFewPages;
#define KV_FEW(MT, SPLIT)                                                                         \
  do {                                                                                            \
    static std::atomic<bool> set[64];                                                             \
    if (hipError_t e = allow_lds(&kv_few_kernel<NG, MT, SPLIT, EXACT>, set)) return e;            \
    kv_few_kernel<NG, MT, SPLIT, EXACT><<<p.groups, 256, lds, s>>>(c, a, sh, dt, q_vec);          \
  } while (0)
  if (p.mt == 1) {
    if (dt == kF32) KV_FEW(1, 2); else KV_FEW(1, 1);
  } else {
    if (dt == kF32) KV_FEW(2, 2); else KV_FEW(2, 1);
  }
#undef KV_FEW
  return hipGetLastError();
}

template <int NG, bool EXACT>
hipError_t launch_many(const KvCache& c, const KvAttention& a, const KvChunks& sp, int dt, bool q_vec, hipStream_t s) {
  const dim3 grid((unsigned)(sp.row_tiles * c.heads * sp.splits), a.seqs);
#define KV_MANY(SPLIT)                                                                            \
  do {                                                                                            \
    static std::atomic<bool> set[64];                                                             \
    if (hipError_t e = allow_lds(&kv_many_kernel<NG, SPLIT, EXACT>, set)) return e;               \
    kv_many_kernel<NG, SPLIT, EXACT><<<grid, 256, many_lds(NG), s>>>(c, a, sp, dt, q_vec);        \
  } while (0)
  if (dt == kF32) KV_MANY(2); else KV_MANY(1);
#undef KV_MANY
  return hipGetLastError();
}

template <int NG, bool EXACT>
hipError_t launch(const KvCache& c, const KvAttention& a, const KvPlan& p, int dt, float* sums, float* stats,
                  bool q_vec, hipStream_t s) {
  const dim3 rows((unsigned)(a.max_queries * a.query_heads), a.seqs);
  if (p.few) {
    const KvShare sh{p.groups, 16 * p.mt, p.bytes ? sums : nullptr, stats};
    const hipError_t e = launch_few<NG, EXACT>(c, a, sh, p, dt, q_vec, s);
    if (e != hipSuccess || p.bytes == 0) return e;
    kv_join_few_kernel<<<rows, 256, 0, s>>>(c, a, sh, dt);
  } else {
    const KvChunks sp{p.chunk, p.splits, p.row_tiles, sums, stats};
    const hipError_t e = launch_many<NG, EXACT>(c, a, sp, dt, q_vec, s);
    if (e != hipSuccess || p.bytes == 0) return e;
    kv_join_many_kernel<<<dim3((rows.x + 3) / 4, rows.y), 256, 0, s>>>(c, a, sp, dt);
  }
  return hipGetLastError();
}

}  // namespace

size_t kv_attention_workspace(const KvCache& c, const KvAttention& a) {
  const size_t one = kv_plan(c, a, 1).bytes, two = kv_plan(c, a, 2).bytes;
  return one > two ? one : two;
}

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, int dt, void* workspace, hipStream_t s) {
  const KvPlan p = kv_plan(c, a, dt == kF32 ? 2 : 1);
  float* sums = reinterpret_cast<float*>(workspace);
  float* stats = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) + p.sums_bytes);
  const bool q_vec = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && (a.q_token | a.q_head) % 8 == 0;
  switch (c.dim) {
    case 64: return launch<1, true>(c, a, p, dt, sums, stats, q_vec, s);
    case 128: return launch<2, true>(c, a, p, dt, sums, stats, q_vec, s);
    case 256: return launch<4, true>(c, a, p, dt, sums, stats, q_vec, s);
  }
  if (c.dim < 64) return launch<1, false>(c, a, p, dt, sums, stats, q_vec, s);
  if (c.dim < 128) return launch<2, false>(c, a, p, dt, sums, stats, q_vec, s);
  if (c.dim <= 192) return launch<3, false>(c, a, p, dt, sums, stats, q_vec, s);
  return launch<4, false>(c, a, p, dt, sums, stats, q_vec, s);
}

}  // namespace nvfp4
