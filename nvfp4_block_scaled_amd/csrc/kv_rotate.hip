// kv_rotate.hip -- queries and keys rotated by their positions, keys and
// values quantized into their slots of an NVFP4 cache, in one launch (gfx950).
//
// The first `rotary` values of a head form pairs (a, b): value i with value
// i + rotary/2, or neighbours (2i, 2i + 1).  With the cosine c and sine s of
// pair i at the token's position, read from a table,
//     a' = a c - b s,   b' = b c + a s
// in float32, each product and sum rounded by itself (no contraction), so that
// the codes are defined to the bit; the rest of a head stays as it is.  Keys
// are encoded from these float32 values, as nvfp4_quantize encodes a row
// (encode_half_group); queries are rounded to T.
//
// Only memory bounds it.  A lane has 8 values; a wave takes as many whole heads
// of one token as have room in it (4 of dim 128: 1 KB of a fused projection's
// row), the cosines and sines in registers, and goes on to the token's next
// heads: read per head, the table would come to as many bytes as the values.
// The second half of a pair, 8 values elsewhere in the same head, is loaded
// along (another lane of the wave loads the same line).  A workgroup's four
// waves take four consecutive tokens, so that a page's codes (64 bytes a token
// and head of dim 128) are written as whole lines.  16384 tokens, 32 query and 8 kv
// heads of 128, bfloat16: 363 MB in 79 us, 4.6 TB/s (91 before a turn's loads went
// out a turn ahead); 64 tokens 4.2 us.
#include "kv_device.h"
#include "layer_internal.h"

namespace nvfp4 {

namespace {

constexpr int kTokens = 4;  // of a workgroup, one a wave

// 8 values as they are loaded, on their way while those before them are encoded.
template <int DT, bool VEC>
struct Eight {
  u32x4 w[DT == kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t e) {
    const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const typename Elem<DT>::T*>(base) + e);
#pragma unroll
    for (int i = 0; i < (DT == kF32 ? 2 : 1); ++i) w[i] = p[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (DT == kF32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i / 4][i % 4]);
    } else {
      unpack8<DT>(w[0], v);
    }
  }
};
template <int DT>
struct Eight<DT, false> {  // (rows that start anywhere)
  typename Elem<DT>::T x[8];
  __device__ __forceinline__ void load(const void* base, int64_t e) {
    const typename Elem<DT>::T* p = reinterpret_cast<const typename Elem<DT>::T*>(base) + e;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32<DT>(x[i]);
  }
};

// Where the 8 values of lane piece u find their pairs.
struct Rotation {
  int kind;    // 0: not rotated, 1: first halves, 2: second halves, 3: neighbours
  int shift;   // elements from a value to its pair (kinds 1 and 2)
  float c[8], s[8];
};
__device__ __forceinline__ void rotate(const Rotation& r, float (&v)[8], const float (&o)[8]) {
#pragma clang fp contract(off)
  if (r.kind == 0) return;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float other = r.kind == 3 ? v[i ^ 1] : o[i];
    const bool first = r.kind == 3 ? (i & 1) == 0 : r.kind == 1;
    const float x = v[i] * r.c[i], y = other * r.s[i];
    w[i] = first ? x - y : x + y;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = w[i];
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(64 * kTokens)
kv_rotate_kernel(KvCache c, KvRotate a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t token = (int64_t)blockIdx.x * kTokens + wave;
  if (token >= a.tokens) return;
  const int pieces = c.dim / 8, each = 64 / pieces;  // heads of a wave
  const int sub = kv_div(lane, a.piece_div), u = lane - sub * pieces;
  const bool in = sub < each;
  const int64_t slot = a.slots[token];
  const int position = a.positions[token];
  const bool there = position >= 0 && position < a.table_rows;
  const bool held = there && slot >= 0 && slot < (int64_t)c.pages * c.page_size;

  Rotation r;
  const int half = a.rotary / 2;
  const int d = 8 * u;
  r.kind = d >= a.rotary ? 0 : a.interleaved ? 3 : d < half ? 1 : 2;
  r.shift = r.kind == 1 ? half : r.kind == 2 ? -half : 0;
  if (r.kind != 0 && there) {
    const float* row = a.table + (int64_t)position * a.rotary;
    if (a.interleaved) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(row + d / 2), y = *reinterpret_cast<const f32x4*>(row + half + d / 2);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r.c[i] = x[i / 2];
        r.s[i] = y[i / 2];
      }
    } else {
      const float* at = row + (r.kind == 1 ? d : d - half);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(at + 4 * j), y = *reinterpret_cast<const f32x4*>(at + half + 4 * j);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          r.c[4 * j + i] = x[i];
          r.s[4 * j + i] = y[i];
        }
      }
    }
  }

  // heads of queries, then keys, then values, `each` at a time
  const int nq = (a.query_heads + each - 1) / each, nk = (c.heads + each - 1) / each;
  const int all = nq + 2 * nk;
  const int from = blockIdx.y * a.turns, to = min(all, from + a.turns);
  const float enc_k = global_encode(c.global_k), enc_v = global_encode(c.global_v);
  const int page = held ? (int)kv_div((uint32_t)slot, c.page_div) : 0;
  const int off = held ? (int)slot - page * c.page_size : 0;
  // A turn's values and their pairs are on their way a turn ahead; lanes without a
  // head load a head that there is.
  auto load = [&](int turn, Eight<DT, VEC>& v, Eight<DT, VEC>& o) {
    const bool of_q = turn < nq, of_v = turn >= nq + nk;
    const int head = (of_q ? turn : of_v ? turn - nq - nk : turn - nq) * each + sub;
    const void* x = of_q ? a.q : of_v ? a.v : a.k;
    const int64_t at = token * (of_q ? a.q_token : of_v ? a.v_token : a.k_token) +
                       min(head, (of_q ? a.query_heads : c.heads) - 1) * (of_q ? a.q_head : of_v ? a.v_head : a.k_head) + d;
    v.load(x, at);
    o.load(x, at + r.shift);
  };
  Eight<DT, VEC> next_v, next_o;
  load(from, next_v, next_o);
  for (int turn = from; turn < to; ++turn) {
    const bool of_q = turn < nq, of_v = turn >= nq + nk;
    const int head = (of_q ? turn : of_v ? turn - nq - nk : turn - nq) * each + sub;
    const bool live = in && head < (of_q ? a.query_heads : c.heads);
    const Eight<DT, VEC> now_v = next_v, now_o = next_o;
    load(min(turn + 1, to - 1), next_v, next_o);
    float v[8], o[8];
    now_v.get(v);
    now_o.get(o);
    if (!of_v) rotate(r, v, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = live && there ? v[i] : 0.0f;
    if (of_q) {
      if (live) store8<DT>(a.q_out, ((token * a.query_heads + head) * c.dim + d) >> 3, v);
    } else {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, __builtin_fabsf(v[i]));
      top = fmaxf(top, __shfl_xor(top, 1, 64));  // (a head has an even number of pieces)
      uint32_t byte;
      const uint32_t word = encode_half_group(v, top, of_v ? enc_v : enc_k, byte);
      if (live && held) {
        const int64_t row = kv_row(c, page, head, off);
        reinterpret_cast<uint32_t*>(of_v ? c.v_codes : c.k_codes)[row * pieces + u] = word;
        if ((u & 1) == 0) (of_v ? c.v_scales : c.k_scales)[row * (c.dim / 16) + (u >> 1)] = (uint8_t)byte;
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_rotate(const KvCache& c, KvRotate a, int dt, hipStream_t s) {
  const int each = 64 / (c.dim / 8);
  const int all = (a.query_heads + each - 1) / each + 2 * ((c.heads + each - 1) / each);
  const unsigned blocks = (unsigned)((a.tokens + kTokens - 1) / kTokens);
  a.piece_div = kv_make_div((uint32_t)(c.dim / 8));
  // a token's heads are split up where the tokens alone are too few workgroups (4 a
  // CU; 8 a CU: within 8 % either way from 64 to 2777 tokens)
  int splits = (int)(4 * device_cu_count() / blocks);
  splits = splits < 1 ? 1 : splits > all ? all : splits;
  a.turns = (all + splits - 1) / splits;
  const dim3 grid(blocks, (unsigned)((all + a.turns - 1) / a.turns));
  const int64_t lane_elems = dt == kF32 ? 4 : 8;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.q)) & 15) == 0 &&
                   (a.k_token | a.k_head | a.v_token | a.v_head | a.q_token | a.q_head) % lane_elems == 0;
#define KV_ROTATE(DT)                                                                       \
  do {                                                                                      \
    if (vec) kv_rotate_kernel<DT, true><<<grid, 64 * kTokens, 0, s>>>(c, a);                \
    else kv_rotate_kernel<DT, false><<<grid, 64 * kTokens, 0, s>>>(c, a);                   \
  } while (0)
  if (dt == kF32) KV_ROTATE(kF32);
  else if (dt == kF16) KV_ROTATE(kF16);
  else KV_ROTATE(kBF16);
#undef KV_ROTATE
  return hipGetLastError();
}

}  // namespace nvfp4
