// mx_norm.hip -- root-mean-square norm with the residual's addition, its
// output encoded in an mx mode (gfx950).
//
// Per row of k values:
//     h = T(x + residual)                     the residual stream, kept
//     r = float32(1 / sqrt(mean(h^2) + eps))
//     y = (h * r) * weight                    float32, each product rounded
// and y's groups of 32 are encoded as nvfp4_mx_quantize does (mx_device.h),
// straight from float32: rounded to T in between, as by a norm and a quantize
// apart, a value may land on the other side of a code's border.
//
// The squares are summed in float64: a group's codes hang on the last bit of r,
// and so the order of the sum, which differs between the launch shapes below,
// does not reach it (but for a row in some 10^8, whose exact r lies that near
// the middle between two float32).  It costs two instructions a value next to 7
// bytes of memory traffic.
//
// Memory bounds it: a row is held in registers between the sum and the encode,
// so each value is read once.  A lane holds pieces of 8 values, the 4 pieces of
// a group in neighbouring lanes.  8192 rows of 4096, bfloat16 with residual to packed
// mxfp8: 236 MB in 47 us, 5.0 TB/s, a large copy's rate (60 us before all loads of a
// row, its weights' too, went out before the sum); one row 3.8 us, a launch and one
// chain of load, sum and store.  Rows longer than 4096 have one shape up to 16384
// values, 64 a lane, and stay below that rate: 4096 rows, the same, of 5120 40 us (3.7
// TB/s), of 7168 50 (4.1), of 8192 53 (4.4), of 16384 96 (4.9); 2048 of 20480, read
// twice, 91.
#include "layer_internal.h"
#include "mx_device.h"
#include "nvfp4_device.h"
#include "nvfp4_internal.h"

namespace nvfp4 {

namespace {

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// e4m3 codes of 8 values of magnitude 448 (1 + 2^-23) at most, or NaN:
// v_cvt_pk_fp8_f32 rounds to nearest even, so what passes 448 by that little
// becomes 448; infinities are cut to it here, as e4m3_encode_signed does.
__device__ __forceinline__ u32x2 mx_pack8(const float (&v)[8], float by) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)
    y[i] = __builtin_amdgcn_fmed3f(v[i] * by, -kE4M3Max, kE4M3Max);
  }
  u32x2 w;
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], b, true);
  w.x = (uint32_t)a;
  w.y = (uint32_t)b;
  return w;
}

// 8 values as they are loaded: converted at once, each load would be waited for
// before the next is issued.
template <int DT>
struct Eight {
  u32x4 w[DT == kF32 ? 2 : 1];
  template <bool STREAM>
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const u32x4* p = reinterpret_cast<const u32x4*>(base) + (DT == kF32 ? 2 : 1) * at;
#pragma unroll
    for (int i = 0; i < (DT == kF32 ? 2 : 1); ++i) w[i] = STREAM ? __builtin_nontemporal_load(p + i) : p[i];
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

// LANES lanes (a wave, or the whole workgroup) take a row, NP pieces a lane;
// LOOP: rows longer than that, whose rest is read twice.
template <int DT, int BITS, int LANES, int NP, bool LOOP>
__global__ void __launch_bounds__(LANES == 64 ? 256 : LANES)
mx_norm_kernel(MxNorm p, int tiles) {
  constexpr int kRows = LANES == 64 ? 4 : 1;  // of a workgroup
  constexpr int kChunk = LANES * NP;
  const int lane = LANES == 64 ? (threadIdx.x & 63) : threadIdx.x;
  int64_t row;
  if (p.packed) {
    // The rows of a tile write parts of the same lines: on one XCD (workgroup
    // index mod 8), one after another, so that its L2 joins them.
    constexpr int kEach = 32 / kRows;  // workgroups of a tile
    const int xcd = blockIdx.x & 7, n = blockIdx.x >> 3;
    const int tile = n / kEach * 8 + xcd;
    if (tile >= tiles) return;
    row = (int64_t)tile * 32 + n % kEach * kRows + (LANES == 64 ? threadIdx.x >> 6 : 0);
  } else {
    row = (int64_t)blockIdx.x * kRows + (LANES == 64 ? threadIdx.x >> 6 : 0);
    if (LANES == 64 && row >= p.rows) return;
  }
  const bool real = row < p.rows;  // else padding of the last tile
  const int pieces = (int)(p.k / 8);
  const int quads = (int)((p.k + 255) / 256);
  const int all = p.packed ? 32 * quads : pieces;  // with the padding behind the row
  const int64_t first = (real ? row : 0) * pieces;

  // No branch stands between the loads: lanes behind the row's end load its last
  // piece again, and what is not there becomes 0.
  float h[NP][8];
  Eight<DT> weight[NP];
  auto load = [&](int from, bool weights) {
    Eight<DT> x[NP], y[NP];
    auto take = [&](Eight<DT>(&into)[NP], const void* base) {
#pragma unroll
      for (int j = 0; j < NP; ++j) into[j].template load<true>(base, first + min(from + j * LANES + lane, pieces - 1));
    };
    take(x, p.x);
    if (p.residual) take(y, p.residual);
    if (weights && p.weight) {
#pragma unroll
      for (int j = 0; j < NP; ++j) weight[j].template load<false>(p.weight, min(from + j * LANES + lane, pieces - 1));
    }
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const bool in = real && from + j * LANES + lane < pieces;
      x[j].get(h[j]);
      if (p.residual) {
        float v[8];
        y[j].get(v);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = to_f32<DT>(from_f32<DT>(h[j][i] + v[i]));
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] = in ? h[j][i] : 0.0f;
    }
  };
  double squares = 0.0;
  auto add = [&]() {
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) squares = __builtin_fma((double)h[j][i], (double)h[j][i], squares);
  };
  load(0, !LOOP);
  add();
  if constexpr (LOOP) {
    for (int from = kChunk; from < pieces; from += kChunk) {
      load(from, false);
      add();
    }
    load(0, true);
  }
  squares = wave_sum_f64(squares);
  if constexpr (LANES > 64) {
    __shared__ double part[LANES / 64];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = squares;
    __syncthreads();
    squares = part[0];
#pragma unroll
    for (int w = 1; w < LANES / 64; ++w) squares += part[w];
  }
  const float r = (float)(1.0 / __builtin_sqrt(squares / (double)p.k + p.eps));

  auto encode = [&](int from) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int at = from + j * LANES + lane;
      if (from + j * LANES >= all) break;
      const bool live = real && at < pieces;
      if (live && p.sum) store8<DT>(p.sum, first + at, h[j]);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = 1.0f;
      if (p.weight) weight[j].get(y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
#pragma clang fp contract(off)
        y[i] = live ? (h[j][i] * r) * y[i] : 0.0f;
      }
      if (live && p.normed) store8<DT>(p.normed, first + at, y);
      // magnitudes as whole numbers: a NaN is above every number
      uint32_t top = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(y[i]) & 0x7FFFFFFFu);
      top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
      float by;
      uint32_t s = mx_scale<BITS>(__uint_as_float(min(top, 0x7F800000u)), by);
      if (top > 0x7F800000u) s = 255u;
      if (at >= all) continue;
      const int g = at >> 2, sub = at & 3;
      if (!p.packed) {
        if constexpr (BITS == 4) reinterpret_cast<uint32_t*>(p.codes)[first + at] = mx_codes4(y, by);
        else reinterpret_cast<u32x2*>(p.codes)[first + at] = mx_pack8(y, by);
        if (sub == 0) p.scales[row * (pieces >> 2) + g] = (uint8_t)s;
      } else {  // the layout of mx_codec.hip (packed_index)
        const int64_t tile = row >> 5;
        const int i = (int)(row & 31), step = g >> 1, half = g & 1;
        const int64_t block = (tile * 4 * quads + step) * MxFormat<BITS>::kPieces + (BITS == 4 ? half : 2 * half);
        if constexpr (BITS == 4)
          *reinterpret_cast<uint32_t*>(p.codes + block * 512 + 16 * i + 4 * sub) = mx_codes4(y, by);
        else
          *reinterpret_cast<u32x2*>(p.codes + (block + (sub >> 1)) * 512 + 16 * i + 8 * (sub & 1)) = mx_pack8(y, by);
        if (sub == 0) p.scales[(tile * quads + (step >> 2)) * 256 + 4 * (i + 32 * half) + (step & 3)] = live ? (uint8_t)s : 0;
      }
    }
  };
  encode(0);
  if constexpr (LOOP) {
    for (int from = kChunk; from < all; from += kChunk) {
      load(from, true);
      encode(from);
    }
  }
}

template <int DT, int BITS>
hipError_t launch(const MxNorm& n, hipStream_t s) {
  const int64_t pieces = n.packed ? (n.k + 255) / 256 * 32 : n.k / 8;
  const int tiles = (int)((n.rows + 31) / 32);
#define MX_NORM(LANES, NP, LOOP)                                                                         \
  do {                                                                                                   \
    constexpr int rows = LANES == 64 ? 4 : 1;                                                            \
    const int64_t grid = n.packed ? (int64_t)(tiles + 7) / 8 * 8 * (32 / rows) : (n.rows + rows - 1) / rows; \
    mx_norm_kernel<DT, BITS, LANES, NP, LOOP><<<(unsigned)grid, LANES == 64 ? 256 : LANES, 0, s>>>(n, tiles); \
    return hipGetLastError();                                                                            \
  } while (0)
  // A workgroup a row but for short ones, also where rows are many: 16 values a lane
  // are little enough for eight waves a SIMD (8192 rows of 4096, bfloat16 with
  // residual to packed mxfp8: 48 us, 4.9 TB/s; a wave a row, 64 values a lane, 55).
  if (pieces <= 128) MX_NORM(64, 2, false);
  if (pieces <= 512) MX_NORM(256, 2, false);
  if (pieces <= kMxNormLong / 8) MX_NORM(256, 8, false);
  MX_NORM(1024, 4, true);
#undef MX_NORM
}

}  // namespace

hipError_t launch_mx_norm(const MxNorm& n, int dt, int bits, hipStream_t s) {
  if (n.rows == 0) return hipSuccess;
  if (bits == 4) return dt == kF32 ? launch<kF32, 4>(n, s) : dt == kF16 ? launch<kF16, 4>(n, s) : launch<kBF16, 4>(n, s);
  return dt == kF32 ? launch<kF32, 8>(n, s) : dt == kF16 ? launch<kF16, 8>(n, s) : launch<kBF16, 8>(n, s);
}

}  // namespace nvfp4
