// kv_attention.hip -- attention of 16-bit or float32 queries over keys and
// values held in NVFP4 (kv_device.h), for gfx950.
//
// Query i of a sequence with n queries and a context of L tokens (its own
// among them) stands at position p = L - n + i.  It sees key j when j < L,
// with `causal` j <= p, and with a window w > 0 also j > p - w:
//     s_j = scale * q . k_j,   lse = log sum_j exp(s_j),
//     out = sum_j exp(s_j - lse) v_j;   no visible key: out = 0, lse = -inf.
//
// One wave per query and query head: 64 keys at a time, a lane computes one
// key's score, then every lane sums its values' columns.
#include "kv_device.h"

namespace nvfp4 {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

template <int DT>
__global__ void __launch_bounds__(64) kv_attention_row_kernel(KvCache c, KvAttention a) {
  __shared__ float q[256];
  __shared__ float p[64];
  __shared__ int64_t rows[64];
  const int lane = threadIdx.x;
  const int token = blockIdx.x, qh = blockIdx.y;
  const int head = qh / a.groups;
  // the sequence that holds this query
  int b = token, first = token, n = 1;
  if (a.query_starts) {
    int lo = 0, hi = a.seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.query_starts[mid] <= token) lo = mid; else hi = mid;
    }
    b = lo;
    first = a.query_starts[b];
    n = a.query_starts[b + 1] - first;
  }
  using T = typename Elem<DT>::T;
  if (token < first || token >= first + n) return;
  const int context = a.context_lens[b];
  const int pos = context - n + (token - first);
  int end = min(context, a.max_keys);
  int begin = 0;
  if (a.causal) {
    end = min(end, pos + 1);
    if (a.window > 0) begin = max(0, pos - a.window + 1);
  }
  const float factor = a.scale * kLog2e * global_decode(c.global_k);
  for (int d = lane; d < c.dim; d += 64)
    q[d] = to_f32<DT>(reinterpret_cast<const T*>(a.q)[token * a.q_token + qh * a.q_head + d]);
  __syncthreads();
  float m = -__builtin_inff(), l = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j0 = begin; j0 < end; j0 += 64) {
    const int j = j0 + lane;
    float s = -__builtin_inff();
    int64_t row = -1;
    if (j < end) {
      const int pi = kv_div(j, c.page_div);
      const int page = a.page_table[(int64_t)b * a.table_stride + pi];
      if (page >= 0 && page < c.pages) {
        row = kv_row(c, page, head, j - pi * c.page_size);
        s = 0.0f;
        for (int g = 0; g < c.dim / 16; ++g) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(c.k_codes + row * (c.dim / 2) + 8 * g);
          float x[8], y[8], sum = 0.0f;
          e2m1_decode8_f32(w[0], x);
          e2m1_decode8_f32(w[1], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += q[16 * g + i] * x[i] + q[16 * g + 8 + i] * y[i];
          s += sum * e4m3_decode(c.k_scales[row * (c.dim / 16) + g]);
        }
        s *= factor;
      }
    }
    const float top = wave_max(s);
    if (top == -__builtin_inff()) continue;  // wave-uniform
    const float m2 = fmaxf(m, top);
    const float keep = __builtin_amdgcn_exp2f(m - m2);
    const float e = __builtin_amdgcn_exp2f(s - m2);
    l = l * keep + wave_sum(e);
    m = m2;
    __syncthreads();
    p[lane] = e;
    rows[lane] = row;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= keep;
    for (int jj = 0; jj < 64; ++jj) {
      if (rows[jj] < 0) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = 64 * i + lane;
        if (d >= c.dim) break;
        const uint32_t byte = c.v_codes[rows[jj] * (c.dim / 2) + d / 2];
        acc[i] += p[jj] * e2m1_decode(byte >> (4 * (d & 1))) * e4m3_decode(c.v_scales[rows[jj] * (c.dim / 16) + d / 16]);
      }
    }
  }
  const float by = l > 0.0f ? global_decode(c.global_v) / l : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = 64 * i + lane;
    if (d < c.dim)
      reinterpret_cast<T*>(a.out)[((int64_t)token * a.query_heads + qh) * c.dim + d] = from_f32<DT>(acc[i] * by);
  }
  if (a.lse && lane == 0)
    a.lse[(int64_t)token * a.query_heads + qh] = l > 0.0f ? (m + __builtin_log2f(l)) / kLog2e : -__builtin_inff();
}

}  // namespace

size_t kv_attention_workspace(const KvCache&, const KvAttention&) { return 0; }

hipError_t launch_kv_attention(const KvCache& c, const KvAttention& a, int dt, void*, hipStream_t s) {
  const dim3 grid((unsigned)a.tokens, a.query_heads);
  if (dt == kF32)
    kv_attention_row_kernel<kF32><<<grid, 64, 0, s>>>(c, a);
  else if (dt == kF16)
    kv_attention_row_kernel<kF16><<<grid, 64, 0, s>>>(c, a);
  else
    kv_attention_row_kernel<kBF16><<<grid, 64, 0, s>>>(c, a);
  return hipGetLastError();
}

}  // namespace nvfp4
