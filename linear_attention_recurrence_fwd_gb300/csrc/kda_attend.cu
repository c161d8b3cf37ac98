// Attention of each sequence's newest tokens over its pages.
//
//     s_j = scale q . k_j,   o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),
//     m = max_j s_j,         lse = m + ln sum_j e^(s_j - m)
//
// over the positions j that the token sees, in one pass: m and the two sums
// are carried and rescaled when m grows.  One warp per (sequence, token,
// query head); lane l holds channels [l d / 32, (l + 1) d / 32).
#include "kda_internal.h"
#include "kda_types.cuh"

namespace kda {
namespace {

template <typename T, typename C, int D>
__global__ void __launch_bounds__(128) attend_kernel(AttendProblem p) {
  constexpr int E = D / 32;
  const long long unit = blockIdx.x * 4LL + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (unit >= (long long)p.cache.n_seq * p.K * p.H_q) return;
  const int h = unit % p.H_q;
  const long long ni = unit / p.H_q;
  const int i = ni % p.K, n = ni / p.K;
  const int hk = h / (p.H_q / p.cache.H_kv);
  const int pos = p.cache.lens[n] + i;
  const bool real = !p.counts || i < p.counts[n];
  int end = real ? pos + 1 : 0;
  if (end > (long long)p.cache.table_width * p.cache.page_size) {
    end = p.cache.table_width * p.cache.page_size;
    if (lane == 0) *p.status = 1;
  }
  const int start = p.window ? max(0, pos - p.window + 1) : 0;
  const T* q = static_cast<const T*>(p.q) + ni * p.q_stride + h * D + lane * E;
  float qr[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qr[e] = to_f32(q[e]) * p.scale * p.cache.k_scale;
    o[e] = 0.f;
  }
  for (int j = start; j < end; ++j) {
    const int page = p.cache.block_table[n * p.cache.table_stride + j / p.cache.page_size];
    if (page < 0 || page >= p.cache.num_pages) {
      if (lane == 0) *p.status = 1;
      continue;
    }
    const long long at = page * p.cache.page_stride + (j % p.cache.page_size) * p.cache.token_stride +
                         hk * p.cache.head_stride + lane * E;
    const C* k = static_cast<const C*>(p.cache.k) + at;
    const C* v = static_cast<const C*>(p.cache.v) + at;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qr[e] * to_f32(k[e]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    if (mn == -INFINITY) continue;
    const float keep = expf(m - mn), w = expf(s - mn);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * to_f32(v[e]);
    m = mn;
  }
  T* out = static_cast<T*>(p.out) + unit * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = from_f32<T>(m == -INFINITY ? 0.f : o[e] * p.cache.v_scale / l);
  if (p.lse && lane == 0) p.lse[unit] = m == -INFINITY ? -INFINITY : m + logf(l);
}

template <typename T, typename C>
cudaError_t launch_typed(const AttendProblem& p, cudaStream_t stream) {
  const long long units = (long long)p.cache.n_seq * p.K * p.H_q;
  const unsigned grid = (unsigned)((units + 3) / 4);
  if (p.cache.d == 128)
    attend_kernel<T, C, 128><<<grid, 128, 0, stream>>>(p);
  else
    attend_kernel<T, C, 64><<<grid, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_cached(const AttendProblem& p, cudaStream_t stream) {
  return p.cache.dtype == KDA_E4M3 ? launch_typed<T, __nv_fp8_e4m3>(p, stream)
                                   : launch_typed<T, T>(p, stream);
}

}  // namespace

size_t attend_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_cache_attend(const AttendProblem& p, void*, cudaStream_t stream) {
  return p.dtype == KDA_BF16 ? launch_cached<__nv_bfloat16>(p, stream)
                             : launch_cached<__half>(p, stream);
}

}  // namespace kda
